"""The choice of experts by score, bias and groups on continuous values: every
row, whichever way 32 bits settle what is nearly equal, has to be a best choice
up to rounding.

Bound: a score's exponential has its argument rounded by |x| 2^-24 and its
factor log2 e by 1.1 |x| 2^-27 (logits here span at most 16 each side, |x| <=
32), the hardware's 2^x and reciprocal add 2^-23 each, the sum of 512 terms over
lanes at most 16 * 2^-23: RTOL = 64 * 2^-23 of the score covers them.  A value v
= s + bias then is known to DELTA = RTOL s + 2^-23 |v|, a group's value to the sum
of its two largest values' DELTA and 2^-23 of itself."""
import itertools

import pytest
import torch

import test_gpu_moe as base

pytestmark = pytest.mark.gpu
RTOL = 64 * 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    mod._load()
    base.M = mod
    yield


def is_best(ids, v, delta, live):
    """Whether ids are the largest v among the live ones, in order, up to delta."""
    got, at = v[ids], live.nonzero()[:, 0]
    if not bool(live[ids].all()) or len(set(ids.tolist())) != len(ids):
        return False
    best = v[at].sort(descending=True).values[:len(ids)]
    # one order statistic is off by at most the largest delta on either side
    return bool(((got - best).abs() <= 2 * delta[at].max()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,topk_groups,k", [(256, 8, 4, 8), (256, 1, 1, 8), (96, 12, 5, 7), (512, 8, 3, 20)])
def test_every_choice_is_a_best_choice(experts, groups, topk_groups, k, score, dtype):
    g = torch.Generator().manual_seed(experts + k)
    tokens = 1500
    l = (1.5 * torch.randn(tokens, experts, generator=g)).clamp(-16, 16).to(base.DT[dtype])
    bias = 0.1 * torch.randn(experts, generator=g)
    w, ids = base.run_route(l, k, bias, score, groups, topk_groups, renorm=False)
    s = base.scores64(l, score)
    v = s + bias.double()
    delta = RTOL * s + 2.0 ** -23 * v.abs()
    top = v.unflatten(-1, (groups, -1)).sort(-1, descending=True).values[..., :2]
    gv = top.sum(-1)
    gdelta = 2 * delta.amax(-1) + 2.0 ** -23 * gv.abs().amax(-1)
    assert (ids >= 0).all() and (ids < experts).all()
    size, unclear, other = experts // groups, 0, 0
    for t in range(tokens):
        order = gv[t].sort(descending=True)
        edge = order.values[topk_groups - 1]
        sure = gv[t] > edge + 2 * gdelta[t]                              # kept whatever rounding does
        near = ((gv[t] - edge).abs() <= 2 * gdelta[t]).nonzero()[:, 0].tolist()
        choices = list(itertools.combinations(near, topk_groups - int(sure.sum())))
        unclear += len(choices) > 1
        ok = False
        for c in choices:
            keep = sure.clone()
            keep[list(c)] = True
            ok = ok or is_best(ids[t], v[t], delta[t], keep.repeat_interleave(size))
        assert ok, (t, ids[t].tolist())
        exact = v[t].masked_fill(~torch.zeros(groups, dtype=torch.bool).index_fill(
            0, order.indices[:topk_groups], True).repeat_interleave(size), float("-inf"))
        other += not torch.equal(exact.sort(descending=True, stable=True).indices[:k], ids[t])
    # the groups, and nearly all choices, are clear: the test is not one of exceptions
    assert unclear <= tokens // 100 and other <= tokens // 20
    ws = s.gather(1, ids)
    assert ((w.double() - ws).abs() <= RTOL * ws).all()


def test_the_check_sees_wrong_choices():
    """A worse expert, a repeated one and one of a dropped group are no best choice."""
    v = torch.linspace(1, 0, 12, dtype=torch.float64)
    delta, live = torch.full((12,), 1e-6, dtype=torch.float64), torch.arange(12) < 8
    ok = lambda *i: is_best(torch.tensor(i), v, delta, live)  # noqa: E731
    assert ok(0, 1, 2) and not ok(0, 1, 3) and not ok(0, 1, 1) and not ok(1, 0, 2) and not ok(0, 1, 9)
    v[1] = v[0] + 1e-7
    assert ok(0, 1, 2) and ok(1, 0, 2)
