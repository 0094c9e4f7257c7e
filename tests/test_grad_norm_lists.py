"""The lists of the gradient norm's and clipping's calls: whatever gives tensors, also those that
nothing else holds, which must live until the kernels are under way."""
import gc
import weakref

import pytest
import torch

import mxfp4_fake_quantization_amd as M
from mxfp4_fake_quantization_amd import adapter_ops

f32 = torch.float32


@pytest.mark.parametrize("call", ["norm", "clip"])
def test_held_until_the_launch(call, monkeypatch):
    """With the library replaced: at its call all of a generator's tensors are there."""
    refs = []

    def made(n):
        for _ in range(n):
            t = torch.zeros(4)
            refs.append(weakref.ref(t))
            yield t
            del t

    class Lib:
        def mxfp4_grad_norm_workspace(self, n, elements):
            return 0

        def alive(self, *args):
            gc.collect()
            assert len(refs) == want and all(r() is not None for r in refs)
            return 0

        mxfp4_grad_norm = mxfp4_grad_clip = alive

    def pack(grads, outs, device, write):
        list(grads)
        if outs is not None:
            list(outs)
        return b"", 0

    monkeypatch.setattr(adapter_ops, "_lib", Lib)
    monkeypatch.setattr(adapter_ops, "_pack", pack)
    monkeypatch.setattr(adapter_ops, "_here", lambda *t: None)
    monkeypatch.setattr(adapter_ops, "_stream", lambda: None)
    want, norm = 3, torch.zeros(1)
    if call == "norm":
        M.mxfp4_grad_norm(made(3), norm)
    else:
        want = 6
        M.mxfp4_grad_clip(made(3), 1.0, norm, outs=made(3))


@pytest.mark.gpu
def test_generators():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M._load()
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = [torch.randn(1000 + i, generator=g, device="cuda") for i in range(40)]
    norm, got = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    outs, want = ([torch.empty_like(t) for t in grads] for _ in range(2))
    M.mxfp4_grad_norm([2 * t for t in grads], norm)
    M.mxfp4_grad_norm((2 * t for t in grads), got)
    assert torch.equal(norm, got)
    M.mxfp4_grad_clip([2 * t for t in grads], 1.0, norm, outs=want)
    M.mxfp4_grad_clip((2 * t for t in grads), 1.0, got, outs=(t for t in outs))
    assert torch.equal(norm, got) and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_clip_takes_torchs_arguments():
    """Every argument of torch.nn.utils.clip_grad_norm_, by name and in its place."""
    import inspect

    from mxfp4_fake_quantization_amd import qat
    theirs = inspect.signature(torch.nn.utils.clip_grad_norm_).parameters
    ours = inspect.signature(qat.clip_grad_norm_).parameters
    assert list(ours) == list(theirs) and all(ours[k].default == theirs[k].default for k in theirs)
    for foreach in (None, True, False):
        assert float(qat.clip_grad_norm_([torch.nn.Parameter(torch.zeros(2))], 1.0, foreach=foreach)) == 0.0
