"""The product with its epilogue (one to three launches) and the epilogue's
backward (two launches and a workspace) on another stream and in replayed graphs:
the same bits as eager calls, on new data each time."""
import pytest
import torch

import test_gpu_moe_product as product

pytestmark = pytest.mark.gpu
M = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global M
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_fake_quantization_amd as mod
    mod._load()
    M = product.M = mod
    yield


def check(step, fill, outs):
    """step() on a side stream and in a graph against eager calls."""
    fill(0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    step()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(1, 5):
        fill(seed)
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
        assert not all(torch.equal(a, b) for a, b in zip(first, outs))     # new data gave new results


@pytest.mark.parametrize("counts,rows,N,act", [
    ([3, 0, 5], 8, 96, "swiglu"),                          # few rows, K shared by the waves
    ([17, 0, 33, 16, 1, 40], 107, 5471, "swiglu"),         # few rows, columns enough for whole waves
    ([200, 90, 310], 600, 1500, "gelu"),                   # the 128 x 128 tiles alone
    ([256, 70, 300, 65, 512, 799], 2002, 6500, "silu"),    # full rounds and their tail
    (None, 2600, 4000, "swiglu"),                          # and a launch for the last 40 rows
    ([300, 220], 530, 8300, "gelu")])                      # bands; rows past the total
def test_product(counts, rows, N, act):
    K, G, nb = 288, len(counts or [1]), 2 * N if act == "swiglu" else N
    a = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    asc = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
    b = torch.empty(G, nb, K // 2, dtype=torch.uint8, device="cuda")
    bsc = torch.empty(G, nb, K // 32, dtype=torch.uint8, device="cuda")
    bias = torch.empty(G, nb, device="cuda")
    res = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    c, z = torch.zeros_like(res), torch.zeros(rows, nb, dtype=torch.bfloat16, device="cuda")
    gl = None if counts is None else torch.zeros(G, dtype=torch.int64, device="cuda")
    if counts is not None:
        order = torch.tensor(counts, device="cuda")

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        a.random_(0, 0x70, generator=g)                    # E4M3 codes up to 240
        b.random_(0, 256, generator=g)
        asc.random_(110, 116, generator=g)
        bsc.random_(118, 124, generator=g)
        bias.normal_(generator=g)
        res.normal_(generator=g)
        if gl is not None:                                  # the groups change with the data
            gl.copy_(order.roll(seed))

    check(lambda: M.mxfp4_grouped_matmul_act(a, asc, b, bsc, c, group_list=gl, act=act, bias=bias, residual=res, z=z),
          fill, (c, z))


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_backward(act):
    counts, rows, cols = [130, 0, 64, 300], 500, 1000
    zc = cols * (2 if act == "swiglu" else 1)
    dc, z = torch.empty(rows, cols, device="cuda"), torch.empty(rows, zc, device="cuda")
    dz, db = torch.zeros(rows, zc, device="cuda"), torch.zeros(4, zc, device="cuda")
    gl, order = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.tensor(counts, device="cuda")
    from mxfp4_fake_quantization_amd import moe_ops
    need = moe_ops._lib().mxfp4_act_bwd_workspace(moe_ops.ACTIVATIONS[act], rows, cols, 4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dc.normal_(generator=g)
        z.normal_(generator=g)
        gl.copy_(order.roll(seed))

    check(lambda: M.mxfp4_act_bwd(dc, z, dz, act=act, grad_bias=db, group_list=gl, workspace=ws), fill, (dz, db))
