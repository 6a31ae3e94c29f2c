"""The RMS norm and the 8-bit activations in graphs and on streams, at offsets past 32 bits, and the norm's
gradients against differences of the fp64 oracle."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from oracle import rmsnorm as orn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_against_differences():
    rng = np.random.default_rng(1)
    rows, dim, eps = 3, 7, 1e-3
    x, r, w = (rng.standard_normal(s).astype(np.float32) for s in ((rows, dim), (rows, dim), (dim,)))
    dy, dres = (rng.standard_normal((rows, dim)).astype(np.float32) for _ in range(2))
    tx, tr, tw, tdy, tdres = (torch.from_numpy(a).cuda() for a in (x, r, w, dy, dres))
    y, h, rstd = torch.empty_like(tx), torch.empty_like(tx), torch.empty(rows, device="cuda")
    zs.zs_rms_norm_forward(tx, tw, y, eps=eps, residual=tr, residual_out=h, rstd=rstd)
    dh, dw = torch.empty_like(tx), torch.empty(dim, device="cuda")
    ws = torch.empty(zs.zs_rms_norm_workspace_bytes(rows, dim), device="cuda", dtype=torch.uint8)
    zs.zs_rms_norm_backward(tdy, h, tw, rstd, dh, dresidual=tdres, dweight=dw, first=True, workspace=ws)
    x, w, e = x.astype(np.float64), w.astype(np.float64), 1e-5

    def value():
        out, hh, _ = orn.rms_norm_forward(x, w, r, eps)
        return (out * dy).sum() + (hh * dres).sum()

    for a, d in ((x, dh), (w, dw)):
        d = d.double().cpu().numpy()
        for at in np.ndindex(a.shape):
            a[at] += e
            up = value()
            a[at] -= 2 * e
            down = value()
            a[at] += e
            # differences are good to e^2 times third derivatives (rstd up to 3) and 1e-15 / e; h and rstd are rounded
            assert abs((up - down) / (2 * e) - d[at]) < 1e-7 + 500 * U


@pytest.mark.parametrize("rows,dim", [(900, 1000), (3, 4096)])
def test_graph_and_streams(rows, dim):
    g = torch.Generator(device="cuda").manual_seed(rows)

    def new(dtype=torch.bfloat16, r=rows, d=dim):
        return torch.randn(r, d, generator=g, device="cuda").to(dtype)

    x, r, dy, w = new(), new(torch.float32), new(), new(torch.float32, 1)[0]
    size = zs.zs_rms_norm_workspace_bytes(rows, dim)

    def buffers():
        return dict(y=torch.empty_like(x), h=torch.empty_like(r), rstd=torch.empty(rows, device="cuda"),
                    codes=torch.empty(rows, dim, device="cuda", dtype=torch.uint8),
                    scales=torch.empty(rows, -(-dim // 128), device="cuda"), dh=torch.empty_like(r),
                    dw=torch.zeros(dim, device="cuda"), ws=torch.empty(size, device="cuda", dtype=torch.uint8),
                    back=torch.empty_like(x))

    def run(b, stream=None):
        zs.zs_rms_norm_forward(x, w, b["y"], residual=r, residual_out=b["h"], rstd=b["rstd"], stream=stream)
        zs.zs_activation_pack(b["h"], b["codes"], b["scales"], stream=stream)
        zs.zs_activation_unpack(b["codes"], b["scales"], b["back"], stream=stream)
        zs.zs_rms_norm_backward(dy, b["codes"], w, b["rstd"], b["dh"], scales=b["scales"], dresidual=r, dweight=b["dw"],
                                workspace=b["ws"], stream=stream)

    captured, eager = buffers(), buffers()
    run(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(captured)
    side = torch.cuda.Stream()
    for _ in range(4):
        x.copy_(new())
        r.copy_(new(torch.float32))
        captured["dw"].zero_()
        eager["dw"].zero_()
        torch.cuda.synchronize()
        graph.replay()
        run(eager, side)
        torch.cuda.synchronize()
        for k in captured:
            if k != "ws":
                assert torch.equal(captured[k], eager[k]), k


def test_offsets_past_32_bits():
    rows, dim = 300001, 8192
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16).normal_(0, 1, generator=g)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    codes, scales = torch.empty(rows, dim, device="cuda", dtype=torch.uint8), torch.empty(rows, dim // 128, device="cuda")
    zs.zs_rms_norm_forward(x, None, y, codes=codes, scales=scales, rstd=rstd)
    at = torch.tensor([0, 1, 262143, 262144, rows - 2, rows - 1], device="cuda")
    one = torch.empty(len(at), dim, device="cuda", dtype=torch.bfloat16)
    c1, s1 = torch.empty(len(at), dim, device="cuda", dtype=torch.uint8), torch.empty(len(at), dim // 128, device="cuda")
    zs.zs_rms_norm_forward(x[at], None, one, codes=c1, scales=s1)
    assert torch.equal(y[at], one) and torch.equal(codes[at], c1) and torch.equal(scales[at], s1)
    zs.zs_activation_unpack(codes, scales, y)
    zs.zs_activation_unpack(c1, s1, one)
    assert torch.equal(y[at], one)
    dw = torch.empty(dim, device="cuda")
    ws = torch.empty(zs.zs_rms_norm_workspace_bytes(rows, dim), device="cuda", dtype=torch.uint8)
    dh = torch.empty_like(x)
    zs.zs_rms_norm_backward(y, codes, None, rstd, dh, scales=scales, dweight=dw, first=True, workspace=ws)
    d1 = torch.empty_like(one)
    zs.zs_rms_norm_backward(y[at], c1, None, rstd[at], d1, scales=s1)
    assert torch.equal(dh[at], d1)
    zs.zs_activation_pack(x, codes, scales)
    zs.zs_activation_pack(x[at], c1, s1)
    assert torch.equal(codes[at], c1) and torch.equal(scales[at], s1)
