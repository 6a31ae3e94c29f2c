"""A cap on the number of workgroups changes no result of the embedding and
layer norm calls: with a few workgroups every kernel that strides over its work
goes through many turns (reuse of its LDS, offsets of later turns), in a child
process each, bitwise against the default launches.

Lookups with and without positions; gradients by each way of sorting, with a
table above 100 MB (zeros by marks), with up to 64 tokens, with runs over
groups of chunks and rows that are streamed; norms.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import numpy as np
import torch
sys.path.insert(0, sys.argv[2])
import fsdp_sharded_optimizer_flatparameter_amd as zs

BF, F32 = torch.bfloat16, torch.float32
out = {}
def h(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.int16).numpy() if t.dtype == BF else t.view(torch.int32).numpy()
def normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)
for n, vocab, dim, dt, gdt, first in ((60, 300, 1100, BF, F32, True), (9001, 701, 513, BF, BF, False),
                                      (20000, 70001, 401, F32, F32, True), (40000, 70001, 403, BF, F32, True),
                                      (40000, 5000, 7, F32, BF, False), (140000, 701, 520, BF, F32, True)):
    print(n, vocab, dim, flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    tokens = torch.randint(-1, vocab + 1, (n,), generator=g, device="cuda")
    tokens[n // 4: n // 4 * 3] = 7  # a run over half of the chunks
    tokens = tokens[torch.randperm(n, generator=g, device="cuda")]
    table, pos = normal(g, vocab, dim, dtype=dt), normal(g, 64, dim, dtype=dt)
    rows = torch.empty(n, dim, device="cuda", dtype=gdt)
    for with_pos in (False, True):
        zs.zs_embed_forward(table, tokens, rows, scale=1.5, pos_table=pos if with_pos else None,
                            positions=torch.arange(n, device="cuda") % 66 if with_pos else None)
        out[f"rows{n}_{dim}_{with_pos}"] = h(rows)
    dout = normal(g, n, dim, dtype=dt)
    grad = torch.full((vocab, dim), float("nan"), device="cuda", dtype=gdt) if first else normal(g, vocab, dim, dtype=gdt)
    ws = torch.full((zs.zs_embed_workspace_bytes(n, vocab, dim),), 0xFF, device="cuda", dtype=torch.uint8)
    zs.zs_embed_backward(dout, tokens, grad, scale=0.5, first=first, workspace=ws)
    out[f"grad{n}_{dim}"] = h(grad)
for rows, dim, dt in ((5000, 769, BF), (3001, 4100, F32), (300, 33003, BF)):
    print(rows, dim, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy, w = normal(g, rows, dim, dtype=dt), normal(g, rows, dim, dtype=dt), normal(g, dim, dtype=dt)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, dw, db = (torch.empty(k, device="cuda") for k in (rows, rows, dim, dim))
    ws = torch.empty(zs.zs_layer_norm_workspace_bytes(rows, dim), device="cuda", dtype=torch.uint8)
    zs.zs_layer_norm_forward(x, w, w, y, mean=mean, rstd=rstd)
    zs.zs_layer_norm_backward(dy, x, w, mean, rstd, dx, dweight=dw, dbias=db, first=True, workspace=ws)
    for k, t in (("y", y), ("dx", dx), ("mean", mean), ("rstd", rstd), ("dw", dw), ("db", db)):
        out[f"{k}{rows}"] = h(t)
np.savez(sys.argv[1], **out)
"""


def _run(tmp_path, cap):
    env = {k: v for k, v in os.environ.items() if not k.startswith("ZS_")}
    if cap:
        env.update(ZS_TUNING="1", ZS_GRID_CAP=str(cap))
    path = str(tmp_path / f"cap{cap}.npz")
    print(f"grid cap {cap}", flush=True)
    res = subprocess.run([sys.executable, "-c", CHILD, path, ROOT], env=env, capture_output=True, text=True,
                         timeout=100, cwd=ROOT)
    assert res.returncode == 0, (cap, res.stdout[-2000:], res.stderr[-2000:])
    return dict(np.load(path))


def test_a_grid_cap_changes_no_result(tmp_path):
    base = _run(tmp_path, 0)
    assert all(np.count_nonzero(v) for v in base.values())
    for cap in (5, 64):
        got = _run(tmp_path, cap)
        assert got.keys() == base.keys()
        for key in base:
            assert np.array_equal(got[key], base[key]), (cap, key)
