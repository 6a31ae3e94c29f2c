"""One micro-batch through the embedding and layer norm entry points of the C
ABI by a standalone program (no Python or PyTorch in the process that calls the
library), checked step by step against the oracle on the program's own
intermediate results: the tolerances are those of test_gpu_embedding.py and
test_gpu_layer_norm.py, whose checks it uses.
"""
import os
import subprocess

import numpy as np
import pytest
import torch

import test_gpu_embedding as emb
import test_gpu_layer_norm as norm
from oracle import embedding as oe

pytestmark = pytest.mark.gpu

DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "zs_rows_driver")


@pytest.mark.parametrize("n,vocab,ctx,dim", [(1, 5, 3, 7), (50, 61, 16, 40), (600, 300, 64, 769), (3000, 1003, 100, 130)])
def test_micro_batch_matches_the_oracle(tmp_path, n, vocab, ctx, dim):
    scale = 1.5
    g = torch.Generator().manual_seed(n)
    tokens = torch.randint(-1, vocab + 1, (n,), generator=g)
    positions = torch.arange(n) % (ctx + 1)  # the last one is outside of the table

    def normal(*shape):
        return torch.randn(*shape, generator=g).bfloat16()

    table, pos, w, b, dy = normal(vocab, dim), normal(ctx, dim), normal(dim), normal(dim), normal(n, dim)
    src, dst = tmp_path / "in.bin", tmp_path / "out.bin"
    with open(src, "wb") as f:
        f.write(np.array([n, vocab, ctx, dim], np.int64).tobytes() + np.array([scale], np.float64).tobytes())
        for t in (tokens, positions):
            f.write(t.numpy().tobytes())
        for t in (table, pos, w, b, dy):
            f.write(t.view(torch.int16).numpy().tobytes())
    print(f"zs_rows_driver n={n} vocab={vocab} ctx={ctx} dim={dim}", flush=True)
    res = subprocess.run([DRIVER, str(src), str(dst)], capture_output=True, text=True, timeout=100)
    assert res.returncode == 0, (res.returncode, res.stdout, res.stderr)
    raw, at = open(dst, "rb").read(), 0

    def take(dtype, *shape):
        nonlocal at
        t = torch.frombuffer(bytearray(raw[at:at + int(np.prod(shape)) * (2 if dtype is torch.bfloat16 else 4)]), dtype=dtype)
        at += t.numel() * t.element_size()
        return t.reshape(shape).cuda()

    bf, f32 = torch.bfloat16, torch.float32
    h, y, mean, rstd = take(bf, n, dim), take(bf, n, dim), take(f32, n), take(f32, n)
    dx, dw, db, dtable, dpos = take(bf, n, dim), take(f32, dim), take(f32, dim), take(f32, vocab, dim), take(bf, ctx, dim)
    assert at == len(raw)

    want = oe.embed_forward(emb.f64(table), tokens.tolist(), scale, emb.f64(pos), positions.tolist())
    half = emb.HALF[bf]
    assert np.all(np.abs(emb.f64(h) - want) <= (emb.U + half + emb.U * half) * np.abs(want))
    norm.check_forward(h, w, b, y, mean, rstd, 1e-5)
    norm.check_backward(dy, h, w, mean, rstd, dx, dw, db, None, None)
    # the table's gradient twice: the second call adds to the first one's fp32 result, which is off by
    # (m + 2) u of the magnitudes and its own rounding at most, on top of the bound of one call
    total, size = oe.embed_backward(emb.f64(dx), tokens.tolist(), vocab, scale)
    m = np.bincount([t for t in tokens.tolist() if 0 <= t < vocab], minlength=vocab)[:, None]
    tol = (2 * (m + 2) * emb.U * 2 * size + 2 * emb.U * 2 * np.abs(total)) * (1 + 2.0 ** -7)
    assert np.all(np.abs(emb.f64(dtable) - 2 * total) <= tol)
    emb.check_backward(dx, positions, dpos, None, 1.0, -1, True)
