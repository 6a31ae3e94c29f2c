"""One micro-batch through the RMS norm, 8-bit activation and loss entry points of
the C ABI by a standalone program (no Python or PyTorch in the process that calls
the library), checked step by step against the oracle on the program's own
intermediate results, with the checks and tolerances of test_gpu_rms_norm.py,
test_gpu_activation.py and test_gpu_head_loss.py.
"""
import os
import subprocess

import numpy as np
import pytest
import torch

import test_gpu_activation as act
import test_gpu_head_loss as head
import test_gpu_rms_norm as norm
from oracle import activation as oa

pytestmark = pytest.mark.gpu

DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "zs_head_driver")


@pytest.mark.parametrize("n,vocab,dim", [(1, 5, 7), (50, 61, 40), (300, 700, 264)])
def test_micro_batch_matches_the_oracle(tmp_path, n, vocab, dim):
    g = torch.Generator().manual_seed(n)
    labels = torch.randint(-1, vocab + 1, (n,), generator=g).to(torch.int32)
    x, w, table = (torch.randn(*s, generator=g).bfloat16() for s in ((n, dim), (dim,), (vocab, dim)))
    table *= 0.25
    r = torch.randn(n, dim, generator=g)
    src, dst = tmp_path / "in.bin", tmp_path / "out.bin"
    with open(src, "wb") as f:
        f.write(np.array([n, vocab, dim], np.int64).tobytes() + labels.numpy().tobytes())
        f.write(x.view(torch.int16).numpy().tobytes() + r.numpy().tobytes())
        f.write(w.view(torch.int16).numpy().tobytes() + table.view(torch.int16).numpy().tobytes())
    print(f"zs_head_driver n={n} vocab={vocab} dim={dim}", flush=True)
    res = subprocess.run([DRIVER, str(src), str(dst)], capture_output=True, text=True, timeout=100)
    assert res.returncode == 0, (res.returncode, res.stdout, res.stderr)
    raw, at = open(dst, "rb").read(), 0

    def take(dtype, *shape):
        nonlocal at
        size = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        t = torch.frombuffer(bytearray(raw[at:at + size]), dtype=dtype)
        at += size
        return t.reshape(shape).cuda()

    bf, f32, u8, blocks = torch.bfloat16, torch.float32, torch.uint8, -(-dim // 128)
    h, y, codes, scales, rstd = take(f32, n, dim), take(bf, n, dim), take(u8, n, dim), take(f32, n, blocks), take(f32, n)
    kept, kept_s, values = take(u8, n, dim), take(f32, n, blocks), take(f32, n, dim)
    loss, lse, dy, dhead = take(f32, n), take(f32, n), take(bf, n, dim), take(f32, vocab, dim)
    dh, dw = take(f32, n, dim), take(f32, dim)
    assert at == len(raw)

    x, w, r, table, labels = (t.cuda() for t in (x, w, r, table, labels))
    norm.check_forward(x, w, r, 1e-5, y, h, rstd, codes, scales)
    act.check(h, kept, kept_s)
    h64 = oa.unpack(kept.cpu().numpy(), kept_s.cpu().numpy())
    np.testing.assert_array_equal(values.double().cpu().numpy(), h64)
    head.check_forward(y, table, labels, loss, lse)
    head.check_backward(y, table, labels, lse, np.full(n, np.float32(1) / np.float32(n), np.float64), dy, dhead, dhead, True)
    norm.check_backward(dy, h64, w, rstd, r, dh, dw, None, True)
