"""From tokens to a loss and an updated shard with the library's calls alone.

A unit with a tied table and two RMS norms, as a Llama-like list has them: tokens
are looked up, normed, added to the residual stream, normed again, and the table
is the head whose loss and gradient close the pass. The head's and the lookup's
gradients go into the same fp32 accumulator, beside the norms'; what the second
norm read may be kept in 8 bits for the backward pass. Checked against the same
model in fp64: under autograd where the kept values are plain, with the kept
values in the norm's backward formula where they are in 8 bits.

Tolerance: fp32 throughout. Each of the six calls on the way of a gradient adds
at most 200 roundings (64 + 6 + 6 for a row's sums, 61 + 32 for the head's) of
terms whose magnitudes are at most 16 times the gradient's norm: 1200 * 16 u < 2^-9
of the norm at the very worst, and as roundings are of both signs their norm
stays below sqrt(1200) * 16 u = 2^-15 of it.
"""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import fsdp_sharded_optimizer_flatparameter_amd as zs

pytestmark = pytest.mark.gpu

VOCAB, DIM, WORLD, MICRO, N, SCALE = 61, 200, 2, 2, 96, 8.0
SHAPES = [("embed_tokens", (VOCAB, DIM)), ("norm1.weight", (DIM,)), ("norm2.weight", (DIM,))]
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
EPS = 1e-5


def test_loss_and_update():
    g = torch.Generator(device="cuda").manual_seed(1)
    numels = [int(np.prod(s)) for _, s in SHAPES]
    offsets, total, padded, shard = zs.zs_flat_layout(numels, WORLD)
    flat = (torch.randn(padded, generator=g, device="cuda") * 0.05).bfloat16()
    flat[offsets[1]:total] += 1.0
    gathered = [torch.empty(s, device="cuda", dtype=torch.bfloat16) for _, s in SHAPES]
    zs.zs_copy_out(flat, zs.ParamTable(gathered))
    table, w1, w2 = (p.float() for p in gathered)

    def f32(*shape):
        return torch.full(shape, float("nan"), device="cuda")

    h0, y1, h1, y2, dy2, dh1, dh0 = (f32(N, DIM) for _ in range(7))
    r1, r2, loss, lse = (f32(N) for _ in range(4))
    codes, scales = torch.empty(N, DIM, device="cuda", dtype=torch.float8_e4m3fn), f32(N, -(-DIM // 128))
    kept = f32(N, DIM)
    ws_e = torch.empty(zs.zs_embed_workspace_bytes(N, VOCAB, DIM), device="cuda", dtype=torch.uint8)
    ws_n = torch.empty(zs.zs_rms_norm_workspace_bytes(N, DIM), device="cuda", dtype=torch.uint8)
    ws_l = torch.empty(max(zs.zs_linear_cross_entropy_workspace_bytes(N, VOCAB, DIM, torch.float32),
                           zs.zs_linear_cross_entropy_workspace_bytes(N, VOCAB, DIM, torch.float32, torch.float32)),
                       device="cuda", dtype=torch.uint8)

    for in_8_bits in (False, True):
        accs = []
        want = [torch.zeros(s, dtype=torch.float64) for _, s in SHAPES]
        for rank in range(WORLD):
            acc = torch.full((padded,), float("nan"), device="cuda")
            acc[total:] = 0.0
            gt, g1, g2 = (acc[o:o + k].view(s) for o, k, (_, s) in zip(offsets, numels, SHAPES))
            for micro in range(MICRO):
                tokens = torch.randint(0, VOCAB, (N,), generator=g, device="cuda")
                labels = tokens.roll(-1).clone()
                labels[::7] = -100
                count = int((labels >= 0).sum())
                first = micro == 0
                zs.zs_embed_forward(table, tokens, h0, scale=SCALE)
                zs.zs_rms_norm_forward(h0, w1, y1, eps=EPS, rstd=r1)
                zs.zs_rms_norm_forward(y1, w2, y2, eps=EPS, residual=h0, residual_out=h1, rstd=r2)
                zs.zs_linear_cross_entropy_forward(y2, table, labels, loss, lse=lse, workspace=ws_l)
                zs.zs_linear_cross_entropy_backward(y2, table, labels, lse, dy2, gt, scale=1.0 / count, first=first,
                                                    workspace=ws_l)
                if in_8_bits:
                    zs.zs_activation_pack(h1, codes, scales)
                    zs.zs_activation_unpack(codes, scales, kept)
                    zs.zs_rms_norm_backward(dy2, codes, w2, r2, dh1, scales=scales, dweight=g2, first=first, workspace=ws_n)
                else:
                    zs.zs_rms_norm_backward(dy2, h1, w2, r2, dh1, dweight=g2, first=first, workspace=ws_n)
                zs.zs_rms_norm_backward(dh1, h0, w1, r1, dh0, dresidual=dh1, dweight=g1, first=first, workspace=ws_n)
                zs.zs_embed_backward(dh0, tokens, gt, scale=SCALE, first=False, workspace=ws_e)

                # the same in fp64
                p = [t.double().cpu().requires_grad_() for t in (table, w1, w2)]
                t, lab = tokens.cpu(), labels.cpu()
                x0 = F.embedding(t, p[0]) * SCALE
                x0.retain_grad()
                x1 = x0 + F.rms_norm(x0, (DIM,), p[1], EPS)
                x1.retain_grad()
                if in_8_bits:
                    # the backward pass sees the kept values, the forward's statistics and dy2
                    with torch.no_grad():
                        rs = 1 / torch.sqrt((x1 * x1).mean(1, keepdim=True) + EPS)
                    n2 = F.rms_norm(x1, (DIM,), p[2], EPS).detach().requires_grad_()
                    each = F.cross_entropy(n2 @ p[0].t(), lab, ignore_index=-100, reduction="none")
                    (each.sum() / count).backward()
                    xh = kept.double().cpu() * rs
                    gw = n2.grad * p[2].detach()
                    p[2].grad = (n2.grad * xh).sum(0)
                    x1.backward(rs * (gw - xh * (gw * xh).mean(1, keepdim=True)))
                else:
                    n2 = F.rms_norm(x1, (DIM,), p[2], EPS)
                    each = F.cross_entropy(n2 @ p[0].t(), lab, ignore_index=-100, reduction="none")
                    (each.sum() / count).backward()
                for a, b in zip(want, p):
                    a += b.grad / (WORLD * MICRO)
                err = (loss.double().cpu() - each.detach()).abs().max()
                assert err < 2.0 ** -13, err  # logits up to 16 in 200 additions
            accs.append(acc)

        flat_want = torch.cat([w.flatten() for w in want] + [torch.zeros(padded - total, dtype=torch.float64)])
        for rank in range(WORLD):
            lo, hi = rank * shard, (rank + 1) * shard
            reduced = torch.empty(shard, device="cuda")
            zs.zs_accumulate_grads([r[lo:hi] for r in accs], reduced, scale=1.0 / MICRO, first=True)
            err = (reduced.double().cpu() - flat_want[lo:hi]).norm() / flat_want[lo:hi].norm()
            assert err < 2.0 ** -15, err
            master = flat[lo:hi].float()
            m, v = torch.zeros(shard, device="cuda"), torch.zeros(shard, device="cuda")
            slot = torch.empty(shard, device="cuda", dtype=torch.bfloat16)
            zs.zs_sharded_step([r[lo:hi].clone() for r in accs], master, m, v, step=1, bf16_out=slot, **HP)
            assert torch.isfinite(master).all() and torch.equal(slot, master.bfloat16())
            assert not torch.equal(master, flat[lo:hi].float())
