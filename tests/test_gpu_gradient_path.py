"""A step from tokens to updated parameters with the library's calls alone.

A unit of GPT-2's parameters outside of its matrix products (token and position
embedding, final layer norm): the gathered bf16 buffer is copied out to the
parameters, every rank runs micro-batches through embedding and layer norm and
back, the gradients go straight into the rank's flat fp32 accumulator (or one
flat bf16 contribution), and the sharded update takes them from there. Checked
against the same model in fp64 under torch's autograd on the CPU.

Tolerance of a gradient element: bf16 activations round the embedding's output
(2^-9 relative on average, at most 2^-8), the norm's output is not used by its
gradient, and dx is rounded once more before the embedding's gradient adds it:
each contribution dy xh and dx is off by a few 2^-8 of its own size, so the sum
is off by at most 8 * 2^-8 of the sum of the contributions' magnitudes, which
the test takes from the fp64 run.
"""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import fsdp_sharded_optimizer_flatparameter_amd as zs

pytestmark = pytest.mark.gpu

VOCAB, CTX, DIM, WORLD, MICRO, BATCH, SEQ, SCALE = 61, 16, 40, 2, 2, 4, 16, 8.0
SHAPES = [("wte", (VOCAB, DIM)), ("wpe", (CTX, DIM)), ("ln_f.weight", (DIM,)), ("ln_f.bias", (DIM,))]
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def test_micro_batches_to_updated_shard():
    g = torch.Generator(device="cuda").manual_seed(1)
    numels = [int(np.prod(s)) for _, s in SHAPES]
    offsets, total, padded, shard = zs.zs_flat_layout(numels, WORLD)
    flat = (torch.randn(padded, generator=g, device="cuda") * 0.1).bfloat16()
    flat[offsets[2]:offsets[3]] += 1.0
    params = [torch.empty(s, device="cuda", dtype=torch.bfloat16) for _, s in SHAPES]
    zs.zs_copy_out(flat, zs.ParamTable(params))
    wte, wpe, lw, lb = params

    n = BATCH * SEQ
    positions = torch.arange(n, device="cuda") % SEQ
    h = torch.empty(n, DIM, device="cuda", dtype=torch.bfloat16)
    y, dh, dx = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ws_t = torch.empty(zs.zs_embed_workspace_bytes(n, VOCAB, DIM), device="cuda", dtype=torch.uint8)
    ws_p = torch.empty(zs.zs_embed_workspace_bytes(n, CTX, DIM), device="cuda", dtype=torch.uint8)
    ws_n = torch.empty(zs.zs_layer_norm_workspace_bytes(n, DIM), device="cuda", dtype=torch.uint8)

    ref = [p.double().cpu().requires_grad_() for p in params]
    sizes = [np.zeros(p.shape) for p in params]
    accs, contributions = [], []
    for rank in range(WORLD):
        acc = torch.full((padded,), float("nan"), device="cuda")
        acc[total:] = 0.0  # the tail pad has no parameter
        contribution = torch.zeros(padded, device="cuda", dtype=torch.bfloat16)
        for micro in range(MICRO):
            tokens = torch.randint(0, VOCAB, (n,), generator=g, device="cuda")
            dy = (torch.randn(n, DIM, generator=g, device="cuda") * 0.1).bfloat16()
            zs.zs_embed_forward(wte, tokens, h, scale=SCALE, pos_table=wpe, positions=positions)
            zs.zs_layer_norm_forward(h, lw, lb, y, mean=mean, rstd=rstd)
            for out, first in ((acc, micro == 0), (contribution, micro == 0)):
                gw, gp, gl, gb = (out[o:o + k].view(s) for o, k, (_, s) in zip(offsets, numels, SHAPES))
                zs.zs_layer_norm_backward(dy, h, lw, mean, rstd, dx, dweight=gl, dbias=gb, first=first, workspace=ws_n)
                zs.zs_embed_backward(dx, tokens, gw, scale=SCALE, first=first, workspace=ws_t)
                zs.zs_embed_backward(dx, positions, gp, first=first, workspace=ws_p)
            # the same in fp64, and the contributions' magnitudes
            t, p = tokens.cpu(), positions.cpu()
            hr = F.embedding(t, ref[0]) * SCALE + F.embedding(p, ref[1])
            hr.retain_grad()
            yr = F.layer_norm(hr, (DIM,), ref[2], ref[3], 1e-5)
            yr.backward(dy.double().cpu() / (WORLD * MICRO))
            hg, hd = hr.grad.abs().numpy(), hr.detach().numpy()
            xh = (hd - hd.mean(1, keepdims=True)) / np.sqrt(hd.var(1, keepdims=True) + 1e-5)
            gd = np.abs(dy.double().cpu().numpy()) / (WORLD * MICRO)
            dense = np.abs(hg) + gd * np.abs(lw.double().cpu().numpy()) / np.sqrt(hd.var(1, keepdims=True))
            np.add.at(sizes[0], t.numpy(), SCALE * dense)
            np.add.at(sizes[1], p.numpy(), dense)
            sizes[2] += (gd * (1 + np.abs(xh))).sum(0)
            sizes[3] += gd.sum(0)
        accs.append(acc)
        contributions.append(contribution)

    # the accumulators are the fp32 contributions of the update, rank by rank
    want = np.concatenate([p.grad.numpy().ravel() for p in ref] + [np.zeros(padded - total)])
    size = np.concatenate([s.ravel() for s in sizes] + [np.zeros(padded - total)])
    for rank in range(WORLD):
        lo, hi = rank * shard, (rank + 1) * shard
        for rows in (accs, contributions):
            reduced = torch.empty(shard, device="cuda")
            zs.zs_accumulate_grads([r[lo:hi] for r in rows], reduced, scale=1.0 / MICRO, first=True)
            err = np.abs(reduced.double().cpu().numpy() - want[lo:hi])
            assert np.all(err <= 8 * 2.0 ** -8 * size[lo:hi] + 1e-30), float((err / np.maximum(size[lo:hi], 1e-30)).max())
        master = flat[lo:hi].float()
        fresh = master.clone()
        m, v = torch.zeros(shard, device="cuda"), torch.zeros(shard, device="cuda")
        rows = [r[lo:hi].clone() for r in accs]
        slot = torch.empty(shard, device="cuda", dtype=torch.bfloat16)
        zs.zs_sharded_step(rows, master, m, v, step=1, bf16_out=slot, **HP)
        # the single pass takes them as they are: the same as its two calls
        grad = torch.empty(shard, device="cuda")
        m2, v2 = torch.zeros_like(m), torch.zeros_like(v)
        zs.zs_reduce_grads(rows, grad)
        zs.zs_adamw_step(fresh, m2, v2, grad, step=1, **HP)
        assert torch.equal(master, fresh) and torch.equal(slot, master.bfloat16())
        assert torch.isfinite(master).all() and not torch.equal(master, flat[lo:hi].float())
