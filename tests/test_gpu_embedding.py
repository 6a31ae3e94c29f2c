"""Embedding lookup and its gradient against the fp64 oracle.

Tolerances, u = 2^-24 (half a step of fp32), h = half a step of the result's
type (2^-24 for fp32, 2^-8 for bf16):
  * forward: the product (or the fused product and sum) is one fp32 rounding
    and the store another: |err| <= (u + h + u h) |out|. With a bf16 result the
    fp32 rounding may also move a value over a tie, which is inside u + h.
  * backward: a token's m rows are added in fp32, whatever the grouping, in at
    most m roundings on the way of any one of them, then come the scale, the
    old value and the store: |err| <= (m + 2) u (|old| + |scale| sum |dout|)
    plus h |grad|, with one more factor (1 + 2^-7) for the products of those.
Results below the smallest normal number do not occur (inputs are near 1).
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from oracle import bf16 as obf16
from oracle import embedding as oe

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IT = {"i32": torch.int32, "i64": torch.int64}
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def matrix(g, rows, dim, dtype, gap=0, fill=None):
    """[rows, dim] view of a wider buffer whose gaps hold NaN."""
    big = torch.full((rows, dim + gap), float("nan"), device="cuda", dtype=DT[dtype])
    v = big[:, :dim]
    v.copy_(torch.randn(rows, dim, generator=g, device="cuda") if fill is None else torch.full((), fill))
    return big, v


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def gaps_untouched(big, dim):
    return bool(torch.isnan(big[:, dim:]).all())


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


@pytest.mark.parametrize("n", [1, 2, 65, 300])
@pytest.mark.parametrize("dim", [1, 3, 8, 64, 511, 513, 769, 1032, 2056])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_forward(n, dim, dtype, out):
    g = gen(n * 10007 + dim)
    vocab, gap = 37, (n + dim) % 3
    _, table = matrix(g, vocab, dim, dtype, gap)
    _, pos = matrix(g, 9, dim, dtype, 2 * gap)
    big, o = matrix(g, n, dim, out, gap, fill=float("nan"))
    tokens = torch.randint(-2, vocab + 3, (n,), generator=g, device="cuda").to(IT["i32" if dim % 2 else "i64"])
    positions = torch.randint(-1, 11, (n,), generator=g, device="cuda").to(tokens.dtype)
    for scale, with_pos in ((1.0, False), (27.75, False), (-0.5, True)):
        zs.zs_embed_forward(table, tokens, o, scale=scale, pos_table=pos if with_pos else None,
                            positions=positions if with_pos else None)
        want = oe.embed_forward(f64(table), tokens.tolist(), scale, f64(pos) if with_pos else None, positions.tolist())
        h = HALF[DT[out]]
        err = np.abs(f64(o) - want)
        assert np.all(err <= (U + h + U * h) * np.abs(want)), (scale, float(err.max()))
        assert gaps_untouched(big, dim)


def test_forward_rounds_every_pattern_to_nearest_even():
    # all upper halves of an fp32 pattern with lower halves around the ties: subnormals, overflow, NaN
    hi = torch.arange(65536, device="cuda", dtype=torch.int64) << 16
    low = torch.tensor([0, 1, 0x7FFF, 0x8000, 0x8001, 0xFFFF], device="cuda")
    table = (hi[:, None] + low[None, :]).to(torch.uint32).view(torch.float32)
    ids = torch.arange(65536, device="cuda", dtype=torch.int32)
    out = torch.empty(65536, 6, device="cuda", dtype=torch.bfloat16)
    zs.zs_embed_forward(table, ids, out)
    got = out.view(torch.int16).cpu().numpy().view(np.uint16)
    x = table.cpu().numpy()
    nan = np.isnan(x)
    assert np.array_equal(got[~nan], obf16.to_bf16_bits(x)[~nan])
    assert np.all((got[nan] & 0x7FC0) == 0x7FC0)  # quiet, and with its sign
    assert np.array_equal(got[nan] >> 15, (x.view(np.uint32)[nan] >> 31).astype(np.uint16))
    same = torch.empty(65536, 6, device="cuda")
    zs.zs_embed_forward(table, ids, same)
    assert np.array_equal(bits(same).cpu().numpy()[~nan], x.view(np.int32)[~nan])


def test_forward_shapes_and_nothing_to_do():
    g = gen(5)
    _, table = matrix(g, 10, 24, "bf16")
    tokens = torch.randint(0, 10, (2, 3), generator=g, device="cuda")
    out = torch.empty(2, 3, 24, device="cuda", dtype=torch.bfloat16)
    zs.zs_embed_forward(table, tokens, out)
    assert torch.equal(out, table[tokens])
    zs.zs_embed_forward(table, tokens[:0].reshape(0), out.reshape(6, 24)[:0])
    zs.zs_embed_forward(table[:0], tokens, out)  # an empty table selects zeros everywhere
    assert torch.count_nonzero(out) == 0


def test_forward_special_values():
    table = torch.tensor([[float("inf"), 1.0], [float("nan"), -0.0], [3e38, -3e38]], device="cuda")
    tokens = torch.tensor([0, 1, 2, 5], device="cuda")
    out = torch.empty(4, 2, device="cuda", dtype=torch.bfloat16)
    zs.zs_embed_forward(table, tokens, out, scale=2.0)
    want = torch.tensor([[float("inf"), 2.0], [float("nan"), -0.0], [float("inf"), float("-inf")], [0, 0]])
    assert torch.equal(out.float().cpu().nan_to_num(7.0, 9.0, -9.0), want.nan_to_num(7.0, 9.0, -9.0))


@pytest.mark.parametrize("far", ["table", "out"])
def test_forward_offsets_beyond_32_bits(far):
    # rows 8 MiB apart: the last row starts past 2^32 bytes (and 2^31 elements)
    ld, rows, dim = 1 << 22, 600, 40
    buf = torch.empty(rows * ld, device="cuda", dtype=torch.bfloat16)
    wide = buf.view(rows, ld)[:, :dim]
    narrow = torch.randn(rows, dim, device="cuda").bfloat16()
    ids = torch.arange(rows - 1, -1, -1, device="cuda")
    if far == "table":
        wide.copy_(narrow)
        out = torch.empty_like(narrow)
        zs.zs_embed_forward(wide, ids, out)
    else:
        zs.zs_embed_forward(narrow, ids, wide)
        out = wide
    assert torch.equal(out, narrow.flip(0))


def make_tokens(g, n, vocab, kind, index):
    if kind == "equal":
        t = torch.full((n,), vocab - 1, device="cuda")
    elif kind == "ignored":
        t = torch.full((n,), -100, device="cuda")
        t[1::2] = vocab
    elif kind == "runs":  # a few tokens share all places: runs that cross many chunks
        t = torch.randint(0, min(vocab, 3), (n,), generator=g, device="cuda") * (vocab // 3)
        t.clamp_(max=vocab - 1)
    elif kind == "distinct":
        t = torch.randperm(max(n, vocab), generator=g, device="cuda")[:n] % vocab
    else:
        t = torch.randint(-1, vocab + 1, (n,), generator=g, device="cuda")
    return t.to(IT[index])


def run_backward(dout, tokens, grad, **kw):
    ws = torch.full((zs.zs_embed_workspace_bytes(tokens.numel(), *grad.shape),), 0xA5, device="cuda", dtype=torch.uint8)
    zs.zs_embed_backward(dout, tokens, grad, workspace=ws, **kw)


def check_backward(dout, tokens, grad, before, scale, padding, first):
    vocab = grad.shape[0]
    t = [x if x != padding else -1 for x in tokens.tolist()]
    want, size = oe.embed_backward(f64(dout), t, vocab, scale, old=None if first else f64(before))
    m = np.bincount([x for x in t if 0 <= x < vocab], minlength=vocab)[:, None]
    tol = ((m + 2) * U * size + HALF[grad.dtype] * np.abs(want)) * (1 + 2.0 ** -7)
    err = np.abs(f64(grad) - want)
    assert np.all(err <= tol), f"{(err > tol).sum()} off, worst {np.max(err / np.maximum(tol, 1e-300))} of the tolerance"
    untouched = torch.from_numpy(m[:, 0] == 0).cuda()
    if first:
        assert torch.count_nonzero(bits(grad[untouched])) == 0  # +0
    else:
        assert torch.equal(bits(grad[untouched]), bits(before[untouched]))


@pytest.mark.parametrize("kind", ["mixed", "equal", "ignored", "runs", "distinct"])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (1, 300, 70), (2, 5, 3), (7, 2, 9), (64, 1, 513), (65, 255, 8),
                                         (129, 256, 130), (513, 600, 17), (1000, 511, 769), (2049, 70000, 24),
                                         (5000, 1003, 65), (300, 300000, 33)])
def test_backward(kind, n, vocab, dim):
    k = (n + vocab + dim) % 4
    dtype, gdt = [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")][k]
    g = gen(n * 31 + dim)
    gap = k
    big_d, dout = matrix(g, n, dim, dtype, gap)
    tokens = make_tokens(g, n, vocab, kind, "i32" if k % 2 else "i64")
    for first, scale, padding in ((True, 1.0, -1), (False, 27.75, 0)):
        big, grad = matrix(g, vocab, dim, gdt, gap, fill=float("nan") if first else None)
        before = grad.clone()
        run_backward(dout, tokens, grad, scale=scale, padding_idx=padding, first=first)
        check_backward(dout, tokens, grad, before, scale, padding, first)
        assert gaps_untouched(big, dim)


@pytest.mark.parametrize("n", [4095, 4096, 4097, 16383, 16384, 16385, 40000, 140000])
@pytest.mark.parametrize("kind", ["mixed", "runs", "equal"])
def test_backward_many_tokens(n, kind):
    # both ways of sorting, around the sizes where one takes over from the other
    g = gen(n)
    vocab, dim = 9001, 10
    _, dout = matrix(g, n, dim, "f32")
    tokens = make_tokens(g, n, vocab, kind, "i64")
    grad = torch.empty(vocab, dim, device="cuda")
    run_backward(dout, tokens, grad, first=True)
    check_backward(dout, tokens, grad, None, 1.0, -1, True)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 1023, 1024, 1025, 2047, 2048, 2049, 32767, 32768, 32769])
@pytest.mark.parametrize("vocab", [255, 510, 511, 512, 2046, 2047, 2048, 262143, 262144])
def test_backward_around_the_sorts_limits(n, vocab, first):
    # where the sort changes its launches, its digits and their number
    g = gen(n + vocab)
    _, dout = matrix(g, n, 3, "f32")
    tokens = make_tokens(g, n, vocab, "mixed", "i32" if vocab % 2 else "i64")
    tokens[n // 2] = vocab - 1  # the largest key
    _, grad = matrix(g, vocab, 3, "f32", fill=float("nan") if first else None)
    before = grad.clone()
    run_backward(dout, tokens, grad, first=first)
    check_backward(dout, tokens, grad, before, 1.0, -1, first)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n", [66, 2047, 2049, 8191, 8192, 8193, 16383, 16385])
@pytest.mark.parametrize("vocab", [1, 2, 8, 9, 2048, 2049, 65537, 131072, 131073, 262143, 262145])
def test_backward_around_the_ranges_of_the_sort(n, vocab, first):
    # where a range of keys grows, the last one is short, and one or two workgroups fit on a compute unit
    g = gen(n + 3 * vocab)
    _, dout = matrix(g, n, 2, "f32")
    tokens = make_tokens(g, n, vocab, "mixed" if vocab % 2 else "distinct", "i32" if n % 2 else "i64")
    tokens[n // 3: n // 3 + n // 4] = vocab // 2  # one that fills whole waves, and some without a row
    tokens[n // 2 + n // 4:: 3] = -100
    tokens[-1], tokens[0] = vocab - 1, 0
    _, grad = matrix(g, vocab, 2, "f32", fill=float("nan") if first else None)
    before = grad.clone()
    run_backward(dout, tokens, grad, first=first)
    check_backward(dout, tokens, grad, before, 1.0, -1, first)


@pytest.mark.parametrize("n", [65, 1500, 2048, 5000, 8192, 12000, 16384])
@pytest.mark.parametrize("kind", ["mixed", "runs", "equal", "ignored"])
def test_backward_has_one_order_however_it_is_sorted(n, kind):
    # a vocabulary too large for the sort by ranges: the same entries, the same sums, bit for bit
    g = gen(n + 11)
    _, dout = matrix(g, n, 5, "f32")
    tokens = make_tokens(g, n, 700, kind, "i64").clamp_(max=699)
    grads = [torch.zeros(vocab, 5, device="cuda") for vocab in (700, 300001)]
    for grad in grads:
        run_backward(dout, tokens, grad)
    assert torch.equal(bits(grads[0]), bits(grads[1][:700]))
    assert torch.count_nonzero(grads[1][700:]) == 0


def reference_on_the_gpu(dout, tokens, grad_shape, before, scale):
    """The gradient and sum of magnitudes in fp64 (adding in another order is 2^-53 of the magnitudes)."""
    keep = (tokens >= 0) & (tokens < grad_shape[0])
    want, size = (torch.zeros(grad_shape, device="cuda", dtype=torch.float64) for _ in range(2))
    rows = dout.double()[keep] * scale
    want.index_add_(0, tokens[keep].long(), rows)
    size.index_add_(0, tokens[keep].long(), rows.abs())
    if before is not None:
        want += before.double()
        size += before.double().abs()
    m = torch.bincount(tokens[keep].long(), minlength=grad_shape[0])[:, None]
    return want, size, m


@pytest.mark.parametrize("n,vocab,dim,dtype,gdt,first", [
    (700, 70001, 801, "f32", "f32", True),      # a table above 200 MB: zeros after the sort, by marks
    (5000, 70001, 800, "bf16", "f32", True),
    (40000, 30001, 2000, "bf16", "bf16", True),  # 160 MB of rows: streamed
    (40000, 9001, 1600, "bf16", "f32", False),
    (33000, 500, 1030, "f32", "f32", False),
])
def test_backward_large(n, vocab, dim, dtype, gdt, first):
    g = gen(n + dim)
    _, dout = matrix(g, n, dim, dtype)
    tokens = make_tokens(g, n, vocab, "mixed", "i64")
    tokens[: n // 10] = 7  # a frequent one
    _, grad = matrix(g, vocab, dim, gdt, fill=float("nan") if first else None)
    before = None if first else grad.clone()
    run_backward(dout, tokens, grad, scale=0.5, first=first)
    want, size, m = reference_on_the_gpu(dout, tokens, (vocab, dim), before, 0.5)
    tol = ((m + 2) * U * size + HALF[grad.dtype] * want.abs()) * (1 + 2.0 ** -7)
    assert bool(((grad.double() - want).abs() <= tol).all())
    if first:
        assert torch.count_nonzero(bits(grad[m[:, 0] == 0])) == 0


@pytest.mark.parametrize("vocab,dim", [(1024, 768), (2048, 64)])
def test_backward_of_a_position_table(vocab, dim):
    # every position many times, in order: the wpe gradient of a batch
    g = gen(vocab)
    _, dout = matrix(g, 4 * vocab, dim, "bf16")
    positions = torch.arange(4 * vocab, device="cuda", dtype=torch.int32) % vocab
    grad = torch.empty(vocab, dim, device="cuda")
    run_backward(dout, positions, grad, first=True)
    # four rows in order, fp32: the same bits
    r = dout.float().view(4, vocab, dim)
    assert torch.equal(grad, ((r[0] + r[1]) + r[2]) + r[3])


@pytest.mark.parametrize("dtype,gdt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_backward_every_type(dtype, gdt):
    g = gen(77)
    for dim in (64, 520, 4100):
        _, dout = matrix(g, 700, dim, dtype)
        tokens = make_tokens(g, 700, 90, "mixed", "i32")
        for first in (True, False):
            _, grad = matrix(g, 90, dim, gdt)
            before = grad.clone()
            run_backward(dout, tokens, grad, scale=-0.75, first=first, padding_idx=4)
            check_backward(dout, tokens, grad, before, -0.75, 4, first)


def test_backward_without_tokens():
    grad = torch.full((70, 33), float("nan"), device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, device="cuda", dtype=torch.int64)
    ws = torch.empty(zs.zs_embed_workspace_bytes(0, 70, 33) or 16, device="cuda", dtype=torch.uint8)
    zs.zs_embed_backward(torch.empty(0, 33, device="cuda"), none, grad, workspace=ws)
    assert torch.isnan(grad).all()  # nothing to add
    zs.zs_embed_backward(torch.empty(0, 33, device="cuda"), none, grad, first=True, workspace=ws)
    assert torch.count_nonzero(bits(grad)) == 0


def test_backward_non_finite_rows_stay_where_they_belong():
    g = gen(8)
    _, dout = matrix(g, 600, 72, "bf16")
    tokens = torch.randint(1, 20, (600,), generator=g, device="cuda")
    tokens[100] = -100
    dout[100] = float("nan")  # ignored: reaches nothing
    tokens[200] = 0
    dout[200, 5] = float("inf")
    tokens[201] = 25
    dout[201, 6] = float("nan")
    grad = torch.empty(30, 72, device="cuda")
    run_backward(dout, tokens, grad, first=True)
    bad = ~torch.isfinite(grad)
    assert bad.sum() == 2 and torch.isinf(grad[0, 5]) and torch.isnan(grad[25, 6])


def test_backward_same_bits_every_time():
    g = gen(9)
    _, dout = matrix(g, 20000, 136, "bf16")
    tokens = make_tokens(g, 20000, 500, "runs", "i64")
    tokens[::3] = torch.randint(0, 500, (6667,), generator=g, device="cuda")
    a, b = torch.empty(500, 136, device="cuda"), torch.empty(500, 136, device="cuda")
    run_backward(dout, tokens, a, first=True)
    for _ in range(5):
        run_backward(dout, tokens, b, first=True)
        assert torch.equal(bits(a), bits(b))


def test_backward_offsets_beyond_32_bits():
    ld, rows, dim = 1 << 22, 600, 40
    buf = torch.empty(rows * ld, device="cuda", dtype=torch.bfloat16)
    wide = buf.view(rows, ld)[:, :dim]
    narrow = torch.randn(rows, dim, device="cuda").bfloat16()
    ids = torch.arange(rows - 1, -1, -1, device="cuda")
    run_backward(narrow, ids, wide, first=True)  # the gradient's last row past 2^32 bytes
    assert torch.equal(wide, narrow.flip(0))
    grad = torch.empty(rows, dim, device="cuda")
    run_backward(wide, ids, grad, first=True)  # dout's rows that far apart
    assert torch.equal(grad, narrow.float())


def test_extreme_sizes():
    # the largest vocabulary, widest rows and many tokens, each alone
    last = 2 ** 31 - 2
    table = torch.zeros(2 ** 31 - 1, 1, device="cuda", dtype=torch.bfloat16)
    table[last] = 3.0
    ids = torch.tensor([last, 0, last + 1, 2 ** 40, -(2 ** 40)], device="cuda")
    out = torch.empty(5, 1, device="cuda")
    zs.zs_embed_forward(table, ids, out, scale=2.0)
    assert out[:, 0].tolist() == [6.0, 0.0, 0.0, 0.0, 0.0]
    run_backward(torch.ones(5, 1, device="cuda"), ids, table, padding_idx=None)
    assert table[last].item() == 4.0 and table[0].item() == 1.0 and torch.count_nonzero(table) == 2
    del table

    dim = 2 ** 24 - 1
    table = torch.randn(2, dim, device="cuda")
    out = torch.empty(3, dim, device="cuda", dtype=torch.bfloat16)
    ids = torch.tensor([1, 0, 1], device="cuda", dtype=torch.int32)
    zs.zs_embed_forward(table, ids, out)
    assert torch.equal(out, table[ids.long()].bfloat16())
    grad = torch.empty(2, dim, device="cuda")
    run_backward(out, ids, grad, first=True)
    assert torch.equal(grad[1], out[0].float() + out[2].float()) and torch.equal(grad[0], out[1].float())

    n, vocab = 20_000_003, 128256
    g = gen(20)
    ids = torch.randint(-3, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    ids[::7] = 11
    dout = torch.randint(-3, 4, (n, 4), generator=g, device="cuda").float()  # small whole numbers: every sum is exact
    grad = torch.empty(vocab, 4, device="cuda")
    run_backward(dout, ids, grad, first=True)
    keep = ids >= 0
    order = torch.sort(ids[keep].long()).indices
    counts = torch.bincount(ids[keep].long(), minlength=vocab)
    sums = torch.cat([torch.zeros(1, 4, device="cuda", dtype=torch.float64), dout[keep][order].double().cumsum(0)])
    ends = counts.cumsum(0)
    assert torch.equal(grad.double(), sums[ends] - sums[ends - counts])


def test_two_streams_at_once_and_another_than_the_current():
    g = gen(11)
    work = []
    for k in range(2):
        _, dout = matrix(g, 9000, 200, "bf16")
        tokens = make_tokens(g, 9000, 3000, "mixed", "i64")
        work.append((dout, tokens, torch.empty(3000, 200, device="cuda"), torch.empty(3000, 200, device="cuda"),
                     torch.empty(zs.zs_embed_workspace_bytes(9000, 3000, 200), device="cuda", dtype=torch.uint8)))
    for d, t, ref, _, ws in work:
        zs.zs_embed_backward(d, t, ref, first=True, workspace=ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(3):
        for s, (d, t, _, out, ws) in zip(streams, work):
            zs.zs_embed_backward(d, t, out, first=True, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, _, ref, out, _ in work:
        assert torch.equal(bits(ref), bits(out))


def test_graph_replays():
    g = gen(12)
    _, table = matrix(g, 500, 264, "bf16")
    _, dout = matrix(g, 3000, 264, "bf16")
    tokens = make_tokens(g, 3000, 500, "mixed", "i64")
    out, eout = (torch.empty(3000, 264, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    acc, eacc = (torch.zeros(500, 264, device="cuda") for _ in range(2))
    ws, ews = (torch.empty(zs.zs_embed_workspace_bytes(3000, 500, 264), device="cuda", dtype=torch.uint8)
               for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zs.zs_embed_forward(table, tokens, out, scale=2.0)
        zs.zs_embed_backward(dout, tokens, acc, workspace=ws)
    for it in range(4):
        tokens.copy_(make_tokens(gen(100 + it), 3000, 500, ("mixed", "runs", "ignored", "equal")[it], "i64"))
        zs.zs_embed_forward(table, tokens, eout, scale=2.0)
        zs.zs_embed_backward(dout, tokens, eacc, workspace=ews)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(eout)) and torch.equal(bits(acc), bits(eacc)), it


def test_refusals_of_the_binding():
    t = torch.zeros(10, 8, device="cuda")
    ids = torch.zeros(4, device="cuda", dtype=torch.int64)
    out = torch.zeros(4, 8, device="cuda")
    ws = torch.empty(1 << 20, device="cuda", dtype=torch.uint8)
    for args, kw in [((t.half(), ids, out), {}), ((t, ids.float(), out), {}), ((t, ids[:3], out), {}),
                     ((t, ids, out[:, :7]), {}), ((t, ids.cpu(), out), {}), ((t, ids, out.t()), {}),
                     ((t, ids, out), dict(pos_table=t)), ((t, ids, out), dict(positions=ids)),
                     ((t, ids, out), dict(pos_table=t, positions=ids.int())),
                     ((t, ids, out), dict(pos_table=t.bfloat16(), positions=ids)),
                     ((t, ids, t[2:6]), {}), ((t, ids, out), dict(scale=float("nan")))]:
        with pytest.raises(ValueError):
            zs.zs_embed_forward(*args, **kw)
    for args, kw in [((out, ids, t.half()), dict(workspace=ws)), ((out, ids[:3], t), dict(workspace=ws)),
                     ((out[:, :7], ids, t), dict(workspace=ws)), ((out, ids, t), dict(workspace=None)),
                     ((out, ids, t), dict(workspace=ws[:64])), ((t[:4], ids, t), dict(workspace=ws)),
                     ((out, ids, t.expand(3, 10, 8)[0].t()), dict(workspace=ws))]:
        with pytest.raises(ValueError):
            zs.zs_embed_backward(*args, **kw)
