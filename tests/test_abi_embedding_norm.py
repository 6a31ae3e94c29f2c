"""Host-only checks of the embedding and layer norm entry points: every refusal
comes with its documented status before any device work, and the binding
refuses tensors that the library could not read. No GPU is touched.
"""
import ctypes as C
import os

import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs

L = pytest.importorskip("fsdp_sharded_optimizer_flatparameter_amd._lib")
OK, NULL, SIZE, DTYPE, HPARAM, WORKSPACE, ALIGN, OVERLAP = 0, -1, -2, -5, -6, -8, -10, -11
FAKE = 0x7F0000000000  # never dereferenced: every call below ends in its host-side checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        pytest.fail("libzs.so is not built (run the package's build step first)")
    return L.load()


def at(i, off=0):
    """Addresses 2^40 apart."""
    return FAKE + (i << 40) + off


def embed_fwd(lib, **kw):
    a = dict(table=at(0), dtype=1, vocab=100, dim=64, table_ld=64, pos_table=None, pos_rows=0, pos_ld=0, tokens=at(1),
             positions=None, itype=3, n=10, scale=1.0, out=at(2), out_dtype=1, out_ld=64)
    a.update(kw)
    return lib.zs_embed_forward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), DTYPE), (dict(out_dtype=7), DTYPE), (dict(itype=0), DTYPE), (dict(itype=4), DTYPE),
    (dict(n=-1), SIZE), (dict(vocab=-1), SIZE), (dict(dim=-1), SIZE), (dict(n=2 ** 31), SIZE),
    (dict(vocab=2 ** 31), SIZE), (dict(dim=2 ** 24, table_ld=2 ** 24, out_ld=2 ** 24), SIZE),
    (dict(table_ld=63), SIZE), (dict(out_ld=63), SIZE), (dict(out_ld=2 ** 60), SIZE), (dict(table_ld=-64), SIZE),
    (dict(pos_table=at(3), positions=at(4), pos_rows=-1, pos_ld=64), SIZE),
    (dict(pos_table=at(3), positions=at(4), pos_rows=8, pos_ld=60), SIZE),
    (dict(scale=float("nan")), HPARAM), (dict(scale=float("inf")), HPARAM),
    (dict(table=None), NULL), (dict(tokens=None), NULL), (dict(out=None), NULL),
    (dict(pos_table=at(3), pos_rows=8, pos_ld=64), NULL),
    (dict(table=at(0, 1)), ALIGN), (dict(out=at(2, 1)), ALIGN), (dict(out_dtype=0, out=at(2, 2)), ALIGN),
    (dict(tokens=at(1, 4)), ALIGN), (dict(itype=2, tokens=at(1, 2)), ALIGN),
    (dict(pos_table=at(3, 1), positions=at(4), pos_rows=8, pos_ld=64), ALIGN),
    (dict(pos_table=at(3), positions=at(4, 4), pos_rows=8, pos_ld=64), ALIGN),
    (dict(out=at(0, 100 * 64 * 2 - 2)), OVERLAP), (dict(out=at(1, 72)), OVERLAP),
    (dict(pos_table=at(3), positions=at(4), pos_rows=8, pos_ld=64, out=at(3, 512)), OVERLAP),
    (dict(pos_table=at(3), positions=at(2, 64), pos_rows=8, pos_ld=64), OVERLAP),
    (dict(n=0, table=None, tokens=None, out=None), OK), (dict(dim=0, table=None, tokens=None, out=None), OK),
])
def test_embed_forward_refusals(lib, kw, want):
    assert embed_fwd(lib, **kw) == want


def embed_bwd(lib, **kw):
    a = dict(dout=at(0), dtype=1, dout_ld=64, tokens=at(1), itype=3, n=10, vocab=100, dim=64, padding=-1, scale=1.0,
             grad=at(2), grad_dtype=0, grad_ld=64, first=0, ws=at(3),
             ws_bytes=None)
    a.update(kw)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = lib.zs_embed_workspace_bytes(a["n"], a["vocab"], a["dim"])
    return lib.zs_embed_backward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), DTYPE), (dict(grad_dtype=2), DTYPE), (dict(itype=1), DTYPE),
    (dict(n=-1, ws_bytes=0), SIZE), (dict(vocab=-1, ws_bytes=0), SIZE), (dict(dim=-1, ws_bytes=0), SIZE),
    (dict(n=2 ** 31), SIZE), (dict(vocab=2 ** 31), SIZE), (dict(dout_ld=63), SIZE), (dict(grad_ld=63), SIZE),
    (dict(scale=float("nan")), HPARAM), (dict(scale=-float("inf")), HPARAM),
    (dict(dout=None), NULL), (dict(tokens=None), NULL), (dict(grad=None), NULL),
    (dict(dout=at(0, 1)), ALIGN), (dict(tokens=at(1, 4)), ALIGN), (dict(grad=at(2, 2)), ALIGN),
    (dict(ws=at(3, 8)), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
    (dict(grad=at(0, 4)), OVERLAP), (dict(grad=at(1, 16)), OVERLAP), (dict(grad=at(3, 64)), OVERLAP),
    (dict(ws=at(0, 16)), OVERLAP), (dict(ws=at(1, 16)), OVERLAP),
    (dict(n=0, dout=None, tokens=None, grad=None, ws=None, ws_bytes=0), OK),
    (dict(n=0, first=1, grad=None), NULL), (dict(n=0, first=1, ws=None), WORKSPACE),
    (dict(vocab=0, grad=None, ws=None, ws_bytes=0), OK), (dict(dim=0, grad=None, ws=None, ws_bytes=0), OK),
])
def test_embed_backward_refusals(lib, kw, want):
    assert embed_bwd(lib, **kw) == want


def norm_fwd(lib, **kw):
    a = dict(x=at(0), dtype=1, x_ld=64, weight=at(1), bias=at(2), wdtype=1, rows=10, dim=64, eps=1e-5, y=at(3), y_ld=64,
             mean=at(4), rstd=at(5))
    a.update(kw)
    return lib.zs_layer_norm_forward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), DTYPE), (dict(wdtype=-1), DTYPE), (dict(rows=-1), SIZE), (dict(dim=0), SIZE), (dict(dim=-3), SIZE),
    (dict(rows=2 ** 31), SIZE), (dict(x_ld=63), SIZE), (dict(y_ld=1), SIZE),
    (dict(eps=-1e-9), HPARAM), (dict(eps=float("nan")), HPARAM), (dict(eps=float("inf")), HPARAM),
    (dict(eps=1e39), HPARAM), (dict(dim=2 ** 24, x_ld=2 ** 24, y_ld=2 ** 24), SIZE),
    (dict(x=None), NULL), (dict(y=None), NULL),
    (dict(x=at(0, 1)), ALIGN), (dict(y=at(3, 1)), ALIGN), (dict(weight=at(1, 1)), ALIGN), (dict(bias=at(2, 1)), ALIGN),
    (dict(wdtype=0, bias=at(2, 2)), ALIGN), (dict(mean=at(4, 2)), ALIGN), (dict(rstd=at(5, 2)), ALIGN),
    (dict(y=at(0)), OVERLAP), (dict(y=at(1, 2)), OVERLAP), (dict(y=at(2, 126)), OVERLAP), (dict(mean=at(0)), OVERLAP),
    (dict(rstd=at(3, 4)), OVERLAP), (dict(rstd=at(4, 36)), OVERLAP), (dict(mean=at(1, 4)), OVERLAP),
    (dict(rows=0, x=None, y=None, dim=0, x_ld=0, y_ld=0), OK),
])
def test_layer_norm_forward_refusals(lib, kw, want):
    assert norm_fwd(lib, **kw) == want


def norm_bwd(lib, **kw):
    a = dict(dy=at(0), dy_ld=64, x=at(1), x_ld=64, dtype=1, weight=at(2), wdtype=1, mean=at(3), rstd=at(4), rows=10,
             dim=64, dx=at(5), dx_ld=64, dw=at(6), db=at(7), gdtype=0, first=0, ws=at(8), ws_bytes=None)
    a.update(kw)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = lib.zs_layer_norm_workspace_bytes(a["rows"], a["dim"])
    return lib.zs_layer_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), DTYPE), (dict(wdtype=2), DTYPE), (dict(gdtype=2), DTYPE),
    (dict(rows=-1, ws_bytes=0), SIZE), (dict(dim=0), SIZE), (dict(dy_ld=63), SIZE), (dict(x_ld=63), SIZE),
    (dict(dx_ld=63), SIZE),
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(mean=None), NULL), (dict(rstd=None), NULL), (dict(dx=None), NULL),
    (dict(dy=at(0, 1)), ALIGN), (dict(x=at(1, 1)), ALIGN), (dict(weight=at(2, 1)), ALIGN), (dict(mean=at(3, 1)), ALIGN),
    (dict(rstd=at(4, 2)), ALIGN), (dict(dx=at(5, 1)), ALIGN), (dict(dw=at(6, 2)), ALIGN), (dict(db=at(7, 2)), ALIGN),
    (dict(ws=at(8, 4)), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(dx=at(0)), OVERLAP), (dict(dx=at(1, 2)), OVERLAP), (dict(dw=at(2, 4)), OVERLAP), (dict(db=at(6, 252)), OVERLAP),
    (dict(dw=at(5)), OVERLAP), (dict(ws=at(5, 64)), OVERLAP), (dict(ws=at(3)), OVERLAP), (dict(db=at(4, 8)), OVERLAP),
    (dict(rows=0, first=0, dy=None, x=None, mean=None, rstd=None, dx=None, ws=None, ws_bytes=0), OK),
    (dict(rows=0, first=1, dw=None, db=None, dy=None, x=None, mean=None, rstd=None, dx=None, ws=None, ws_bytes=0), OK),
])
def test_layer_norm_backward_refusals(lib, kw, want):
    assert norm_bwd(lib, **kw) == want


def test_workspace_sizes(lib):
    e, n = lib.zs_embed_workspace_bytes, lib.zs_layer_norm_workspace_bytes
    for bad in ((-1, 10, 8), (10, -1, 8), (10, 10, -1), (2 ** 31, 10, 8), (10, 2 ** 31, 8), (10, 10, 2 ** 24)):
        assert e(*bad) == 0
    assert n(-1, 8) == 0 and n(8, -1) == 0 and n(2 ** 31, 8) == 0 and n(8, 2 ** 24) == 0
    # room for the two sorted arrays of keys and positions at the least, and it never shrinks with n
    sizes = [e(k, 50257, 768) for k in (0, 1, 100, 8192, 16384, 16385, 100000, 1 << 20)]
    assert all(s >= 8 * k for s, k in zip(sizes, (0, 1, 100, 8192, 16384, 16385, 100000, 1 << 20)))
    assert n(0, 8) == 0 and n(1, 8) >= 2 * 8 * 4
    assert n(1 << 30, 8192) == n(1 << 20, 8192) < 1 << 28  # the partials do not grow with the rows


def test_binding_refuses_host_tensors():
    x, w, ids = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        zs.zs_embed_forward(x, ids, x)
    with pytest.raises(ValueError):
        zs.zs_embed_backward(x, ids, x, workspace=None)
    with pytest.raises(ValueError):
        zs.zs_layer_norm_forward(x, w, w, x)
    with pytest.raises(ValueError):
        zs.zs_layer_norm_backward(x, x, w, w, w, x)
    with pytest.raises(ValueError):
        zs.zs_embed_forward(None, ids, x)


def test_int_types_match_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "zs.h")).read()
    assert f"#define ZS_I32 {L.ZS_I32}\n" in text and f"#define ZS_I64 {L.ZS_I64}\n" in text


def test_ctypes_arguments_match_the_calls():
    # every argument of the fixtures above went through the declared argument types
    assert len(L.SIGNATURES["zs_embed_forward"][1]) == 17
    assert len(L.SIGNATURES["zs_embed_backward"][1]) == 17
    assert len(L.SIGNATURES["zs_layer_norm_forward"][1]) == 14
    assert len(L.SIGNATURES["zs_layer_norm_backward"][1]) == 20
    assert L.SIGNATURES["zs_layer_norm_forward"][1][8] is C.c_double
