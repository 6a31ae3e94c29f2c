"""Python binding of libzs: the C-ABI calls under the same names, taking torch tensors.

Argument marshalling only -- every step of the update runs in the HIP kernels
of libzs. PyTorch supplies device memory and the stream (by default the
current stream of the tensors' device); every call is asynchronous on it.

Errors from the library raise ZsArgumentError (a ValueError) for bad
arguments and ZsError (a RuntimeError) for HIP failures; tensors that are not
contiguous device tensors of the expected dtype raise ValueError before the
library is called.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib as L
from ._lib import ZS_BF16, ZS_F32, ZsArgumentError, ZsError  # noqa: F401

_DTYPES = {torch.float32: ZS_F32, torch.bfloat16: ZS_BF16}


def _lib():
    return L.load()


def _dev(t: torch.Tensor, name: str, dtype=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def _hparams(lr, beta1, beta2, eps, weight_decay, step) -> L.AdamWHParams:
    return L.AdamWHParams(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                          int(step))


# ---------------------------------------------------------------- layout

def zs_flat_layout(numels, world: int, align: int = 1):
    """(offsets, total T, padded P, shard S) of a FlatParameter over `world`
    ranks, S rounded up to a multiple of `align` elements (1: no rounding)."""
    n = len(numels)
    arr = (C.c_int64 * max(n, 1))(*[int(x) for x in numels])
    offs = (C.c_int64 * max(n, 1))()
    total, padded, shard = C.c_int64(), C.c_int64(), C.c_int64()
    L.check("zs_flat_layout", _lib().zs_flat_layout(
        arr, n, int(world), int(align), offs, C.byref(total), C.byref(padded), C.byref(shard)))
    return list(offs[:n]), total.value, padded.value, shard.value


class ParamTable:
    """Descriptor table of one unit's parameters, in flat order.

    The host copy is checked by zs_check_layout; the device copy (24 bytes per
    parameter) is what the pack and copy-out kernels read. The tensors are
    kept referenced for the table's lifetime.
    """

    def __init__(self, tensors, device=None):
        if len(tensors) == 0:
            raise ValueError("a unit needs at least one parameter")
        dtype = tensors[0].dtype
        if dtype not in _DTYPES:
            raise ValueError(f"unsupported parameter dtype {dtype}")
        for i, t in enumerate(tensors):
            _dev(t, f"param[{i}]", dtype)
        self.tensors = list(tensors)
        self.dtype = dtype
        self.nparams = len(tensors)
        self.offsets, self.total, _, _ = zs_flat_layout([t.numel() for t in tensors], 1)
        host = (L.ParamDesc * self.nparams)()
        for i, (t, off) in enumerate(zip(self.tensors, self.offsets)):
            host[i].ptr = t.data_ptr()
            host[i].flat_offset = off
            host[i].numel = t.numel()
        L.check("zs_check_layout", _lib().zs_check_layout(host, self.nparams, self.total, _DTYPES[dtype]))
        device = device if device is not None else tensors[0].device
        raw = torch.frombuffer(bytearray(bytes(host)), dtype=torch.uint8)
        self.device_table = raw.to(device)
        torch.cuda.current_stream(device).synchronize()  # the host staging copy is released

    @property
    def ptr(self):
        return C.c_void_p(self.device_table.data_ptr())


# ---------------------------------------------------------------- pack / copy-out

def zs_pack_shard(table: ParamTable, world: int, rank: int, master, exp_avg=None, exp_avg_sq=None,
                  stream=None, align: int = 1):
    _dev(master, "master", torch.float32)
    for name, t in (("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        if t is not None:
            _dev(t, name, torch.float32)
            if t.numel() != master.numel():
                raise ValueError(f"{name} must have the master's size")
    L.check("zs_pack_shard", _lib().zs_pack_shard(
        table.ptr, table.nparams, table.total, _DTYPES[table.dtype], int(world), int(rank),
        int(align), master.numel(), _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq),
        _stream(stream, master.device)))


def zs_copy_out(gathered, table: ParamTable, stream=None):
    _dev(gathered, "gathered", torch.bfloat16)
    if table.dtype != torch.bfloat16:
        raise ValueError("copy-out destinations must be bf16")
    L.check("zs_copy_out", _lib().zs_copy_out(
        _ptr(gathered), gathered.numel(), table.ptr, table.nparams, table.total,
        _stream(stream, gathered.device)))


# ---------------------------------------------------------------- per-parameter dim-0 sharding

def zs_dim0_layout(shapes, world: int):
    """(chunks, local offsets, local total L) of per-parameter dim-0 sharding over `world` ranks.

    A 0-d parameter is one row of one element.
    """
    n = len(shapes)
    d0 = [int(s[0]) if len(s) else 1 for s in shapes]
    rs = []
    for s in shapes:
        r = 1
        for x in s[1:]:
            r *= int(x)
        rs.append(r)
    a = (C.c_int64 * max(n, 1))(*d0)
    b = (C.c_int64 * max(n, 1))(*rs)
    chunk = (C.c_int64 * max(n, 1))()
    loff = (C.c_int64 * max(n, 1))()
    lt = C.c_int64()
    L.check("zs_dim0_layout", _lib().zs_dim0_layout(a, b, n, int(world), chunk, loff, C.byref(lt)))
    return list(chunk[:n]), list(loff[:n]), lt.value


class Dim0Table:
    """Descriptor table of one unit's parameters under dim-0 sharding over `world` ranks.

    The host copy is checked by zs_check_dim0_layout; the device copy (40 bytes
    per parameter) is what the pack and copy-out kernels read. The tensors are
    kept referenced for the table's lifetime.
    """

    def __init__(self, tensors, world: int, device=None):
        if len(tensors) == 0:
            raise ValueError("a unit needs at least one parameter")
        dtype = tensors[0].dtype
        if dtype not in _DTYPES:
            raise ValueError(f"unsupported parameter dtype {dtype}")
        for i, t in enumerate(tensors):
            _dev(t, f"param[{i}]", dtype)
        self.tensors = list(tensors)
        self.dtype = dtype
        self.world = int(world)
        self.nparams = len(tensors)
        self.chunks, self.local_offsets, self.local_total = zs_dim0_layout(
            [tuple(t.shape) for t in tensors], self.world)
        self.offsets, self.total, _, _ = zs_flat_layout([t.numel() for t in tensors], 1)
        host = (L.Dim0Desc * self.nparams)()
        for i, t in enumerate(self.tensors):
            host[i].ptr = t.data_ptr()
            host[i].flat_offset = self.offsets[i]
            host[i].numel = t.numel()
            host[i].chunk = self.chunks[i]
            host[i].local_offset = self.local_offsets[i]
        L.check("zs_check_dim0_layout", _lib().zs_check_dim0_layout(
            host, self.nparams, self.world, self.total, self.local_total, _DTYPES[dtype]))
        device = device if device is not None else tensors[0].device
        raw = torch.frombuffer(bytearray(bytes(host)), dtype=torch.uint8)
        self.device_table = raw.to(device)
        torch.cuda.current_stream(device).synchronize()  # the host staging copy is released

    @property
    def ptr(self):
        return C.c_void_p(self.device_table.data_ptr())


def zs_pack_shard_dim0(table: Dim0Table, rank: int, master, exp_avg=None, exp_avg_sq=None,
                       stream=None):
    _dev(master, "master", torch.float32)
    if master.numel() != table.local_total:
        raise ValueError(f"master must hold the rank's {table.local_total} elements")
    for name, t in (("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        if t is not None:
            _dev(t, name, torch.float32)
            if t.numel() != master.numel():
                raise ValueError(f"{name} must have the master's size")
    L.check("zs_pack_shard_dim0", _lib().zs_pack_shard_dim0(
        table.ptr, table.nparams, _DTYPES[table.dtype], table.world, int(rank), table.local_total,
        _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), _stream(stream, master.device)))


def zs_copy_out_dim0(gathered, table: Dim0Table, stream=None):
    _dev(gathered, "gathered", torch.bfloat16)
    if table.dtype != torch.bfloat16:
        raise ValueError("copy-out destinations must be bf16")
    L.check("zs_copy_out_dim0", _lib().zs_copy_out_dim0(
        _ptr(gathered), gathered.numel(), table.ptr, table.nparams, table.world, table.total,
        table.local_total, _stream(stream, gathered.device)))


# ---------------------------------------------------------------- reduce / AdamW / cast

def _rows(rows, n):
    if len(rows) == 0:
        raise ValueError("need at least one gradient contribution")
    dtype = rows[0].dtype
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported contribution dtype {dtype}")
    for i, r in enumerate(rows):
        _dev(r, f"rows[{i}]", dtype)
        if r.numel() != n:
            raise ValueError(f"rows[{i}] has {r.numel()} elements, expected {n}")
    arr = (C.c_void_p * len(rows))(*[r.data_ptr() for r in rows])
    return arr, len(rows), _DTYPES[dtype]


def zs_workspace_bytes(n: int) -> int:
    return int(_lib().zs_workspace_bytes(int(n)))


def zs_reduce_grads(rows, grad_out, sumsq_out=None, workspace=None, stream=None):
    _dev(grad_out, "grad_out", torch.float32)
    arr, world, dt = _rows(rows, grad_out.numel())
    ws_bytes = 0
    if sumsq_out is not None:
        _dev(sumsq_out, "sumsq_out", torch.float64)
    if workspace is not None:
        _dev(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    L.check("zs_reduce_grads", _lib().zs_reduce_grads(
        arr, world, dt, grad_out.numel(), _ptr(grad_out), _ptr(sumsq_out), _ptr(workspace),
        ws_bytes, _stream(stream, grad_out.device)))


def zs_reduce_grads_noalloc(rows, grad_out, sumsq_out=None, stream=None):
    """zs_reduce_grads without a workspace: the sum of squares uses the
    library's static scratch (no device allocation by the library)."""
    _dev(grad_out, "grad_out", torch.float32)
    arr, world, dt = _rows(rows, grad_out.numel())
    if sumsq_out is not None:
        _dev(sumsq_out, "sumsq_out", torch.float64)
    L.check("zs_reduce_grads_noalloc", _lib().zs_reduce_grads_noalloc(
        arr, world, dt, grad_out.numel(), _ptr(grad_out), _ptr(sumsq_out), _stream(stream, grad_out.device)))


def _state(master, exp_avg, exp_avg_sq):
    _dev(master, "master", torch.float32)
    _dev(exp_avg, "exp_avg", torch.float32)
    _dev(exp_avg_sq, "exp_avg_sq", torch.float32)
    n = master.numel()
    if exp_avg.numel() != n or exp_avg_sq.numel() != n:
        raise ValueError("master, exp_avg and exp_avg_sq must have the same size")
    return n


def _opt_out(bf16_out, grad_scale, n):
    if bf16_out is not None:
        _dev(bf16_out, "bf16_out", torch.bfloat16)
        if bf16_out.numel() != n:
            raise ValueError("bf16_out must have the master's size")
    if grad_scale is not None:
        _dev(grad_scale, "grad_scale", torch.float32)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale is a single fp32 value")


def zs_adamw_step(master, exp_avg, exp_avg_sq, grad, *, lr, beta1, beta2, eps, weight_decay, step,
                  grad_scale=None, bf16_out=None, stream=None):
    n = _state(master, exp_avg, exp_avg_sq)
    _dev(grad, "grad", torch.float32)
    if grad.numel() != n:
        raise ValueError("grad must have the master's size")
    _opt_out(bf16_out, grad_scale, n)
    hp = _hparams(lr, beta1, beta2, eps, weight_decay, step)
    L.check("zs_adamw_step", _lib().zs_adamw_step(
        _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(grad), n, C.byref(hp),
        _ptr(grad_scale), _ptr(bf16_out), _stream(stream, master.device)))


def zs_cast_for_gather(master, gather_slot, stream=None):
    _dev(master, "master", torch.float32)
    _dev(gather_slot, "gather_slot", torch.bfloat16)
    if gather_slot.numel() != master.numel():
        raise ValueError("gather_slot must have the master's size")
    L.check("zs_cast_for_gather", _lib().zs_cast_for_gather(
        _ptr(master), master.numel(), _ptr(gather_slot), _stream(stream, master.device)))


def zs_sharded_step(rows, master, exp_avg, exp_avg_sq, *, lr, beta1, beta2, eps, weight_decay,
                    step, grad_scale=None, bf16_out=None, stream=None):
    n = _state(master, exp_avg, exp_avg_sq)
    arr, world, dt = _rows(rows, n)
    _opt_out(bf16_out, grad_scale, n)
    hp = _hparams(lr, beta1, beta2, eps, weight_decay, step)
    L.check("zs_sharded_step", _lib().zs_sharded_step(
        arr, world, dt, n, _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), C.byref(hp),
        _ptr(grad_scale), _ptr(bf16_out), _stream(stream, master.device)))


class ShardedStep:
    """zs_sharded_step with its arguments checked and marshalled once.

    Calling the object with a step number issues one C call with the prepared
    arguments: the per-step host cost is a single ctypes call, which is what a
    small (launch-bound) shard needs. The tensors are kept referenced. The
    stream is fixed when the object is made (default: the current stream of
    the master's device at that moment), so an object used under HIP graph
    capture must be made inside the capture. The library still validates
    every call.
    """

    def __init__(self, rows, master, exp_avg, exp_avg_sq, *, lr, beta1, beta2, eps, weight_decay,
                 grad_scale=None, bf16_out=None, stream=None):
        n = _state(master, exp_avg, exp_avg_sq)
        self._rows, self._world, self._dtype = _rows(rows, n)
        _opt_out(bf16_out, grad_scale, n)
        self._keep = (list(rows), master, exp_avg, exp_avg_sq, grad_scale, bf16_out)
        self._hp = _hparams(lr, beta1, beta2, eps, weight_decay, 1)
        self._fn = _lib().zs_sharded_step
        self._args = (self._rows, self._world, self._dtype, n, _ptr(master), _ptr(exp_avg),
                      _ptr(exp_avg_sq), C.byref(self._hp), _ptr(grad_scale), _ptr(bf16_out),
                      _stream(stream, master.device))

    def __call__(self, step: int) -> None:
        self._hp.step = int(step)
        st = self._fn(*self._args)
        if st != 0:
            L.check("zs_sharded_step", st)


def zs_accumulate_grads(rows, acc, *, scale=1.0, first=False, sumsq_out=None, workspace=None,
                        stream=None):
    _dev(acc, "acc", torch.float32)
    arr, world, dt = _rows(rows, acc.numel())
    ws_bytes = 0
    if sumsq_out is not None:
        _dev(sumsq_out, "sumsq_out", torch.float64)
    if workspace is not None:
        _dev(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    L.check("zs_accumulate_grads", _lib().zs_accumulate_grads(
        arr, world, dt, acc.numel(), _ptr(acc), float(scale), int(bool(first)), _ptr(sumsq_out),
        _ptr(workspace), ws_bytes, _stream(stream, acc.device)))


def zs_accumulate_local(grad, acc, *, first=False, stream=None):
    _dev(acc, "acc", torch.float32)
    _dev(grad, "grad")
    if grad.dtype not in _DTYPES:
        raise ValueError(f"unsupported gradient dtype {grad.dtype}")
    if grad.numel() != acc.numel():
        raise ValueError("grad and acc must have the same size")
    L.check("zs_accumulate_local", _lib().zs_accumulate_local(
        _ptr(grad), _DTYPES[grad.dtype], acc.numel(), _ptr(acc), int(bool(first)),
        _stream(stream, acc.device)))


def zs_clip_coefficient(partials, max_norm, coef_out, norm_out=None, stream=None):
    _dev(partials, "partials", torch.float64)
    _dev(coef_out, "coef_out", torch.float32)
    if coef_out.numel() != 1:
        raise ValueError("coef_out is a single fp32 value")
    if norm_out is not None:
        _dev(norm_out, "norm_out", torch.float64)
    L.check("zs_clip_coefficient", _lib().zs_clip_coefficient(
        _ptr(partials), partials.numel(), float(max_norm), _ptr(coef_out), _ptr(norm_out),
        _stream(stream, partials.device)))


# ---------------------------------------------------------------- embedding, layer norm

_Tensor = torch.Tensor
_INDEX_TYPES = {torch.int32: L.ZS_I32, torch.int64: L.ZS_I64}


def _rows2d(t, name, dev):
    """(rows, dim, row stride) of a tensor whose last dimension is a row: two
    dimensions with any stride between rows, or contiguous with any number."""
    if isinstance(t, _Tensor) and t.get_device() == dev and t.dtype in _DTYPES:
        shape = t.shape
        if len(shape) == 2:
            rows, dim = shape
            ld, unit = t.stride()
            if unit == 1 and ld >= dim:
                return rows, dim, ld
            if (unit == 1 or dim <= 1) and (ld >= dim or rows <= 1):
                return rows, dim, max(ld, dim)
            raise ValueError(f"{name}: the elements of a row must be contiguous and rows must not overlap")
        if not shape or not t.is_contiguous():
            raise ValueError(f"{name} must have two dimensions or be contiguous")
        dim = shape[-1]
        return (t.numel() // dim if dim else 0), dim, dim
    _on_device(t, name, dev)
    raise ValueError(f"unsupported dtype {t.dtype} of {name}")


def _shape2d(t, name):
    """_rows2d's sizes for a tensor of another type."""
    if t.dim() == 2:
        rows, dim = t.shape
        ld, unit = t.stride()
        if (unit == 1 or dim <= 1) and (ld >= dim or rows <= 1):
            return rows, dim, max(ld, dim)
        raise ValueError(f"{name}: the elements of a row must be contiguous and rows must not overlap")
    if not t.dim() or not t.is_contiguous():
        raise ValueError(f"{name} must have two dimensions or be contiguous")
    dim = t.shape[-1]
    return (t.numel() // dim if dim else 0), dim, dim


def _on_device(t, name, dev):
    if not isinstance(t, _Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")


def _ids(t, name, n, dev):
    if not (isinstance(t, _Tensor) and t.get_device() == dev and t.is_contiguous()):
        _on_device(t, name, dev)
        raise ValueError(f"{name} must be contiguous")
    itype = _INDEX_TYPES.get(t.dtype)
    if itype is None:
        raise ValueError(f"{name} must be int32 or int64, got {t.dtype}")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    return itype


def _vector(t, name, n, dev, dtype=None):
    """Pointer of an optional contiguous vector of n elements on device `dev`."""
    if t is None:
        return None
    if not (isinstance(t, _Tensor) and t.get_device() == dev and t.is_contiguous()):
        _on_device(t, name, dev)
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    return t.data_ptr()


def _int64(v):
    """An integer as the library's 64-bit type, the nearest one where it does not fit: ctypes would
    drop its upper bits, which makes an id of a table or a size that is accepted out of it."""
    return max(-2 ** 63, min(2 ** 63 - 1, int(v)))


def _device_index(t, name):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    if not (isinstance(ws, _Tensor) and ws.get_device() == dev and ws.is_contiguous()):
        _on_device(ws, "workspace", dev)
        raise ValueError("workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# The current stream's handle without a Stream object around it (1.1 us of a
# call of 6), and the current device, straight from torch's bindings where this
# torch has them there.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, dev, stream, *args):
    """One library call with device `dev` current: the null stream is the current device's."""
    if stream is None:
        stream = _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device_index != dev:
            raise ValueError("the stream is another device's")
        stream = stream.cuda_stream
    else:
        stream = int(stream)
    fn = getattr(_lib(), name)
    if _current_device() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != 0:
        L.check(name, st)


def zs_embed_forward(table, tokens, out, *, scale=1.0, pos_table=None, positions=None, stream=None):
    """out[i] = scale * table[tokens[i]] (+ pos_table[positions[i]]); ids outside of a table
    select zeros. `out` has a row per token."""
    dev = _device_index(table, "table")
    vocab, dim, table_ld = _rows2d(table, "table", dev)
    n, out_dim, out_ld = _rows2d(out, "out", dev)
    itype = _ids(tokens, "tokens", n if out_dim else None, dev)
    if out_dim != dim:
        raise ValueError(f"out has rows of {out_dim} elements, the table's have {dim}")
    pos_ptr = positions_ptr = None
    pos_rows = pos_ld = 0
    if (pos_table is None) != (positions is None):
        raise ValueError("pos_table and positions come together")
    if pos_table is not None:
        pos_rows, pos_dim, pos_ld = _rows2d(pos_table, "pos_table", dev)
        if pos_dim != dim or pos_table.dtype != table.dtype:
            raise ValueError("pos_table must have the table's width and dtype")
        if _ids(positions, "positions", n, dev) != itype:
            raise ValueError("positions must have the tokens' dtype")
        pos_ptr, positions_ptr = pos_table.data_ptr(), positions.data_ptr()
    _call("zs_embed_forward", dev, stream, table.data_ptr(), _DTYPES[table.dtype], vocab, dim, table_ld,
          pos_ptr, pos_rows, pos_ld, tokens.data_ptr(), positions_ptr, itype, n, float(scale), out.data_ptr(),
          _DTYPES[out.dtype], out_ld)


def zs_embed_workspace_bytes(n: int, vocab: int, dim: int) -> int:
    return int(_lib().zs_embed_workspace_bytes(_int64(n), _int64(vocab), _int64(dim)))


def zs_embed_backward(dout, tokens, grad, *, scale=1.0, padding_idx=-1, first=False, workspace, stream=None):
    """grad[v] = (0 if first else grad[v]) + scale * sum of dout[i] over tokens[i] == v; ids outside of
    the table and padding_idx (None or an id outside: none) contribute nothing."""
    dev = _device_index(grad, "grad")
    vocab, dim, grad_ld = _rows2d(grad, "grad", dev)
    n, dout_dim, dout_ld = _rows2d(dout, "dout", dev)
    itype = _ids(tokens, "tokens", n if dout_dim else None, dev)
    if dout_dim != dim:
        raise ValueError(f"dout has rows of {dout_dim} elements, grad's have {dim}")
    ws, ws_bytes = _workspace(workspace, dev)
    _call("zs_embed_backward", dev, stream, dout.data_ptr(), _DTYPES[dout.dtype], dout_ld, tokens.data_ptr(),
          itype, n, vocab, dim, -1 if padding_idx is None else _int64(padding_idx), float(scale), grad.data_ptr(),
          _DTYPES[grad.dtype], grad_ld, 1 if first else 0, ws, ws_bytes)


def zs_layer_norm_forward(x, weight, bias, y, *, eps=1e-5, mean=None, rstd=None, stream=None):
    """y = (x - mean) * rstd * weight + bias over the last dimension; weight and bias may be
    None; mean and rstd (fp32, one per row) are written where given."""
    dev = _device_index(x, "x")
    rows, dim, x_ld = _rows2d(x, "x", dev)
    y_rows, y_dim, y_ld = _rows2d(y, "y", dev)
    if y_rows != rows or y_dim != dim or y.dtype != x.dtype:
        raise ValueError("y must have x's rows, width and dtype")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    w = _vector(weight, "weight", dim, dev)
    b = _vector(bias, "bias", dim, dev)
    wdtype = (weight if weight is not None else bias if bias is not None else x).dtype
    if wdtype not in _DTYPES:
        raise ValueError(f"unsupported weight dtype {wdtype}")
    _call("zs_layer_norm_forward", dev, stream, x.data_ptr(), _DTYPES[x.dtype], x_ld, w, b, _DTYPES[wdtype],
          rows, dim, float(eps), y.data_ptr(), y_ld, _vector(mean, "mean", rows, dev, torch.float32),
          _vector(rstd, "rstd", rows, dev, torch.float32))


def zs_layer_norm_workspace_bytes(rows: int, dim: int) -> int:
    return int(_lib().zs_layer_norm_workspace_bytes(_int64(rows), _int64(dim)))


def zs_layer_norm_backward(dy, x, weight, mean, rstd, dx, *, dweight=None, dbias=None, first=False,
                           workspace=None, stream=None):
    """dx, and (0 if first else the old value) + the sums over rows in dweight and dbias
    where given, which then need a workspace."""
    dev = _device_index(x, "x")
    rows, dim, x_ld = _rows2d(x, "x", dev)
    dy_rows, dy_dim, dy_ld = _rows2d(dy, "dy", dev)
    dx_rows, dx_dim, dx_ld = _rows2d(dx, "dx", dev)
    if dy_rows != rows or dy_dim != dim or dx_rows != rows or dx_dim != dim:
        raise ValueError("dy and dx must have x's rows and width")
    if dy.dtype != x.dtype or dx.dtype != x.dtype:
        raise ValueError("dy and dx must have x's dtype")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are those of the forward pass")
    w = _vector(weight, "weight", dim, dev)
    wdtype = x.dtype if weight is None else weight.dtype
    if wdtype not in _DTYPES:
        raise ValueError(f"unsupported weight dtype {wdtype}")
    if dweight is not None and dbias is not None and dweight.dtype != dbias.dtype:
        raise ValueError("dweight and dbias must have one dtype")
    dw = _vector(dweight, "dweight", dim, dev)
    db = _vector(dbias, "dbias", dim, dev)
    gdtype = (dweight if dweight is not None else dbias if dbias is not None else x).dtype
    if gdtype not in _DTYPES:
        raise ValueError(f"unsupported gradient dtype {gdtype}")
    ws, ws_bytes = _workspace(workspace, dev)
    _call("zs_layer_norm_backward", dev, stream, dy.data_ptr(), dy_ld, x.data_ptr(), x_ld, _DTYPES[x.dtype], w,
          _DTYPES[wdtype], _vector(mean, "mean", rows, dev, torch.float32),
          _vector(rstd, "rstd", rows, dev, torch.float32), rows, dim, dx.data_ptr(), dx_ld, dw, db,
          _DTYPES[gdtype], 1 if first else 0, ws, ws_bytes)


# ---------------------------------------------------------------- RMS norm, activations in 8 bits

_CODE_TYPES = (torch.uint8, torch.float8_e4m3fn)
SCALE_BLOCK = 128


def _codes(codes, scales, rows, dim, dev):
    """(pointer, row stride) of codes and of their scales."""
    if codes is None or scales is None:
        raise ValueError("codes and scales come together")
    if not (isinstance(codes, _Tensor) and codes.get_device() == dev):
        _on_device(codes, "codes", dev)
    if codes.dtype not in _CODE_TYPES:
        raise ValueError(f"codes must be uint8 or float8_e4m3fn, got {codes.dtype}")
    c_rows, c_dim, c_ld = _shape2d(codes, "codes")
    if not (isinstance(scales, _Tensor) and scales.get_device() == dev):
        _on_device(scales, "scales", dev)
    if scales.dtype is not torch.float32:
        raise ValueError(f"scales must be torch.float32, got {scales.dtype}")
    s_rows, s_dim, s_ld = _shape2d(scales, "scales")
    if (c_rows, c_dim) != (rows, dim):
        raise ValueError(f"codes are {c_rows} x {c_dim}, the rows {rows} x {dim}")
    if dim and (s_rows, s_dim) != (rows, -(-dim // SCALE_BLOCK)):
        raise ValueError(f"scales are {s_rows} x {s_dim}, expected {rows} x {-(-dim // SCALE_BLOCK)}")
    return codes.data_ptr(), c_ld, scales.data_ptr(), s_ld


def zs_activation_pack(x, codes, scales, *, stream=None):
    """x's rows as e4m3 codes (uint8 or float8_e4m3fn) and an fp32 scale, a power of two, for each
    block of 128 elements of a row: scales is [rows, ceil(dim / 128)]."""
    dev = _device_index(x, "x")
    rows, dim, x_ld = _rows2d(x, "x", dev)
    c, c_ld, sc, sc_ld = _codes(codes, scales, rows, dim, dev)
    _call("zs_activation_pack", dev, stream, x.data_ptr(), _DTYPES[x.dtype], x_ld, rows, dim, c, c_ld, sc, sc_ld)


def zs_activation_unpack(codes, scales, out, *, stream=None):
    """out = code * scale."""
    dev = _device_index(out, "out")
    rows, dim, out_ld = _rows2d(out, "out", dev)
    c, c_ld, sc, sc_ld = _codes(codes, scales, rows, dim, dev)
    _call("zs_activation_unpack", dev, stream, c, c_ld, sc, sc_ld, rows, dim, out.data_ptr(), _DTYPES[out.dtype], out_ld)


def zs_rms_norm_forward(x, weight, y=None, *, eps=1e-5, residual=None, residual_out=None, codes=None, scales=None,
                        rstd=None, stream=None):
    """y = h * rstd * weight for h = x + residual (residual None: x) and rstd = 1 / sqrt(mean(h^2) + eps).
    residual_out takes h (it may be residual, or x where the types are the same), codes and scales take
    y in 8 bits, rstd (fp32, one per row) the statistics, each where given; y may be None with codes.
    residual and residual_out have x's dtype or fp32."""
    dev = _device_index(x, "x")
    rows, dim, x_ld = _rows2d(x, "x", dev)
    xcode = sum_code = _DTYPES[x.dtype]
    y_ptr = r_ptr = s_ptr = c_ptr = sc_ptr = None
    y_ld = r_ld = s_ld = c_ld = sc_ld = 0
    if y is not None:
        y_rows, y_dim, y_ld = _rows2d(y, "y", dev)
        if y_rows != rows or y_dim != dim or y.dtype != x.dtype:
            raise ValueError("y must have x's rows, width and dtype")
        y_ptr = y.data_ptr()
    elif codes is None:
        raise ValueError("y may be None only with codes")
    if residual is not None:
        r_rows, r_dim, r_ld = _rows2d(residual, "residual", dev)
        if r_rows != rows or r_dim != dim:
            raise ValueError("residual must have x's rows and width")
        r_ptr, sum_code = residual.data_ptr(), _DTYPES[residual.dtype]
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out comes with a residual")
        s_rows, s_dim, s_ld = _rows2d(residual_out, "residual_out", dev)
        if s_rows != rows or s_dim != dim or residual_out.dtype != residual.dtype:
            raise ValueError("residual_out must have residual's rows, width and dtype")
        s_ptr = residual_out.data_ptr()
    if codes is not None or scales is not None:
        c_ptr, c_ld, sc_ptr, sc_ld = _codes(codes, scales, rows, dim, dev)
    w = _vector(weight, "weight", dim, dev)
    wdtype = x.dtype if weight is None else weight.dtype
    if wdtype not in _DTYPES:
        raise ValueError(f"unsupported weight dtype {wdtype}")
    _call("zs_rms_norm_forward", dev, stream, x.data_ptr(), xcode, x_ld, r_ptr, r_ld, s_ptr, s_ld, sum_code, w,
          _DTYPES[wdtype], rows, dim, float(eps), y_ptr, y_ld, c_ptr, c_ld, sc_ptr, sc_ld,
          _vector(rstd, "rstd", rows, dev, torch.float32))


def zs_rms_norm_workspace_bytes(rows: int, dim: int) -> int:
    return int(_lib().zs_rms_norm_workspace_bytes(_int64(rows), _int64(dim)))


def zs_rms_norm_backward(dy, h, weight, rstd, dh, *, scales=None, dresidual=None, dweight=None, first=False,
                         workspace=None, stream=None):
    """dh = rstd * (dy * weight - xh * mean(dy * weight * xh)) (+ dresidual) for xh = h * rstd, and (0 if
    first else the old value) + the sum of dy * xh over rows in dweight where given, which then needs a
    workspace. h is what was normed, in dh's dtype, or its codes with their scales; dh has dy's
    dtype or fp32 and may be dresidual."""
    dev = _device_index(dy, "dy")
    rows, dim, dy_ld = _rows2d(dy, "dy", dev)
    dh_rows, dh_dim, dh_ld = _rows2d(dh, "dh", dev)
    if dh_rows != rows or dh_dim != dim:
        raise ValueError("dh must have dy's rows and width")
    sc_ptr, sc_ld = None, 0
    if scales is not None or (isinstance(h, _Tensor) and h.dtype in _CODE_TYPES):
        h_ptr, h_ld, sc_ptr, sc_ld = _codes(h, scales, rows, dim, dev)
        h_code = L.ZS_E4M3
    else:
        h_rows, h_dim, h_ld = _rows2d(h, "h", dev)
        if h_rows != rows or h_dim != dim or h.dtype != dh.dtype:
            raise ValueError("h must have dy's rows and width and dh's dtype, or be codes")
        h_ptr, h_code = h.data_ptr(), _DTYPES[h.dtype]
    r_ptr, r_ld = None, 0
    if dresidual is not None:
        r_rows, r_dim, r_ld = _rows2d(dresidual, "dresidual", dev)
        if r_rows != rows or r_dim != dim or dresidual.dtype != dh.dtype:
            raise ValueError("dresidual must have dy's rows and width and dh's dtype")
        r_ptr = dresidual.data_ptr()
    if rstd is None:
        raise ValueError("rstd is that of the forward pass")
    w = _vector(weight, "weight", dim, dev)
    wdtype = dy.dtype if weight is None else weight.dtype
    if wdtype not in _DTYPES:
        raise ValueError(f"unsupported weight dtype {wdtype}")
    gdtype = dy.dtype if dweight is None else dweight.dtype
    dw = _vector(dweight, "dweight", dim, dev)
    if gdtype not in _DTYPES:
        raise ValueError(f"unsupported gradient dtype {gdtype}")
    ws, ws_bytes = _workspace(workspace, dev)
    _call("zs_rms_norm_backward", dev, stream, dy.data_ptr(), _DTYPES[dy.dtype], dy_ld, h_ptr, h_code, h_ld, sc_ptr,
          sc_ld, w, _DTYPES[wdtype], _vector(rstd, "rstd", rows, dev, torch.float32), r_ptr, r_ld, rows, dim,
          dh.data_ptr(), dh_ld, _DTYPES[dh.dtype], dw, _DTYPES[gdtype], 1 if first else 0, ws, ws_bytes)


# ---------------------------------------------------------------- loss over a vocabulary

def _float_code(dtype, name):
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported {name} {dtype}")
    return _DTYPES[dtype]


def zs_linear_cross_entropy_workspace_bytes(n: int, vocab: int, dim: int, dtype, grad_dtype=None) -> int:
    """Workspace of the backward pass with a dweight of `grad_dtype`, or (None) of the forward pass,
    for hidden states and weight of `dtype` (torch dtypes)."""
    return int(_lib().zs_linear_cross_entropy_workspace_bytes(
        _int64(n), _int64(vocab), _int64(dim), _float_code(dtype, "dtype"),
        -1 if grad_dtype is None else _float_code(grad_dtype, "grad_dtype")))


def _head(hidden, weight, labels):
    """What both passes read: device, sizes, strides and the labels' type."""
    dev = _device_index(weight, "weight")
    vocab, dim, weight_ld = _rows2d(weight, "weight", dev)
    n, hidden_dim, hidden_ld = _rows2d(hidden, "hidden", dev)
    itype = _ids(labels, "labels", n if hidden_dim else None, dev)
    if hidden_dim != dim:
        raise ValueError(f"hidden has rows of {hidden_dim} elements, weight's have {dim}")
    if hidden.dtype != weight.dtype:
        raise ValueError("hidden and weight must have one dtype")
    return dev, n, vocab, dim, hidden_ld, weight_ld, itype


def zs_linear_cross_entropy_forward(hidden, weight, labels, loss, *, lse=None, workspace, stream=None):
    """loss[i] = log(sum_v exp(z_iv)) - z_i,labels[i] for z = hidden @ weight.T, without keeping z; 0 for
    tokens whose label is outside of the vocabulary. lse (the first term) is written where given."""
    dev, n, vocab, dim, hidden_ld, weight_ld, itype = _head(hidden, weight, labels)
    if loss is None:
        raise ValueError("loss must be a device tensor")
    ws, ws_bytes = _workspace(workspace, dev)
    _call("zs_linear_cross_entropy_forward", dev, stream, hidden.data_ptr(), hidden_ld, _DTYPES[hidden.dtype],
          weight.data_ptr(), weight_ld, labels.data_ptr(), itype, n, vocab, dim,
          _vector(loss, "loss", n, dev, torch.float32), _vector(lse, "lse", n, dev, torch.float32), ws, ws_bytes)


def zs_linear_cross_entropy_backward(hidden, weight, labels, lse, dhidden, dweight, *, dloss=None, scale=1.0,
                                     first=False, workspace, stream=None):
    """dhidden, and (0 if first else the old value) + the head's gradient in dweight, for a loss whose
    gradient is scale * dloss[i] for token i (dloss None: ones); lse is the forward pass's."""
    dev, n, vocab, dim, hidden_ld, weight_ld, itype = _head(hidden, weight, labels)
    dh_rows, dh_dim, dh_ld = _rows2d(dhidden, "dhidden", dev)
    dw_rows, dw_dim, dw_ld = _rows2d(dweight, "dweight", dev)
    if dh_rows != n or dh_dim != dim or dhidden.dtype != hidden.dtype:
        raise ValueError("dhidden must have hidden's rows, width and dtype")
    if dw_rows != vocab or dw_dim != dim:
        raise ValueError("dweight must have weight's rows and width")
    if lse is None:
        raise ValueError("lse is that of the forward pass")
    ws, ws_bytes = _workspace(workspace, dev)
    _call("zs_linear_cross_entropy_backward", dev, stream, hidden.data_ptr(), hidden_ld, _DTYPES[hidden.dtype],
          weight.data_ptr(), weight_ld, labels.data_ptr(), itype, _vector(lse, "lse", n, dev, torch.float32),
          _vector(dloss, "dloss", n, dev, torch.float32), float(scale), n, vocab, dim, dhidden.data_ptr(), dh_ld,
          dweight.data_ptr(), _DTYPES[dweight.dtype], dw_ld, 1 if first else 0, ws, ws_bytes)


def zs_version() -> int:
    return int(_lib().zs_version())
