"""Binding of the block operators (include/lc_moe_block.h): argument marshalling only.

Low-level entry points carry the C names; ``select``, ``route_select``, ``select_backward``,
``forward_picks``, ``block_norm``, ``block_norm_backward``, ``quantize_matrix``, ``matmul_fp8``,
``linear_fp8`` and ``linear_fp8_backward`` check their tensors (dtype, shape, device, contiguous),
allocate outputs and a workspace with torch where needed and call them on the current stream of
the tensors' device.
"""
from __future__ import annotations

import ctypes

import torch

from . import BF16, LcMoeError, Shape, Weights, _check, _weights, lc_moe_workspace_size, lib
from .train import _apart, _dtype_code, _nbytes, _need, _on, _on_gpu, _p, _space, _stream

SCORES = {"softmax": 0, "sigmoid": 1}
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2


class Gating(ctypes.Structure):
    """How a router's logits become picks and gates (see lc_moe_gating): score "softmax" or
    "sigmoid"; the experts in `groups` equal runs of which a token picks from the `top_groups` best,
    judged by the sum of their `group_rank` largest scores; renorm: a token's gates sum to scale."""
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_rank", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, score="softmax", groups=1, top_groups=1, group_rank=1, renorm=False, scale=1.0):
        if score not in SCORES:
            raise ValueError(f"score {score!r}, expected one of {sorted(SCORES)}")
        super().__init__(SCORES[score], groups, top_groups, group_rank, int(bool(renorm)), scale)


class Norm(ctypes.Structure):
    _fields_ = [("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("gate_kind", ctypes.c_int32)]


_vp, _sz, _i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
_P = ctypes.POINTER
_int = ctypes.c_int
_SIG = {
    "lc_moe_select": (_int, [_P(Shape), _P(Gating)] + [_vp] * 6),
    "lc_moe_route_select": (_int, [_P(Shape), _P(Gating)] + [_vp] * 7 + [_sz, _vp]),
    "lc_moe_select_backward": (_int, [_P(Shape), _P(Gating)] + [_vp] * 6),
    "lc_moe_forward_picks": (_int, [_P(Shape), _vp, _P(Weights)] + [_vp] * 5 + [_sz, _vp]),
    "lc_moe_block_norm": (_int, [_i32] * 3 + [_P(Norm)] + [_vp] * 8),
    "lc_moe_block_norm_backward_workspace_size": (_sz, [_i32] * 3),
    "lc_moe_block_norm_backward": (_int, [_i32] * 3 + [_P(Norm)] + [_vp] * 13 + [_sz, _vp]),
    "lc_moe_fp8_matrix_size": (_sz, [_i32] * 2),
    "lc_moe_quantize_matrix": (_int, [_vp] + [_i32] * 3 + [_vp] * 3),
    "lc_moe_matmul_fp8_workspace_size": (_sz, [_i32] * 3),
    "lc_moe_matmul_fp8": (_int, [_i32] * 3 + [_vp] * 5 + [_sz, _vp]),
    "lc_moe_linear_fp8_workspace_size": (_sz, [_i32] * 3),
    "lc_moe_linear_fp8": (_int, [_i32] * 3 + [_vp] * 5 + [_sz, _vp]),
    "lc_moe_linear_fp8_backward_workspace_size": (_sz, [_i32] * 3),
    "lc_moe_linear_fp8_backward": (_int, [_i32] * 3 + [_vp] * 7 + [_sz, _vp]),
}
EXPORTED = tuple(_SIG)
_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        handle = lib()
        for name, (res, args) in _SIG.items():
            f = getattr(handle, name)
            f.restype, f.argtypes = res, args
        _LIB = handle
    return _LIB


# ---- low-level: same names and argument order as the C-ABI ------------------------------

def lc_moe_select(shape, gating, logits, bias, token_mask, topk_idx, topk_gate, stream=None):
    _check(_lib().lc_moe_select(ctypes.byref(shape), ctypes.byref(gating), _p(logits), _p(bias), _p(token_mask),
                               _p(topk_idx), _p(topk_gate), _stream(stream)), "lc_moe_select")


def lc_moe_route_select(shape, gating, x, w_router, bias, token_mask, topk_idx, topk_gate, workspace, stream=None):
    _check(_lib().lc_moe_route_select(ctypes.byref(shape), ctypes.byref(gating), _p(x), _p(w_router), _p(bias),
                                     _p(token_mask), _p(topk_idx), _p(topk_gate), _p(workspace), _nbytes(workspace),
                                     _stream(stream)), "lc_moe_route_select")


def lc_moe_select_backward(shape, gating, logits, topk_idx, dgate, dlogits_aux, dlogits, stream=None):
    _check(_lib().lc_moe_select_backward(ctypes.byref(shape), ctypes.byref(gating), _p(logits), _p(topk_idx),
                                        _p(dgate), _p(dlogits_aux), _p(dlogits), _stream(stream)),
           "lc_moe_select_backward")


def lc_moe_forward_picks(shape, x, weights, topk_idx, topk_gate, y, load, workspace, stream=None):
    _check(_lib().lc_moe_forward_picks(ctypes.byref(shape), _p(x), ctypes.byref(weights), _p(topk_idx), _p(topk_gate),
                                      _p(y), _p(load), _p(workspace), _nbytes(workspace), _stream(stream)),
           "lc_moe_forward_picks")


def lc_moe_block_norm(T, d, dtype, norm, x, y, gate, w_post, w_pre, h, z, stream=None):
    _check(_lib().lc_moe_block_norm(T, d, dtype, ctypes.byref(norm), _p(x), _p(y), _p(gate), _p(w_post), _p(w_pre),
                                   _p(h), _p(z), _stream(stream)), "lc_moe_block_norm")


def lc_moe_block_norm_backward_workspace_size(T, d, dtype) -> int:
    return _lib().lc_moe_block_norm_backward_workspace_size(T, d, dtype)


def lc_moe_block_norm_backward(T, d, dtype, norm, h, dh, dz, y, gate, w_post, w_pre, dx, dy, dw_pre, dw_post, dgate,
                               workspace, stream=None):
    _check(_lib().lc_moe_block_norm_backward(T, d, dtype, ctypes.byref(norm), _p(h), _p(dh), _p(dz), _p(y), _p(gate),
                                            _p(w_post), _p(w_pre), _p(dx), _p(dy), _p(dw_pre), _p(dw_post), _p(dgate),
                                            _p(workspace), _nbytes(workspace), _stream(stream)),
           "lc_moe_block_norm_backward")


def lc_moe_fp8_matrix_size(rows, cols) -> int:
    return _lib().lc_moe_fp8_matrix_size(rows, cols)


def lc_moe_quantize_matrix(x, rows, cols, block_rows, out, out_t, stream=None):
    _check(_lib().lc_moe_quantize_matrix(_p(x), rows, cols, block_rows, _p(out), _p(out_t), _stream(stream)),
           "lc_moe_quantize_matrix")


def lc_moe_matmul_fp8_workspace_size(M, N, K) -> int:
    return _lib().lc_moe_matmul_fp8_workspace_size(M, N, K)


def lc_moe_matmul_fp8(M, N, K, a, b, add, out, workspace, stream=None):
    _check(_lib().lc_moe_matmul_fp8(M, N, K, _p(a), _p(b), _p(add), _p(out), _p(workspace), _nbytes(workspace),
                                   _stream(stream)), "lc_moe_matmul_fp8")


def lc_moe_linear_fp8_workspace_size(T, k, n) -> int:
    return _lib().lc_moe_linear_fp8_workspace_size(T, k, n)


def lc_moe_linear_fp8(T, k, n, x, w, add, y, workspace, stream=None):
    _check(_lib().lc_moe_linear_fp8(T, k, n, _p(x), _p(w), _p(add), _p(y), _p(workspace), _nbytes(workspace),
                                   _stream(stream)), "lc_moe_linear_fp8")


def lc_moe_linear_fp8_backward_workspace_size(T, k, n) -> int:
    return _lib().lc_moe_linear_fp8_backward_workspace_size(T, k, n)


def lc_moe_linear_fp8_backward(T, k, n, dy, x, w_t, dx_add, dx, dw, workspace, stream=None):
    _check(_lib().lc_moe_linear_fp8_backward(T, k, n, _p(dy), _p(x), _p(w_t), _p(dx_add), _p(dx), _p(dw),
                                            _p(workspace), _nbytes(workspace), _stream(stream)),
           "lc_moe_linear_fp8_backward")


# ---- choice of experts --------------------------------------------------------------------

def _split(E):
    """(N, Z) with N + Z = E: these operators read only the sum."""
    return (E, 0) if E <= 2048 else (2048, E - 2048)


def _select_shape(T, E, K):
    N, Z = _split(E)
    return Shape(T, 8, N, Z, K, 8, BF16)


def select(logits, bias, K, gating, token_mask=None):
    """(topk_idx int32 [T,K], topk_gate fp32 [T,K]) from router logits fp32 [T,E]: see lc_moe_select.
    bias fp32 [E] or None; token_mask uint8 [T] or None."""
    T, E = logits.shape
    dev = logits.device
    _need(logits, "logits", (T, E), torch.float32, dev)
    if bias is not None:
        _need(bias, "bias", (E,), torch.float32, dev)
    if token_mask is not None:
        _need(token_mask, "token_mask", (T,), torch.uint8, dev)
    _on_gpu(dev)
    idx = torch.empty(T, K, dtype=torch.int32, device=dev)
    gate = torch.empty_like(idx, dtype=torch.float32)
    _on(dev, lc_moe_select, _select_shape(T, E, K), gating, logits, bias, token_mask, idx, gate)
    return idx, gate


def route_select(x, w_router, bias, K, N, gating, token_mask=None, workspace=None):
    """(topk_idx, topk_gate) of tokens x [T,d]: router logits with w_router fp32 [E,d], the first N
    of them FFN experts, then ``select``.  workspace: that of the layer (``forward_picks`` on the same one keeps the logits
    where ``forward_saved`` finds them); default a new one."""
    T, d = x.shape
    E, dev = w_router.shape[0], x.device
    _need(x, "x", (T, d), x.dtype, dev)
    _need(w_router, "w_router", (E, d), torch.float32, dev)
    if bias is not None:
        _need(bias, "bias", (E,), torch.float32, dev)
    if token_mask is not None:
        _need(token_mask, "token_mask", (T,), torch.uint8, dev)
    shape = Shape(T, d, N, E - N, K, 8, _dtype_code(x, "x"))
    ws = _space(lc_moe_workspace_size(shape), workspace, dev, "lc_moe_workspace_size", (x, w_router, bias, token_mask))
    idx = torch.empty(T, K, dtype=torch.int32, device=dev)
    gate = torch.empty_like(idx, dtype=torch.float32)
    _on(dev, lc_moe_route_select, shape, gating, x, w_router, bias, token_mask, idx, gate, ws)
    return idx, gate


def select_backward(logits, topk_idx, dgate, gating, dlogits_aux=None):
    """dlogits fp32 [T,E]: see lc_moe_select_backward.  ``router_backward`` takes it as dlogits_aux
    (with dgate None) to the tokens and the router weight."""
    T, E = logits.shape
    K, dev = topk_idx.shape[1], logits.device
    _need(logits, "logits", (T, E), torch.float32, dev)
    _need(topk_idx, "topk_idx", (T, K), torch.int32, dev)
    _need(dgate, "dgate", (T, K), torch.float32, dev)
    if dlogits_aux is not None:
        _need(dlogits_aux, "dlogits_aux", (T, E), torch.float32, dev)
    _on_gpu(dev)
    dlogits = torch.empty_like(logits)
    _on(dev, lc_moe_select_backward, _select_shape(T, E, K), gating, logits, topk_idx, dgate, dlogits_aux, dlogits)
    return dlogits


def forward_picks(x, topk_idx, topk_gate, w_gate, w_up, w_down, Z, workspace=None, fp8=None, packed=None,
                  fp8_act=False):
    """dict(y, load): the layer for the picks and gates given; Z zero-computation experts.  Weights
    as ``forward`` takes them: with fp8 or packed, w_gate, w_up and w_down are not read (tensors
    without storage, of their sizes, will do)."""
    T, d = x.shape
    N, I, _ = w_gate.shape
    K, dev = topk_idx.shape[1], x.device
    _need(x, "x", (T, d), x.dtype, dev)
    _need(topk_idx, "topk_idx", (T, K), torch.int32, dev)
    _need(topk_gate, "topk_gate", (T, K), torch.float32, dev)
    plain = fp8 is None and packed is None
    for name, w, size in (("w_gate", w_gate, (N, I, d)), ("w_up", w_up, (N, I, d)), ("w_down", w_down, (N, d, I))):
        if plain:
            _need(w, name, size, x.dtype, dev)
        elif w.shape != size:
            raise ValueError(f"{name}: shape {tuple(w.shape)}, expected {size}")
    shape = Shape(T, d, N, Z, K, I, _dtype_code(x, "x"))
    ws = _space(lc_moe_workspace_size(shape), workspace, dev, "lc_moe_workspace_size",
                (x, topk_idx, topk_gate, *((w_gate, w_up, w_down) if plain else (fp8, packed))))
    y = torch.empty_like(x)
    load = torch.empty(N + Z, dtype=torch.int32, device=dev)
    _on(dev, lc_moe_forward_picks, shape, x, _weights(None, None, w_gate, w_up, w_down, fp8, packed, fp8_act), topk_idx,
        topk_gate, y, load, ws)
    return dict(y=y, load=load)


# ---- norms around a block -----------------------------------------------------------------

def _norm_args(rows, name, y, gate, w_post, w_pre, residual_scale, block_scale, eps):
    T, d = rows.shape
    dev, code = rows.device, _dtype_code(rows, name)
    _need(rows, name, (T, d), rows.dtype, dev)
    if y is not None:
        _need(y, "y", (T, d), rows.dtype, dev)
    elif gate is not None or w_post is not None:
        raise TypeError("gate and w_post need y")
    kind = GATE_NONE
    if gate is not None:
        kind = GATE_TOKEN if gate.dim() == 2 else GATE_CHANNEL
        _need(gate, "gate", (T, 1) if kind == GATE_TOKEN else (d,), torch.float32, dev)
    for n, w in (("w_post", w_post), ("w_pre", w_pre)):
        if w is not None:
            _need(w, n, (d,), torch.float32, dev)
    _on_gpu(dev)
    return T, d, code, Norm(residual_scale, block_scale, eps, kind)


def block_norm(x, w_pre, y=None, w_post=None, gate=None, residual_scale=1.0, block_scale=1.0, eps=1e-6):
    """(h, z): h = residual_scale x + block_scale gate rms(y) w_post, z = rms(h) w_pre (see
    lc_moe_block_norm).  x, y [T,d]; w_pre, w_post fp32 [d] or None (no z; y as it is); gate fp32
    [d] (a factor of each channel), [T,1] (of each token) or None.  Without y, h is None when it
    would be x itself."""
    T, d, code, norm = _norm_args(x, "x", y, gate, w_post, w_pre, residual_scale, block_scale, eps)
    h = torch.empty_like(x) if y is not None or residual_scale != 1.0 else None
    z = torch.empty_like(x) if w_pre is not None else None
    _on(x.device, lc_moe_block_norm, T, d, code, norm, x, y, gate, w_post, w_pre, h, z)
    return h, z


def block_norm_backward(h, w_pre, dz, dh=None, y=None, w_post=None, gate=None, residual_scale=1.0, block_scale=1.0,
                        eps=1e-6, workspace=None):
    """The gradient of block_norm: dict(dx, and those of dy, dw_pre, dw_post, dgate whose inputs
    are given).  h: the forward's (x itself where that was None); dz, dh: the gradients of z and h
    or None; the rest as in the forward."""
    if dz is not None and w_pre is None:
        raise TypeError("dz needs w_pre")
    T, d, code, norm = _norm_args(h, "h", y, gate, w_post, w_pre, residual_scale, block_scale, eps)
    dev = h.device
    for n, t in (("dz", dz), ("dh", dh)):
        if t is not None:
            _need(t, n, (T, d), h.dtype, dev)
    ws = _space(lc_moe_block_norm_backward_workspace_size(T, d, code), workspace, dev,
                "lc_moe_block_norm_backward_workspace_size", (h, dh, dz, y, gate, w_post, w_pre))
    out = dict(dx=torch.empty_like(h))
    if y is not None:
        out["dy"] = torch.empty_like(y)
    for n, w in (("dw_pre", w_pre), ("dw_post", w_post), ("dgate", gate)):
        if w is not None:
            out[n] = torch.empty_like(w)
    _on(dev, lc_moe_block_norm_backward, T, d, code, norm, h, dh, dz, y, gate, w_post, w_pre, out["dx"], out.get("dy"),
        out.get("dw_pre"), out.get("dw_post"), out.get("dgate"), ws)
    return out


# ---- products in block FP8 ----------------------------------------------------------------

class Fp8Matrix:
    """A matrix in block FP8: `data` its buffer (codes and scales, see lc_moe_fp8_matrix_size), and
    `t` the buffer of its transpose, either None if it was not asked for.  block_rows: rows that
    share a scale; with 128 both forms hold the same values, with 1 each has its own."""

    def __init__(self, rows, cols, data, t, block_rows=128):
        self.rows, self.cols, self.data, self.t, self.block_rows = rows, cols, data, t, block_rows
        self.device = (data if data is not None else t).device


def quantize_matrix(x, block_rows=128, rows=True, transposed=False):
    """Block-FP8 form of a bf16 matrix [R,C] (C a multiple of 8): a scale for each 128 x 128 block
    (block_rows 128) or for each run of 128 of a row, in the transpose of a column (block_rows 1).
    rows, transposed: which of the two forms are made."""
    R, C = x.shape
    dev = x.device
    _need(x, "x", (R, C), torch.bfloat16, dev)
    _on_gpu(dev)
    if not rows and not transposed:
        raise ValueError("quantize_matrix: rows or transposed is needed")

    def room(r, c):
        size = lc_moe_fp8_matrix_size(r, c)
        if size == 0:
            raise LcMoeError(2, "lc_moe_fp8_matrix_size")
        return torch.empty(size, dtype=torch.uint8, device=dev)

    m = Fp8Matrix(R, C, room(R, C) if rows else None, room(C, R) if transposed else None, block_rows)
    _on(dev, lc_moe_quantize_matrix, x, R, C, block_rows, m.data, m.t)
    return m


def _buffer(buf, name, rows, cols, dev):
    if buf is None:
        raise TypeError(f"{name} lacks the form that is needed (quantize_matrix makes both)")
    _need(buf, name, (lc_moe_fp8_matrix_size(rows, cols),), torch.uint8, dev)


def _added(add, out, name, size, dev, others):
    if add is not None:
        _need(add, name, size, torch.bfloat16, dev)
    if out is not None:
        _need(out, "out", size, torch.bfloat16, dev)
        same = add is not None and add.data_ptr() == out.data_ptr()
        _apart("out", out, (*others, None if same else add))
        return out
    return torch.empty(*size, dtype=torch.bfloat16, device=dev)


def matmul_fp8(a, b, add=None, out=None, workspace=None):
    """A B^T + add, bf16 [M,N], of Fp8Matrix A [M,K] and B [N,K] (see lc_moe_matmul_fp8).  out: where
    to write it (may be add itself); default a new tensor."""
    M, K, N, dev = a.rows, a.cols, b.rows, a.device
    if b.cols != K:
        raise ValueError(f"{K} columns of a, {b.cols} of b")
    _buffer(a.data, "a", M, K, dev)
    _buffer(b.data, "b", N, K, dev)
    out = _added(add, out, "add", (M, N), dev, (a.data, b.data))
    ws = _space(lc_moe_matmul_fp8_workspace_size(M, N, K), workspace, dev, "lc_moe_matmul_fp8_workspace_size",
                (a.data, b.data, add, out))
    _on(dev, lc_moe_matmul_fp8, M, N, K, a.data, b.data, add, out, ws)
    return out


def linear_fp8(x, w, add=None, out=None, workspace=None):
    """y = Q(x) W^T + add, bf16 [T,n]: x bf16 [T,k], w the quantize_matrix of a weight [n,k] (see
    lc_moe_linear_fp8).  out: where to write it (may be add itself)."""
    T, k = x.shape
    n, dev = w.rows, x.device
    _need(x, "x", (T, w.cols), torch.bfloat16, dev)
    _buffer(w.data, "w", n, k, dev)
    y = _added(add, out, "add", (T, n), dev, (x, w.data))
    ws = _space(_lib().lc_moe_linear_fp8_workspace_size(T, k, n), workspace, dev, "lc_moe_linear_fp8_workspace_size",
                (x, w.data, add, y))
    _on(dev, lc_moe_linear_fp8, T, k, n, x, w.data, add, y, ws)
    return y


def linear_fp8_backward(dy, x, w, dx_add=None, dx=None, need_dx=True, need_dw=True, workspace=None):
    """The gradient of linear_fp8 with FP8 operands: dict(dx [T,k], dw [n,k]), bf16 (see
    lc_moe_linear_fp8_backward).  w: quantize_matrix(weight, transposed=True), whose transpose holds the
    values that linear_fp8 multiplied by.  dx: where to write it (may be dx_add itself)."""
    T, k = x.shape
    n, dev = w.rows, x.device
    _need(x, "x", (T, w.cols), torch.bfloat16, dev)
    _need(dy, "dy", (T, n), torch.bfloat16, dev)
    out = {}
    if need_dx:
        if w.block_rows != 128:
            raise ValueError(f"w: block_rows {w.block_rows}, expected 128: its transpose holds other values than w")
        _buffer(w.t, "w", k, n, dev)
        out["dx"] = _added(dx_add, dx, "dx_add", (T, k), dev, (x, dy, w.t))
    if need_dw:
        out["dw"] = torch.empty(n, k, dtype=torch.bfloat16, device=dev)
    ws = _space(_lib().lc_moe_linear_fp8_backward_workspace_size(T, k, n), workspace, dev,
                "lc_moe_linear_fp8_backward_workspace_size", (x, dy, w.t, dx_add, out.get("dx")))
    _on(dev, lc_moe_linear_fp8_backward, T, k, n, dy, x, w.t, dx_add, out.get("dx"), out.get("dw"), ws)
    return out
