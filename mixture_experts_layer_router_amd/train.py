"""Binding of the training operators (include/lc_moe_train.h): argument marshalling only.

Low-level entry points carry the C names (``lc_moe_forward_saved``, ``lc_moe_balance_loss``,
``lc_moe_gate_backward``, ``lc_moe_router_backward``, ``lc_moe_adamw`` and the two workspace
sizes); ``forward_saved``, ``balance_loss``, ``gate_backward``, ``router_backward``,
``layer_backward`` and ``AdamW`` check their tensors (dtype, shape, device, contiguous),
allocate outputs and a workspace with torch where needed and call them on the current stream
of the tensors' device.
"""
from __future__ import annotations

import ctypes

import torch

from . import BF16, F32, LcMoeError, Shape, _check, ffn_backward, lib


class Saved(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("ffn_rows", ctypes.c_void_p), ("slot_row", ctypes.c_void_p),
                ("ffn_offsets", ctypes.c_void_p), ("perm_token", ctypes.c_void_p)]


class BalanceCoef(ctypes.Structure):
    _fields_ = [("balance", ctypes.c_float), ("z", ctypes.c_float)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("weight_decay", ctypes.c_float), ("lr_scale", ctypes.c_float)]


class AdamwHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("state_bits", ctypes.c_int32), ("step", ctypes.c_int32), ("step_dev", ctypes.c_void_p),
                ("grad_scale", ctypes.c_void_p), ("seed", ctypes.c_uint32)]


_vp, _sz, _i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
_P = ctypes.POINTER
_SIG = {
    "lc_moe_forward_saved": (ctypes.c_int, [_P(Shape), _vp, _sz, _P(Saved)]),
    "lc_moe_balance_workspace_size": (_sz, [_P(Shape), _i32]),
    "lc_moe_balance_loss": (ctypes.c_int, [_P(Shape), _P(BalanceCoef), _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                           _vp, _sz, _vp]),
    "lc_moe_gate_backward": (ctypes.c_int, [_P(Shape), _vp, _vp, _i32, _vp, _vp, _vp, _vp]),
    "lc_moe_router_backward_workspace_size": (_sz, [_P(Shape)]),
    "lc_moe_router_backward": (ctypes.c_int, [_P(Shape)] + [_vp] * 11 + [_sz, _vp]),
    "lc_moe_adamw": (ctypes.c_int, [_P(AdamwTensor), _i32, _P(AdamwHyper), _vp]),
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
# Addresses go as plain integers (the argument types are declared above): a call costs a few
# microseconds, which counts for layers of few tokens.

def _p(t):
    return None if t is None else t.data_ptr()


def _nbytes(t):
    return 0 if t is None else t.nbytes


def _stream(stream):
    """The stream's handle; None: the current stream of the current device."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def lc_moe_forward_saved(shape, workspace) -> Saved:
    out = Saved()
    _check(_lib().lc_moe_forward_saved(ctypes.byref(shape), _p(workspace), _nbytes(workspace), ctypes.byref(out)),
           "lc_moe_forward_saved")
    return out


def lc_moe_balance_workspace_size(shape, num_seqs) -> int:
    return _lib().lc_moe_balance_workspace_size(ctypes.byref(shape), num_seqs)


def lc_moe_balance_loss(shape, coef, logits, topk_idx, seq_offsets, num_seqs, token_mask, loss, load, prob, dlogits,
                        workspace, stream=None):
    _check(_lib().lc_moe_balance_loss(ctypes.byref(shape), ctypes.byref(coef), _p(logits), _p(topk_idx),
                                     _p(seq_offsets), num_seqs, _p(token_mask), _p(loss), _p(load), _p(prob),
                                     _p(dlogits), _p(workspace), _nbytes(workspace), _stream(stream)),
           "lc_moe_balance_loss")


def lc_moe_gate_backward(shape, x, ffn_rows, num_rows, slot_row, dy, dgate, stream=None):
    _check(_lib().lc_moe_gate_backward(ctypes.byref(shape), _p(x), _p(ffn_rows), num_rows, _p(slot_row), _p(dy),
                                      _p(dgate), _stream(stream)), "lc_moe_gate_backward")


def lc_moe_router_backward_workspace_size(shape) -> int:
    return _lib().lc_moe_router_backward_workspace_size(ctypes.byref(shape))


def lc_moe_router_backward(shape, x, w_router, logits, topk_idx, dgate, dlogits_aux, dx_add, dx, dw_router, dlogits,
                           workspace, stream=None):
    _check(_lib().lc_moe_router_backward(ctypes.byref(shape), _p(x), _p(w_router), _p(logits), _p(topk_idx), _p(dgate),
                                        _p(dlogits_aux), _p(dx_add), _p(dx), _p(dw_router), _p(dlogits),
                                        _p(workspace), _nbytes(workspace), _stream(stream)), "lc_moe_router_backward")


def lc_moe_adamw(tensors, count, hyper, stream=None):
    _check(_lib().lc_moe_adamw(tensors, count, ctypes.byref(hyper), _stream(stream)), "lc_moe_adamw")


# ---- checked wrappers -------------------------------------------------------------------

def _need(t, name, shape, dtype, device):
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _given(t, name):
    if t is None:
        raise TypeError(f"{name} is required")


def _dtype_code(t, name):
    if t.dtype is torch.bfloat16:
        return BF16
    if t.dtype is torch.float32:
        return F32
    raise TypeError(f"{name}: {t.dtype}, expected torch.bfloat16 or torch.float32")


def _on(device, call, *args):
    """call(*args) with the tensors' device current: a launch goes to the device its stream
    belongs to."""
    if device.type != "cuda" or device.index == torch._C._cuda_getDevice():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _on_gpu(device):
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}; the operators run on the GPU")


def _apart(name, t, others):
    """t, which a call writes, shares no memory with the others (contiguous tensors or None)."""
    lo, hi = t.data_ptr(), t.data_ptr() + t.nbytes
    for q in others:
        if q is not None and q.nbytes and lo < q.data_ptr() + q.nbytes and q.data_ptr() < hi:
            raise ValueError(f"{name} overlaps another tensor of the call")


def _space(size, given, device, where, used=()):
    if given is not None:
        if given.device != device or not given.is_contiguous():
            raise ValueError(f"workspace: a contiguous tensor on {device} is needed")
        _apart("workspace", given, used)
    _on_gpu(device)
    if size == 0:
        raise LcMoeError(2, where)
    return torch.empty(size, dtype=torch.uint8, device=device) if given is None else given


def forward_saved(x, N, Z, K, I, workspace):
    """The forward's intermediates as views of its workspace, valid until another call uses
    it: dict(logits fp32 [T,E], ffn_rows [T*K,d], slot_row int32 [T,K], ffn_offsets int32
    [N+1], perm_token int32 [T*K]).  x and the sizes are those of the forward."""
    T, d = x.shape
    shape = Shape(T, d, N, Z, K, I, _dtype_code(x, "x"))
    s = lc_moe_forward_saved(shape, workspace)
    base, flat = workspace.data_ptr(), workspace.view(torch.uint8).reshape(-1)

    def view(addr, dtype, *size):
        n = torch.empty((), dtype=dtype).element_size()
        for v in size:
            n *= v
        return flat[addr - base:addr - base + n].view(dtype).view(size)

    return dict(logits=view(s.logits, torch.float32, T, N + Z), ffn_rows=view(s.ffn_rows, x.dtype, T * K, d),
                slot_row=view(s.slot_row, torch.int32, T, K), ffn_offsets=view(s.ffn_offsets, torch.int32, N + 1),
                perm_token=view(s.perm_token, torch.int32, T * K))


def balance_loss(logits, topk_idx, N, balance_coef, z_coef=0.0, seq_offsets=None, token_mask=None, need_grad=True,
                 workspace=None):
    """dict(loss fp32 [2] (balance, z), load int32 [S,E], prob fp32 [S,E], dlogits fp32 [T,E]
    or None): see lc_moe_balance_loss.  logits fp32 [T,E]; topk_idx int32 [T,K]; seq_offsets
    int32 [S+1] or None (one sequence); token_mask uint8 [T] or None."""
    T, E = logits.shape
    K, dev = topk_idx.shape[1], logits.device
    S = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
    _need(logits, "logits", (T, E), torch.float32, dev)
    _need(topk_idx, "topk_idx", (T, K), torch.int32, dev)
    if seq_offsets is not None:
        _need(seq_offsets, "seq_offsets", (S + 1,), torch.int32, dev)
    if token_mask is not None:
        _need(token_mask, "token_mask", (T,), torch.uint8, dev)
    shape = Shape(T, 8, N, E - N, K, 8, BF16)
    ws = _space(lc_moe_balance_workspace_size(shape, S), workspace, dev, "lc_moe_balance_workspace_size",
                (logits, topk_idx, seq_offsets, token_mask))
    out = dict(loss=logits.new_empty(2), load=topk_idx.new_empty((S, E)), prob=logits.new_empty((S, E)),
               dlogits=torch.empty_like(logits) if need_grad else None)
    _on(dev, lc_moe_balance_loss, shape, BalanceCoef(balance_coef, z_coef), logits, topk_idx, seq_offsets, S,
        token_mask, out["loss"], out["load"], out["prob"], out["dlogits"], ws)
    return out


def gate_backward(x, ffn_rows, slot_row, dy):
    """dgate fp32 [T,K]: gradient of sum <dy, y> with respect to every pick's gate; x, dy [T,d];
    ffn_rows [R,d] and slot_row int32 [T,K] as forward_saved gives them."""
    T, d = x.shape
    K, dev = slot_row.shape[1], x.device
    code = _dtype_code(x, "x")
    _need(x, "x", (T, d), x.dtype, dev)
    _need(dy, "dy", (T, d), x.dtype, dev)
    _need(slot_row, "slot_row", (T, K), torch.int32, dev)
    _need(ffn_rows, "ffn_rows", (ffn_rows.shape[0], d), x.dtype, dev)
    _on_gpu(dev)
    N = min(K, 2048)
    dgate = torch.empty((T, K), dtype=torch.float32, device=dev)
    _on(dev, lc_moe_gate_backward, Shape(T, d, N, K - N, K, 8, code), x, ffn_rows, min(ffn_rows.shape[0], T * K),
        slot_row, dy, dgate)
    return dgate


def router_backward(x, w_router, logits, topk_idx, dgate, N, dlogits_aux=None, dx_add=None, dx=None, need_dx=True,
                    need_dw=True, need_dlogits=False, workspace=None):
    """dict(dx [T,d], dw_router fp32 [E,d] and, if asked for, dlogits fp32 [T,E]): see
    lc_moe_router_backward.  dgate None: no gradient from the gates (logits and topk_idx may
    then be None).  dx: where to write it (may be dx_add itself); default a new tensor."""
    T, d = x.shape
    E, dev = w_router.shape[0], x.device
    code = _dtype_code(x, "x")
    K = topk_idx.shape[1] if topk_idx is not None else 1
    _need(x, "x", (T, d), x.dtype, dev)
    _need(w_router, "w_router", (E, d), torch.float32, dev)
    if dgate is not None:
        _given(logits, "logits")
        _given(topk_idx, "topk_idx")
        _need(dgate, "dgate", (T, K), torch.float32, dev)
        _need(logits, "logits", (T, E), torch.float32, dev)
        _need(topk_idx, "topk_idx", (T, K), torch.int32, dev)
    if dlogits_aux is not None:
        _need(dlogits_aux, "dlogits_aux", (T, E), torch.float32, dev)
    if dx_add is not None:
        _need(dx_add, "dx_add", (T, d), x.dtype, dev)
    if dx is not None:
        _need(dx, "dx", (T, d), x.dtype, dev)
        same = dx_add is not None and dx_add.data_ptr() == dx.data_ptr()
        _apart("dx", dx, (x, w_router, logits, topk_idx, dgate, dlogits_aux, None if same else dx_add))
    shape = Shape(T, d, N, E - N, K, 8, code)
    ws = _space(lc_moe_router_backward_workspace_size(shape), workspace, dev, "lc_moe_router_backward_workspace_size",
                (x, w_router, logits, topk_idx, dgate, dlogits_aux, dx_add, dx))
    out = {}
    if need_dx:
        out["dx"] = dx if dx is not None else torch.empty_like(x)
    if need_dw:
        out["dw_router"] = torch.empty_like(w_router)
    if need_dlogits:
        out["dlogits"] = torch.empty((T, E), dtype=torch.float32, device=dev)
    _on(dev, lc_moe_router_backward, shape, x, w_router, logits, topk_idx, dgate, dlogits_aux, dx_add, out.get("dx"),
        out.get("dw_router"), out.get("dlogits"), ws)
    return out


def layer_backward(x, w_router, w_gate, w_up, w_down, out, dy, workspace, balance_coef=0.0, z_coef=0.0,
                   seq_offsets=None, token_mask=None):
    """The gradient of a whole layer, sum <dy, y> + balance loss + z loss: dict(dx, dw_router,
    dw_gate, dw_up, dw_down, dgate, loss, load, prob).  ``out`` and ``workspace`` are those of
    ``forward(x, ..., workspace=workspace)`` on bf16 tensors; the workspace is read and not
    written.  The losses are left out (loss None) if both coefficients are 0."""
    T, _ = x.shape
    N, I, _ = w_gate.shape
    E, K = w_router.shape[0], out["topk_idx"].shape[1]
    saved = forward_saved(x, N, E - N, K, I, workspace)
    bal = dict(loss=None, load=None, prob=None, dlogits=None)
    if balance_coef or z_coef:
        bal = balance_loss(saved["logits"], out["topk_idx"], N, balance_coef, z_coef, seq_offsets, token_mask)
    dgate = gate_backward(x, saved["ffn_rows"], saved["slot_row"], dy)
    grads = _on(x.device, ffn_backward, x, w_gate, w_up, w_down, out["topk_idx"], out["topk_gate"], dy, E - N)
    r = router_backward(x, w_router, saved["logits"], out["topk_idx"], dgate, N, dlogits_aux=bal["dlogits"],
                        dx_add=grads["dx"], dx=grads["dx"])
    return dict(grads, dw_router=r["dw_router"], dgate=dgate, loss=bal["loss"], load=bal["load"], prob=bal["prob"])


def adamw_state(param, state_bits=32):
    """(m, v, m_scale, v_scale) of a new optimizer: zeros in fp32, or codes and exponent bytes."""
    n, dev = param.numel(), param.device
    if state_bits == 32:
        return (torch.zeros(n, dtype=torch.float32, device=dev), torch.zeros(n, dtype=torch.float32, device=dev),
                None, None)
    blocks = -(-n // 128)
    codes = [torch.zeros(n, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.full((blocks,), 127, dtype=torch.uint8, device=dev) for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


class AdamW:
    """AdamW over a fixed list of tensors (see lc_moe_adamw): bf16 or fp32 weights, gradients
    in buffers that keep their place, states fp32 (state_bits 32) or E4M3 (8).  States that
    are not given start as zeros.  masters: fp32 copies of weights, or None where there is
    none.  weight_decay and lr_scale: one number, or one for each tensor.  The object holds its
    tensors, so their addresses stay valid; it keeps no other state."""

    def __init__(self, params, grads, m=None, v=None, m_scales=None, v_scales=None, masters=None, state_bits=32,
                 weight_decay=0.0, lr_scale=1.0):
        n = len(params)
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        if n == 0:
            raise ValueError("AdamW needs at least one tensor")
        if (m is None) != (v is None):
            raise ValueError("m and v are given together")
        if m is None:
            made = [adamw_state(p, state_bits) for p in params]
            m, v, m_scales, v_scales = ([t[i] for t in made] for i in range(4))
        masters = masters if masters is not None else [None] * n
        if state_bits == 32:
            m_scales = v_scales = [None] * n
        wd = [weight_decay] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        ls = [lr_scale] * n if isinstance(lr_scale, (int, float)) else list(lr_scale)
        lists = (grads, m, v, m_scales, v_scales, masters, wd, ls)
        if any(a is None or len(a) != n for a in lists):
            raise ValueError(f"AdamW: every list needs {n} entries")
        # what a step writes shares no memory with anything else of it; gradients may be shared
        spans = []
        for name, ts in (("params", params), ("m", m), ("v", v), ("m_scales", m_scales), ("v_scales", v_scales),
                         ("masters", masters), ("grads", grads)):
            spans += [(t.data_ptr(), t.data_ptr() + t.nbytes, f"{name}[{i}]") for i, t in enumerate(ts)
                      if t is not None and t.numel()]
        end, last, grads_end, last_grad = 0, "", 0, ""
        for lo, hi, name in sorted(spans):
            written = not name.startswith("grads")
            if lo < end or (written and lo < grads_end):
                raise ValueError(f"AdamW: {name} overlaps {last if lo < end else last_grad}")
            if written:
                end, last = hi, name
            elif hi > grads_end:
                grads_end, last_grad = hi, name
        self.params, self.grads, self.m, self.v = list(params), list(grads), list(m), list(v)
        self.m_scales, self.v_scales, self.masters = list(m_scales), list(v_scales), list(masters)
        self.state_bits, self.device = state_bits, params[0].device
        self._tensors = (AdamwTensor * n)()
        state = torch.float32 if state_bits == 32 else torch.uint8
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        for i, t in enumerate(self.params):
            size, blocks = t.numel(), (-(-t.numel() // 128),)
            _need(t, f"params[{i}]", t.shape, t.dtype, self.device)
            _need(self.grads[i], f"grads[{i}]", t.shape, self.grads[i].dtype, self.device)
            for name, q in (("m", self.m[i]), ("v", self.v[i])):
                _need(q, f"{name}[{i}]", q.shape, state, self.device)
                if q.numel() != size:
                    raise ValueError(f"{name}[{i}]: {q.numel()} elements, expected {size}")
            if state_bits == 8:
                _need(self.m_scales[i], f"m_scales[{i}]", blocks, torch.uint8, self.device)
                _need(self.v_scales[i], f"v_scales[{i}]", blocks, torch.uint8, self.device)
            if self.masters[i] is not None:
                _need(self.masters[i], f"masters[{i}]", t.shape, torch.float32, self.device)
            self._tensors[i] = AdamwTensor(p(t), p(self.masters[i]), p(self.grads[i]), p(self.m[i]), p(self.v[i]),
                                           p(self.m_scales[i]), p(self.v_scales[i]), size,
                                           _dtype_code(t, f"params[{i}]"),
                                           _dtype_code(self.grads[i], f"grads[{i}]"), wd[i], ls[i])
        _on_gpu(self.device)

    def step(self, lr, beta1=0.9, beta2=0.95, eps=1e-8, step=None, seed=0, grad_scale=None, step_dev=None):
        """One step on the current stream.  step: its number, from 1 on (the object does not count),
        or step_dev: an int32 tensor of one element to read it from; one of the two is needed.
        grad_scale: an fp32 tensor of one element."""
        if step_dev is not None:
            step = 1  # not read
        elif step is None or not 1 <= step < 1 << 31:
            raise ValueError(f"AdamW: step {step}: the number of the step, from 1 on, or step_dev is needed")
        for name, t, dtype in (("grad_scale", grad_scale, torch.float32), ("step_dev", step_dev, torch.int32)):
            if t is not None and (t.dtype != dtype or t.numel() != 1 or t.device != self.device):
                raise ValueError(f"{name}: one {dtype} on {self.device} is needed")
        hyper = AdamwHyper(lr, beta1, beta2, eps, self.state_bits, step,
                           None if step_dev is None else step_dev.data_ptr(),
                           None if grad_scale is None else grad_scale.data_ptr(), seed & 0xFFFFFFFF)
        _on(self.device, lc_moe_adamw, self._tensors, len(self._tensors), hyper)
