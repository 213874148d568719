"""The training operators' entry points (include/lc_moe_train.h): every declared one is
exported and bound, a C99 program can include and call them, and bad arguments are refused on
the host with the documented status before anything is enqueued."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import mixture_experts_layer_router_amd as lm
from mixture_experts_layer_router_amd import train as lt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lc_moe_train.h")
P = 1 << 20
MIS = P + 4


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(lc_moe_[a-z0-9_]+)\s*\(", src)))


def shape(**kw):
    a = dict(T=64, d=128, N=8, Z=4, K=2, I=256, dtype=lm.BF16)
    a.update(kw)
    return lm.make_shape(**a)


def test_every_declared_symbol_is_exported():
    assert set(declared()) == set(lt.EXPORTED)
    for n in declared():
        assert hasattr(lm.lib(), n), n


def test_forward_saved():
    s = shape()
    n = lm.lc_moe_workspace_size(s)
    out = lt.Saved()
    f = lt._lib().lc_moe_forward_saved
    assert f(ctypes.byref(s), P, n, ctypes.byref(out)) == 0
    assert out.logits >= P and P <= out.ffn_rows < P + n and out.slot_row % 256 == 0
    assert out.ffn_rows + 64 * 2 * 128 * 2 <= P + n
    assert f(None, P, n, ctypes.byref(out)) == 1
    assert f(ctypes.byref(s), P, n, None) == 1
    assert f(ctypes.byref(s), None, n, ctypes.byref(out)) == 1
    assert f(ctypes.byref(s), MIS, n, ctypes.byref(out)) == 4
    assert f(ctypes.byref(s), P, n - 1, ctypes.byref(out)) == 5
    assert f(ctypes.byref(shape(K=13)), P, n, ctypes.byref(out)) == 2


def test_balance_refusals():
    s = shape()
    size = lt.lc_moe_balance_workspace_size
    n = size(s, 3)
    assert n > 0 and size(s, 0) == 0 and size(s, 65536) == 0 and size(shape(T=0), 1) == 0 and size(s, 65535) > 0
    coef = lt.BalanceCoef(0.01, 0.0)

    def call(sh=s, c=coef, logits=P, idx=P, off=P, seqs=3, mask=P, loss=P, load=P, prob=P, dl=P, ws=P, nb=n):
        return lt._lib().lc_moe_balance_loss(ctypes.byref(sh) if sh is not None else None,
                                             ctypes.byref(c) if c is not None else None, logits, idx, off, seqs, mask,
                                             loss, load, prob, dl, ws, nb, None)

    assert call(sh=None) == 1 and call(c=None) == 1
    for k in ("logits", "idx", "off", "loss", "load", "prob", "ws"):
        assert call(**{k: None}) == 1, k
    for k in ("logits", "idx", "off", "mask", "loss", "load", "prob", "dl", "ws"):
        assert call(**{k: MIS}) == 4, k
    assert call(seqs=0) == 2 and call(seqs=65536) == 2 and call(seqs=-1) == 2
    assert call(nb=n - 1) == 5
    assert call(sh=shape(K=13)) == 2 and call(sh=shape(dtype=9)) == 3


def test_gate_refusals():
    def call(sh=shape(), x=P, rows=P, num=128, slot=P, dy=P, dg=P):
        return lt._lib().lc_moe_gate_backward(ctypes.byref(sh) if sh is not None else None, x, rows, num, slot, dy, dg,
                                              None)
    assert call(sh=None) == 1
    for k in ("x", "rows", "slot", "dy", "dg"):
        assert call(**{k: None}) == 1, k
        assert call(**{k: MIS}) == 4, k
    assert call(num=129) == 2 and call(num=-1) == 2 and call(sh=shape(d=100)) == 2 and call(sh=shape(dtype=3)) == 3


def test_router_backward_refusals():
    s = shape()
    n = lt.lc_moe_router_backward_workspace_size(s)
    assert n > 0 and lt.lc_moe_router_backward_workspace_size(shape(d=4)) == 0
    # as large as the layer itself may be
    huge = shape(T=1 << 20, d=1 << 14, K=1, dtype=lm.F32)
    assert lm.lc_moe_workspace_size(huge) > 0 and lt.lc_moe_router_backward_workspace_size(huge) > 0

    def call(sh=s, x=P, w=P, lg=P, idx=P, dg=P, aux=P, add=P, dx=P, dw=P, dl=P, ws=P, nb=n):
        return lt._lib().lc_moe_router_backward(ctypes.byref(sh) if sh is not None else None, x, w, lg, idx, dg, aux,
                                                add, dx, dw, dl, ws, nb, None)
    assert call(sh=None) == 1
    for k in ("x", "w", "lg", "idx", "ws"):
        assert call(**{k: None}) == 1, k
    for k in ("x", "w", "lg", "idx", "dg", "aux", "add", "dx", "dw", "dl", "ws"):
        assert call(**{k: MIS}) == 4, k
    assert call(nb=n - 1) == 5 and call(sh=shape(K=13)) == 2 and call(sh=shape(dtype=2)) == 3


def test_adamw_refusals():
    f = lt._lib().lc_moe_adamw
    good = dict(param=P, master=None, grad=P, m=P, v=P, m_scale=P, v_scale=P, n=100, param_dtype=1, grad_dtype=0,
                weight_decay=0.1, lr_scale=1.0)
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, state_bits=8, step=1, step_dev=None, grad_scale=None, seed=0)

    def call(h=None, count=1, null=False, **kw):
        t = (lt.AdamwTensor * 1)(lt.AdamwTensor(**dict(good, **kw)))
        return f(None if null else t, count, ctypes.byref(lt.AdamwHyper(**dict(hyper, **(h or {})))), None)

    assert f(None, 0, None, None) == 1
    assert call(count=0) == 0 and call(count=0, null=True) == 0 and call(null=True) == 1 and call(count=-1) == 2
    assert call(n=0, param=None, grad=None, m=None) == 0
    for k in ("param", "grad", "m", "v", "m_scale", "v_scale"):
        assert call(**{k: None}) == 1, k
    for k in ("param", "master", "grad", "m", "v", "m_scale", "v_scale"):
        assert call(**{k: MIS}) == 4, k
    assert call(n=-1) == 2 and call(n=1 << 40) == 2
    assert call(param_dtype=2) == 3 and call(grad_dtype=-1) == 3
    for h in (dict(state_bits=16), dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0),
              dict(beta1=float("nan")), dict(eps=float("nan"))):
        assert call(h=h) == 2, h
    assert call(h=dict(step_dev=MIS)) == 4 and call(h=dict(grad_scale=MIS)) == 4


def test_adamw_refuses_a_subnormal_eps():
    f = lt._lib().lc_moe_adamw
    for eps, status in ((0.0, 0), (2.0 ** -126, 0), (2.0 ** -127, 2), (2.0 ** -149, 2)):
        h = lt.AdamwHyper(1e-3, 0.9, 0.95, eps, 32, 1, None, None, 0)
        assert f(None, 0, ctypes.byref(h), None) == status, eps


def test_wrapper_refusals():
    """The checked wrappers refuse tensors of another type, shape or layout (on the CPU: they
    get no further than their checks)."""
    import torch
    T, E, K, d = 6, 8, 2, 16
    lg, idx = torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32)
    bad = [lambda: lm.balance_loss(lg.double(), idx, 4, 0.1), lambda: lm.balance_loss(lg, idx.long(), 4, 0.1),
           lambda: lm.balance_loss(lg.t().contiguous().t(), idx, 4, 0.1), lambda: lm.balance_loss(lg, idx[:-1], 4, 0.1),
           lambda: lm.balance_loss(lg, idx, 4, 0.1, token_mask=torch.ones(T, dtype=torch.bool)),
           lambda: lm.balance_loss(lg, idx, 4, 0.1, seq_offsets=torch.zeros(3)),
           lambda: lm.gate_backward(torch.zeros(T, d), torch.zeros(5, d + 4), idx, torch.zeros(T, d)),
           lambda: lm.gate_backward(torch.zeros(T, d, dtype=torch.float16), torch.zeros(5, d), idx, torch.zeros(T, d)),
           lambda: lm.router_backward(torch.zeros(T, d), torch.zeros(E, d), lg, idx, torch.zeros(T, K + 1), 4),
           lambda: lm.router_backward(torch.zeros(T, d), torch.zeros(E, d), None, idx, torch.zeros(T, K), 4),
           lambda: lm.AdamW([], []), lambda: lm.AdamW([lg], [lg], state_bits=16),
           lambda: lm.AdamW([lg], [lg, lg]), lambda: lm.AdamW([lg], [lg[:3]]),
           lambda: lm.AdamW([lg], [lg], m=[lg]), lambda: lm.AdamW([lg], [lg], masters=[lg.double()]),
           lambda: lm.AdamW([lg], [lg], m=[lg], v=[lg], state_bits=8),
           # one tensor twice
           lambda: lm.AdamW([lg, lg], [lg, lg]),
           # all in order, but not on a GPU
           lambda: lm.balance_loss(lg, idx, 4, 0.1), lambda: lm.AdamW([lg], [lg]),
           lambda: lm.gate_backward(torch.zeros(T, d), torch.zeros(5, d), idx, torch.zeros(T, d)),
           lambda: lm.router_backward(torch.zeros(T, d), torch.zeros(E, d), lg, idx, torch.zeros(T, K), 4)]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            f()
            pytest.fail(f"call {i} was not refused")


def test_wrappers_refuse_overlaps():
    """What a call writes may not lie over what else it reads or writes, but for what the header
    allows (the CPU tensors of the allowed calls are refused for being on the CPU)."""
    import torch
    T, E, K, d, n = 6, 8, 2, 16, 100
    f = torch.zeros(4 * n)
    p, g, m, v = (f[i * n:(i + 1) * n] for i in range(4))
    b = torch.zeros(n, dtype=torch.uint8)
    s = [torch.zeros(1, dtype=torch.uint8) for _ in range(2)]
    lg, idx = torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32)
    x, w, add, dg = torch.zeros(T, d), torch.zeros(E, d), torch.zeros(T, d), torch.zeros(T, K)
    two = torch.zeros(2 * T * d)
    space = lambda t: t.view(-1).view(torch.uint8)  # noqa: E731
    bad = [lambda: lm.AdamW([p], [g], m=[m], v=[m]), lambda: lm.AdamW([p], [p], m=[m], v=[v]),
           lambda: lm.AdamW([p], [g], m=[g], v=[v]), lambda: lm.AdamW([p], [g], masters=[p]),
           lambda: lm.AdamW([f[:n], f[n - 1:2 * n - 1]], [v, v]), lambda: lm.AdamW([f[1:n]], [f[:n - 1]]),
           lambda: lm.AdamW([p], [g], m=[b], v=[b.clone()], m_scales=s[:1], v_scales=s[:1], state_bits=8),
           lambda: lm.AdamW([f[n:2 * n], f[2 * n:3 * n]], [f[:n], f[:n]], masters=[f[3 * n:], f[3 * n:]]),
           # a long gradient in front of short weights
           lambda: lm.AdamW([f[:1], f[2:3], f[:0]], [f[1:2], f[1:2], f[:0]], m=[f[4:5], f[5:6], p[:0]],
                            v=[f[6:7], f[5:6], p[:0]]),
           lambda: lm.router_backward(x, w, lg, idx, dg, 4, dx=x),
           lambda: lm.router_backward(x, w, lg, idx, dg, 4, dx_add=two[:T * d].view(T, d), dx=two[4:T * d + 4].view(T, d)),
           lambda: lm.router_backward(x, w, lg, idx, dg, 4, workspace=space(lg)),
           lambda: lm.router_backward(x, w, lg, idx, dg, 4, dx_add=add, dx=add, workspace=space(add)),
           lambda: lm.balance_loss(lg, idx, 4, 0.1, workspace=space(lg)),
           lambda: lm.balance_loss(lg, idx, 4, 0.1, workspace=space(idx))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="overlaps"):
            call()
            pytest.fail(f"call {i} was not refused")
    good = [lambda: lm.AdamW([p, v], [g, g]), lambda: lm.AdamW([p], [g], m=[m], v=[v]),
            lambda: lm.AdamW([p[:0], p, p[:0]], [g[:0], g, g[:0]]),
            lambda: lm.router_backward(x, w, lg, idx, dg, 4, dx_add=add, dx=add),
            lambda: lm.router_backward(x, w, lg, idx, dg, 4, dx_add=x, workspace=torch.zeros(4))]
    for call in good:
        with pytest.raises(ValueError, match="run on the GPU"):
            call()


PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include "lc_moe_train.h"
static void* const entry_points[] = { @POINTS@ };
int main(void) {
  const lc_moe_shape s = {64, 128, 8, 4, 2, 256, LC_MOE_BF16};
  lc_moe_adamw_hyper h;
  int fails = 0;
  size_t i;
  for (i = 0; i < sizeof entry_points / sizeof entry_points[0]; ++i) fails += entry_points[i] == NULL;
  fails += lc_moe_balance_workspace_size(&s, 4) == 0;
  fails += lc_moe_router_backward_workspace_size(&s) == 0;
  memset(&h, 0, sizeof h);
  fails += lc_moe_adamw(NULL, 0, &h, NULL) != LC_MOE_E_SHAPE; /* state_bits 0 */
  h.state_bits = 32;
  h.step = 1;
  fails += lc_moe_adamw(NULL, 0, &h, NULL) != LC_MOE_OK;
  printf("failures %d\n", fails);
  return fails != 0;
}
"""


def test_c99_program(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text(PROGRAM.replace("@POINTS@", ", ".join(f"(void*){n}" for n in declared())))
    pkg = os.path.join(ROOT, "mixture_experts_layer_router_amd")
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                        "-isystem", "/opt/rocm/include", str(src), "-L", pkg, "-llc_moe", "-L/opt/rocm/lib",
                        "-lamdhip64", f"-Wl,-rpath,{pkg}:/opt/rocm/lib", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
