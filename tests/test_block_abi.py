"""The block operators' entry points (include/lc_moe_block.h): every declared one is exported and
bound, a C99 program can include and call them, and bad arguments are refused on the host with
the documented status before anything is enqueued."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import mixture_experts_layer_router_amd as lm
from mixture_experts_layer_router_amd import block as lb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lc_moe_block.h")
P = 1 << 20
Q = 1 << 21
MIS = P + 4
OK, NULLPTR, SHAPE, DTYPE, ALIGN, WORKSPACE = range(6)
BIG = 1 << 50


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(lc_moe_[a-z0-9_]+)\s*\(", src)))


def shape(**kw):
    a = dict(T=64, d=128, N=8, Z=4, K=2, I=256, dtype=lm.BF16)
    a.update(kw)
    return lm.make_shape(**a)


def test_every_declared_symbol_is_exported():
    assert set(declared()) == set(lb.EXPORTED)
    for n in declared():
        assert hasattr(lm.lib(), n), n


def test_c_program_links(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "p.c"
    src.write_text('#include "lc_moe_block.h"\nstatic void* const e[] = {%s};\nint main(void) {\n'
                   "  const lc_moe_gating g = {LC_MOE_SIGMOID, 1, 1, 1, 1, 2.5f};\n"
                   "  int f = 0; unsigned i; for (i = 0; i < sizeof e / sizeof e[0]; ++i) f += e[i] == 0;\n"
                   "  f += lc_moe_select(0, &g, 0, 0, 0, 0, 0, 0) != LC_MOE_E_NULLPTR;\n"
                   "  f += lc_moe_fp8_matrix_size(1, 1) != 256 + 256 + 256;\n  return f;\n}\n"
                   % ", ".join("(void*)" + n for n in declared()))
    pkg = os.path.dirname(lm.LIB_PATH)
    exe = tmp_path / "p"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-isystem", "/opt/rocm/include", str(src), "-L", pkg, "-llc_moe", "-L", "/opt/rocm/lib",
                    "-lamdhip64", "-Wl,-rpath," + pkg, "-Wl,-rpath,/opt/rocm/lib", "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def ref(v):
    return ctypes.byref(v) if v is not None else None


def gating(**kw):
    return lm.Gating(**kw)


def raw_gating(score=0, groups=1, top=1, rank=1, renorm=0, scale=1.0):
    g = lm.Gating()
    g.score, g.groups, g.top_groups, g.group_rank, g.renorm, g.scale = score, groups, top, rank, renorm, scale
    return g


def test_select_refusals():
    def call(sh=shape(), g=raw_gating(), logits=P, bias=P, mask=P, idx=P, gate=P):
        return lb._lib().lc_moe_select(ref(sh), ref(g), logits, bias, mask, idx, gate, None)
    assert call(sh=None) == NULLPTR and call(g=None) == NULLPTR
    for k in ("logits", "idx", "gate"):
        assert call(**{k: None}) == NULLPTR, k
    for k in ("logits", "bias", "mask", "idx", "gate"):
        assert call(**{k: MIS}) == ALIGN, k
    for kw in (dict(score=2), dict(groups=0), dict(groups=5), dict(groups=4, top=5), dict(top=0), dict(rank=0),
               dict(rank=3), dict(groups=12, top=12, rank=2), dict(groups=12, top=1), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(g=raw_gating(**kw)) == SHAPE, kw
    assert call(sh=shape(N=128, K=65)) == SHAPE and call(sh=shape(T=0)) == SHAPE
    assert call(sh=shape(N=130, Z=0), g=raw_gating(groups=65, top=65)) == SHAPE
    assert call(sh=shape(dtype=7)) == DTYPE


def test_route_select_refusals():
    s = shape()
    n = lm.lc_moe_workspace_size(s)

    def call(sh=s, g=raw_gating(), x=P, w=P, bias=P, mask=P, idx=P, gate=P, ws=P, nb=n):
        return lb._lib().lc_moe_route_select(ref(sh), ref(g), x, w, bias, mask, idx, gate, ws, nb, None)
    for k in ("x", "w", "idx", "gate", "ws"):
        assert call(**{k: None}) == NULLPTR, k
    for k in ("x", "w", "bias", "mask", "idx", "gate", "ws"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(nb=n - 1) == WORKSPACE and call(g=raw_gating(groups=5)) == SHAPE


def test_select_backward_refusals():
    def call(sh=shape(), g=raw_gating(), logits=P, idx=P, dg=P, aux=P, dl=P):
        return lb._lib().lc_moe_select_backward(ref(sh), ref(g), logits, idx, dg, aux, dl, None)
    assert call(sh=None) == NULLPTR and call(g=None) == NULLPTR
    for k in ("logits", "idx", "dg", "dl"):
        assert call(**{k: None}) == NULLPTR, k
    for k in ("logits", "idx", "dg", "aux", "dl"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(g=raw_gating(score=-1)) == SHAPE and call(sh=shape(N=128, K=65)) == SHAPE
    assert call(g=raw_gating(scale=float("nan"))) == SHAPE


def test_forward_picks_refusals():
    s = shape()
    n = lm.lc_moe_workspace_size(s)

    def call(sh=s, x=P, idx=P, gate=P, y=P, load=P, ws=P, nb=n, null=False, **w):
        wt = lm.Weights(None, None, *[w.get(k, P) for k in ("w_gate", "w_up", "w_down")], w.get("fp8"), w.get("packed"),
                        w.get("fp8_act", 0))
        return lb._lib().lc_moe_forward_picks(ref(sh), x, None if null else ref(wt), idx, gate, y, load, ws, nb, None)
    assert call(sh=None) == NULLPTR and call(null=True) == NULLPTR
    for k in ("x", "idx", "gate", "y", "ws", "w_gate", "w_up", "w_down"):
        assert call(**{k: None}) == NULLPTR, k
    for k in ("x", "idx", "gate", "y", "load", "ws", "w_gate", "fp8"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(fp8=P, packed=P) == DTYPE and call(fp8_act=1) == DTYPE and call(nb=n - 1) == WORKSPACE


def norm(a=1.0, b=1.0, eps=1e-6, kind=0):
    return lb.Norm(a, b, eps, kind)


def test_block_norm_refusals():
    def call(T=4, d=64, dt=lm.BF16, n=norm(kind=1), x=P, y=P, gate=P, wp=P, wq=P, h=P, z=Q):
        return lb._lib().lc_moe_block_norm(T, d, dt, ref(n), x, y, gate, wp, wq, h, z, None)
    assert call(n=None) == NULLPTR
    for k in ("x", "gate", "wq", "y"):
        assert call(**{k: None}) == NULLPTR, k
    for k in ("x", "y", "gate", "wp", "wq", "h", "z"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(T=-1) == SHAPE and call(T=1 << 24) == SHAPE and call(d=0) == SHAPE and call(d=60) == SHAPE
    assert call(d=16392) == SHAPE and call(dt=2) == DTYPE and call(z=P) == SHAPE
    for bad in (norm(eps=0.0), norm(eps=1e-39), norm(eps=float("nan")), norm(eps=float("inf")), norm(a=float("inf")),
                norm(b=float("nan")), norm(kind=3), norm(kind=-1)):
        assert call(n=bad) == SHAPE
    assert call(T=0, x=None, y=None, gate=None, h=None, z=None) == OK
    assert call(h=None, z=None) == OK  # nothing to write
    assert call(n=norm(), y=None, gate=None, wp=P) == NULLPTR


def test_block_norm_backward_refusals():
    size = lb.lc_moe_block_norm_backward_workspace_size
    n = size(4, 64, lm.BF16)
    assert n > 0 and size(0, 64, lm.F32) > 0
    assert size(-1, 64, 1) == size(4, 60, 1) == size(4, 64, 5) == size(4, 16392, 1) == 0

    def call(T=4, d=64, dt=lm.BF16, nm=norm(kind=1), h=P, dh=P, dz=P, y=P, gate=P, wp=P, wq=P, dx=P, dy=Q, dwq=P, dwp=P,
             dg=P, ws=P, nb=n):
        return lb._lib().lc_moe_block_norm_backward(T, d, dt, ref(nm), h, dh, dz, y, gate, wp, wq, dx, dy, dwq, dwp, dg,
                                                    ws, nb, None)
    assert call(nm=None) == NULLPTR
    for k in ("h", "y", "gate", "wq", "wp", "ws"):
        assert call(**{k: None}) == NULLPTR, k
    for k in ("h", "dh", "dz", "y", "gate", "wp", "wq", "dx", "dy", "dwq", "dwp", "dg", "ws"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(nb=n - 1) == WORKSPACE and call(dx=Q) == SHAPE and call(d=12) == SHAPE and call(dt=9) == DTYPE
    assert call(nm=norm(kind=0)) == SHAPE  # a gradient of no gate


def test_fp8_sizes_and_refusals():
    f = lb.lc_moe_fp8_matrix_size
    assert f(300, 200) == -(-300 * 256 // 256) * 256 + 2 * 512 + 256
    assert f(0, 8) == f(8, 0) == f(-1, 8) == f(1 << 24, 8) == f(8, 1 << 24) == f((1 << 24) - 1, (1 << 24) - 1) == 0
    q = lb._lib().lc_moe_quantize_matrix
    assert q(P, 4, 12, 1, P, None, None) == SHAPE and q(P, 4, 16, 2, P, None, None) == SHAPE
    assert q(P, -1, 16, 1, P, None, None) == SHAPE and q(P, 1 << 24, 16, 1, P, None, None) == SHAPE
    assert q(None, 4, 16, 1, P, None, None) == NULLPTR and q(MIS, 4, 16, 1, P, None, None) == ALIGN
    assert q(P, 4, 16, 1, MIS, None, None) == ALIGN and q(P, 4, 16, 1, None, MIS, None) == ALIGN
    assert q(P, 4, 16, 128, P, P, None) == SHAPE
    assert q(None, 0, 16, 1, None, None, None) == OK and q(P, 4, 16, 1, None, None, None) == OK


def test_matmul_refusals():
    size = lb.lc_moe_matmul_fp8_workspace_size
    n = size(64, 128, 256)
    assert n > 0 and size(0, 128, 256) > 0 and size(64, 12, 256) == 0 and size(-1, 8, 8) == 0 and size(8, 8, 0) == 0
    assert size((1 << 24) - 1, (1 << 24) - 8, 8) == 0  # more tiles than a grid holds

    def call(M=64, N=128, K=256, a=P, b=P, add=P, out=P, ws=P, nb=n):
        return lb._lib().lc_moe_matmul_fp8(M, N, K, a, b, add, out, ws, nb, None)
    for k in ("a", "b", "out", "ws"):
        assert call(**{k: None}) == NULLPTR, k
    for k in ("a", "b", "add", "out", "ws"):
        assert call(**{k: MIS}) == ALIGN, k
    assert call(N=4) == SHAPE and call(M=-1) == SHAPE and call(K=0) == SHAPE
    assert call(M=0, a=None, b=None, out=None, ws=None, nb=0) == OK
    assert call(nb=n - 1) == WORKSPACE


def test_linear_refusals():
    lib = lb._lib()
    n = lib.lc_moe_linear_fp8_workspace_size(64, 256, 128)
    nb_ = lib.lc_moe_linear_fp8_backward_workspace_size(64, 256, 128)
    assert n > 0 and nb_ > 0
    for T, k, m in ((-1, 256, 128), (64, 12, 128), (64, 256, 12), (64, 0, 128), (1 << 24, 256, 128)):
        assert lib.lc_moe_linear_fp8_workspace_size(T, k, m) == 0
        assert lib.lc_moe_linear_fp8_backward_workspace_size(T, k, m) == 0
        assert lib.lc_moe_linear_fp8(T, k, m, P, P, None, P, P, BIG, None) == SHAPE
        assert lib.lc_moe_linear_fp8_backward(T, k, m, P, P, P, None, P, P, P, BIG, None) == SHAPE

    def fw(T=64, x=P, w=P, add=P, y=P, ws=P, nb=n):
        return lib.lc_moe_linear_fp8(T, 256, 128, x, w, add, y, ws, nb, None)
    for k in ("x", "w", "y", "ws"):
        assert fw(**{k: None}) == NULLPTR, k
    for k in ("x", "w", "add", "y", "ws"):
        assert fw(**{k: MIS}) == ALIGN, k
    assert fw(nb=n - 1) == WORKSPACE and fw(T=0, x=None, w=None, y=None, ws=None, nb=0) == OK
    assert fw() == SHAPE and fw(add=None) == SHAPE  # y is x

    def bw(T=64, dy=P, x=P, w=P, add=P, dx=P, dw=P, ws=P, nb=nb_):
        return lib.lc_moe_linear_fp8_backward(T, 256, 128, dy, x, w, add, dx, dw, ws, nb, None)
    for k in ("dy", "x", "w", "ws"):
        assert bw(**{k: None}) == NULLPTR, k
    for k in ("dy", "x", "w", "add", "dx", "dw", "ws"):
        assert bw(**{k: MIS}) == ALIGN, k
    assert bw(nb=nb_ - 1) == WORKSPACE and bw(T=0, dw=None) == OK and bw(dx=None, dw=None) == OK
    assert bw() == SHAPE and bw(dw=None) == SHAPE  # dx is dy


def test_wrappers_refuse_tensors_off_the_gpu():
    import torch
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    lg = torch.zeros(4, 16)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: lm.select(lg, None, 2, lm.Gating()),
                 lambda: lm.route_select(x, lg, None, 2, 16, lm.Gating()),
                 lambda: lm.select_backward(lg, idx, torch.zeros(4, 2), lm.Gating()),
                 lambda: lm.block_norm(x, torch.ones(16)),
                 lambda: lm.block_norm_backward(x, torch.ones(16), x),
                 lambda: lm.quantize_matrix(x)):
        with pytest.raises(ValueError):
            call()


def test_wrappers_check_their_tensors():
    import torch
    lg, b = torch.zeros(4, 16), torch.zeros(16)
    with pytest.raises(ValueError):
        lm.Gating("tanh")
    with pytest.raises(TypeError):
        lm.select(lg.double(), b, 2, lm.Gating())
    with pytest.raises(ValueError):
        lm.select(lg, b[:8], 2, lm.Gating())
    with pytest.raises(ValueError):
        lm.select(torch.zeros(16, 4).t(), b, 2, lm.Gating())
    with pytest.raises(TypeError):
        lm.select(lg, b, 2, lm.Gating(), token_mask=torch.ones(4, dtype=torch.bool))
    x = torch.zeros(4, 16)
    with pytest.raises(TypeError):
        lm.block_norm(x, b, gate=b)
    with pytest.raises(ValueError):
        lm.block_norm(x, b, y=x, gate=torch.ones(4, 2))
    with pytest.raises(ValueError):
        lm.block_norm(x, b, y=x[:2])
    with pytest.raises(TypeError):
        lm.block_norm(x.double(), b)
    with pytest.raises(TypeError):
        lm.block_norm_backward(x, None, x)
    with pytest.raises(TypeError):
        lm.quantize_matrix(x)
    m = lm.Fp8Matrix(8, 16, torch.zeros(lb.lc_moe_fp8_matrix_size(8, 16), dtype=torch.uint8), None)
    y = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        lm.linear_fp8_backward(torch.zeros(4, 8, dtype=torch.bfloat16), y, m)  # lacks the transpose
    with pytest.raises(ValueError):
        lm.linear_fp8(y[:, :8].contiguous(), m)
    out = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lm.linear_fp8(y, m, out=y.view(-1)[:32].view(4, 8))  # over the tokens
    with pytest.raises(ValueError):
        lm.linear_fp8(y, m, add=out, out=out.view(-1)[1:].new_zeros(8, 4))
