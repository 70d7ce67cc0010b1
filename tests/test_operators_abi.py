"""Refusals of the norm, the scored router and the FP8 calls: statuses from the host's checks
before any launch (no GPU), the binding's checks of tensors, and the same host code under
AddressSanitizer."""
import math
import os
import subprocess

import pytest
import torch

import mixture_experts_layer_33_amd as moe
from mixture_experts_layer_33_amd import _lib
from mixture_experts_layer_33_amd import build as libbuild

FAKE, ODD = 0x1000, 0x1008
L = _lib.lib


def shape(dtype="bf16", T=16, d=256, E=8, k=2, f=128, C=None):
    return moe.make_shape(T, d, E, k, f, C, dtype=dtype)


def norm(s, x=FAKE, r=FAKE, w=FAKE, eps=1e-6, h=FAKE, y=FAKE, y8=None, ys=None, rstd=FAKE):
    return L().moe_add_rmsnorm(s, x, r, w, eps, h, y, y8, ys, rstd, None)


def test_norm_refusals():
    s = shape()
    for bad in (dict(x=None), dict(w=None), dict(y=None)):
        assert norm(s, **bad) == _lib.MOE_ERR_NULL, bad
    for bad in (dict(x=ODD), dict(r=ODD), dict(w=ODD), dict(h=ODD), dict(y=ODD), dict(rstd=FAKE + 2)):
        assert norm(s, **bad) == _lib.MOE_ERR_ALIGN, bad
    for eps in (-1e-6, math.nan, math.inf):
        assert norm(s, eps=eps) == _lib.MOE_ERR_SHAPE
    assert norm(s, y8=FAKE, ys=FAKE) == _lib.MOE_ERR_DTYPE            # 8-bit rows need an 8-bit layer
    assert norm(shape("f32"), y8=FAKE, ys=FAKE) == _lib.MOE_ERR_DTYPE
    for ty in ("fp8", "mxfp8"):
        assert norm(shape(ty), y8=FAKE) == _lib.MOE_ERR_NULL
        assert norm(shape(ty), ys=FAKE) == _lib.MOE_ERR_NULL
        assert norm(shape(ty), y8=ODD, ys=FAKE) == _lib.MOE_ERR_ALIGN
    assert norm(shape("f32", T=(1 << 23) + 1, d=8, f=8)) == _lib.MOE_ERR_SHAPE
    assert norm(shape(d=100)) == _lib.MOE_ERR_SHAPE and norm(None) == _lib.MOE_ERR_NULL
    assert norm(shape(T=0), x=None, r=None, h=None, y=None, rstd=None) == _lib.MOE_OK


def norm_bwd(s, dy=FAKE, dh=FAKE, h=FAKE, w=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 30):
    return L().moe_add_rmsnorm_backward(s, dy, dh, h, w, rstd, dx, dw, ws, n, None)


def test_norm_backward_refusals():
    s = shape()
    for bad in (dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(ws=None)):
        assert norm_bwd(s, **bad) == _lib.MOE_ERR_NULL, bad
    for bad in (dict(dy=ODD), dict(dh=ODD), dict(h=ODD), dict(w=ODD), dict(dx=ODD), dict(dw=ODD), dict(ws=ODD)):
        assert norm_bwd(s, **bad) == _lib.MOE_ERR_ALIGN, bad
    need = moe.workspace_bytes(s, moe.OP_NORM_BACKWARD)
    assert need >= 256 * 4 and norm_bwd(s, n=need - 1) == _lib.MOE_ERR_WORKSPACE


def rule(score=1, groups=4, top_groups=2, group_top=2, renormalise=1, scale=2.5):
    return _lib.MoeRouter(score, groups, top_groups, group_top, renormalise, scale)


def route(s, r, x=FAKE, w=FAKE, idx=FAKE, gate=FAKE, cnt=FAKE, ws=FAKE, n=1 << 30):
    return L().moe_route_scored(s, r, x, w, None, None, idx, gate, cnt, None, ws, n, None)


def route_bwd(s, r, dg=FAKE, x=FAKE, w=FAKE, l=FAKE, idx=FAKE, dxi=None, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 30):
    return L().moe_route_scored_backward(s, r, dg, None, x, w, l, idx, dxi, dx, dw, None, ws, n, None)


@pytest.mark.parametrize("bad", [dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=65),
                                 dict(top_groups=0), dict(top_groups=5), dict(group_top=0), dict(group_top=3),
                                 dict(groups=8, top_groups=2, group_top=2), dict(groups=8, top_groups=1, group_top=1),
                                 dict(renormalise=2), dict(scale=math.nan), dict(scale=math.inf)], ids=str)
def test_rules_refused(bad):
    s = shape()                 # 8 experts, top 2
    assert route(s, rule(**bad)) == _lib.MOE_ERR_SHAPE
    assert route_bwd(s, rule(**bad)) == _lib.MOE_ERR_SHAPE


def test_route_scored_refusals():
    s, r = shape(), rule()
    assert route(s, None) == _lib.MOE_ERR_NULL and route_bwd(s, None) == _lib.MOE_ERR_NULL
    for bad in (dict(x=None), dict(w=None), dict(idx=None), dict(gate=None), dict(cnt=None), dict(ws=None)):
        assert route(s, r, **bad) == _lib.MOE_ERR_NULL, bad
    for bad in (dict(x=ODD), dict(w=ODD), dict(ws=ODD)):
        assert route(s, r, **bad) == _lib.MOE_ERR_ALIGN, bad
    assert route(s, r, n=moe.workspace_bytes(s, moe.OP_ROUTE) - 1) == _lib.MOE_ERR_WORKSPACE
    for bad in (dict(dg=None), dict(x=None), dict(w=None), dict(l=None), dict(idx=None), dict(dx=None), dict(dw=None), dict(ws=None)):
        assert route_bwd(s, r, **bad) == _lib.MOE_ERR_NULL, bad
    for bad in (dict(x=ODD), dict(w=ODD), dict(dxi=ODD), dict(dx=ODD), dict(dw=ODD), dict(ws=ODD)):
        assert route_bwd(s, r, **bad) == _lib.MOE_ERR_ALIGN, bad
    assert route_bwd(s, r, n=moe.workspace_bytes(s, moe.OP_ROUTE_BACKWARD) - 1) == _lib.MOE_ERR_WORKSPACE
    many = shape("f32", T=(1 << 21) + 1, d=8, f=8)
    assert route(many, r) == _lib.MOE_ERR_SHAPE and route_bwd(many, r) == _lib.MOE_ERR_SHAPE
    wide = shape(T=1, d=64 * 16384, E=1024, f=64)      # d * 4 E is 2^32
    assert route_bwd(wide, r) == _lib.MOE_ERR_SHAPE
    assert route_bwd(shape(T=1, d=64 * 16383, E=1024, f=64), r, n=0) == _lib.MOE_ERR_WORKSPACE
    with pytest.raises(KeyError):
        moe.make_router(score="tanh")


def test_backward_experts_refusals():
    def call(s, head=0, dg=FAKE, n=1 << 40):
        return L().moe_backward_experts(s, *([FAKE] * 7), head, *([FAKE] * 8), dg, FAKE, n, None)
    assert call(shape("mxfp8")) == _lib.MOE_ERR_DTYPE and call(shape("fp8")) == _lib.MOE_ERR_DTYPE
    assert call(shape(d=192)) == _lib.MOE_ERR_SHAPE
    s = shape()
    assert call(s, head=s.capacity) == _lib.MOE_ERR_SHAPE and call(s, dg=None) == _lib.MOE_ERR_NULL
    assert call(s, n=moe.workspace_bytes(s, moe.OP_BACKWARD) - 1) == _lib.MOE_ERR_WORKSPACE


def test_fp8_layer_refusals():
    for bad in (dict(d=192), dict(f=64), dict(d=100)):
        assert L().moe_check_shape(shape("fp8", **bad)) == _lib.MOE_ERR_SHAPE
    s = shape("fp8")
    assert L().moe_check_shape(s) == _lib.MOE_OK
    assert L().moe_dispatch(s, FAKE, FAKE, 0, FAKE, None, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == _lib.MOE_ERR_NULL
    ffn = [s, FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE]
    for i in (2, 8, 9, 10):      # every scale is needed
        a = list(ffn)
        a[i] = None
        assert L().moe_expert_ffn(*a, 1 << 30, None) == _lib.MOE_ERR_NULL
    assert L().moe_expert_ffn(*ffn, moe.workspace_bytes(s, moe.OP_EXPERT_FFN) - 1, None) == _lib.MOE_ERR_WORKSPACE
    for i in (1, 5, 6, 7, 11, 12, 13):
        a = list(ffn)
        a[i] = ODD
        assert L().moe_expert_ffn(*a, 1 << 30, None) == _lib.MOE_ERR_ALIGN, i
    for i in (2, 8, 9, 10):
        a = list(ffn)
        a[i] = FAKE + 2
        assert L().moe_expert_ffn(*a, 1 << 30, None) == _lib.MOE_ERR_ALIGN, i
    for x, ring, scale in ((ODD, FAKE, FAKE), (FAKE, ODD, FAKE), (FAKE, FAKE, FAKE + 2)):
        assert L().moe_dispatch(s, x, FAKE, 0, ring, scale, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == _lib.MOE_ERR_ALIGN
    # what has no FP8 form says so
    assert L().moe_forward(s, *([FAKE] * 6), 0, *([FAKE] * 10), 0, FAKE, 1 << 40, None) == _lib.MOE_ERR_DTYPE
    assert L().moe_backward_mx(s, *([FAKE] * 8), 0, *([FAKE] * 11), 1 << 40, None) == _lib.MOE_ERR_DTYPE
    assert moe.workspace_bytes(s, moe.OP_BACKWARD) == 0


def test_dispatch_q_refusals():
    def call(s, x=FAKE, xs=FAKE, head=0, ring=FAKE, rs=FAKE, n=1 << 30):
        return L().moe_dispatch_q(s, x, xs, FAKE, head, ring, rs, FAKE, FAKE, FAKE, FAKE, n, None)
    assert call(shape()) == _lib.MOE_ERR_DTYPE and call(shape("f32")) == _lib.MOE_ERR_DTYPE
    for ty in ("fp8", "mxfp8"):
        s = shape(ty)
        for bad in (dict(x=None), dict(xs=None), dict(ring=None), dict(rs=None)):
            assert call(s, **bad) == _lib.MOE_ERR_NULL
        for bad in (dict(x=ODD), dict(ring=ODD), dict(xs=FAKE + 2), dict(rs=FAKE + 1)):
            assert call(s, **bad) == _lib.MOE_ERR_ALIGN
        assert call(s, head=-1) == _lib.MOE_ERR_SHAPE and call(s, head=s.capacity) == _lib.MOE_ERR_SHAPE
        assert call(s, n=moe.workspace_bytes(s, moe.OP_DISPATCH) - 1) == _lib.MOE_ERR_WORKSPACE


def test_quantise_and_matmul_refusals():
    q = L().moe_quantize_fp8
    assert q(FAKE, 4, 96, 1, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(FAKE, 4, 128, 32, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(FAKE, -1, 128, 1, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(None, 4, 128, 1, FAKE, FAKE, None) == _lib.MOE_ERR_NULL
    assert q(ODD, 4, 128, 128, FAKE, FAKE, None) == _lib.MOE_ERR_ALIGN
    assert q(FAKE, 1 << 31, 128, 1, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(None, 0, 128, 1, None, None, None) == _lib.MOE_OK

    def mm(M=16, N=256, K=256, ty=_lib.MOE_BF16, a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, out=FAKE, ws=FAKE, n=1 << 30):
        return L().moe_matmul_fp8(a, sa, w, sw, M, N, K, ty, out, ws, n, None)
    for bad in (dict(K=192), dict(K=0), dict(M=-1), dict(N=-1), dict(M=1 << 25), dict(N=1 << 25), dict(M=1 << 31)):
        assert mm(**bad) == _lib.MOE_ERR_SHAPE, bad
    assert mm(M=1 << 22, N=1 << 22, K=128) == _lib.MOE_ERR_SHAPE
    assert mm(ty=_lib.MOE_FP8) == _lib.MOE_ERR_DTYPE
    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None)):
        assert mm(**bad) == _lib.MOE_ERR_NULL, bad
    for bad in (dict(a=ODD), dict(w=ODD), dict(sa=FAKE + 2), dict(sw=FAKE + 2), dict(out=FAKE + 1), dict(out=FAKE + 2, ty=_lib.MOE_F32)):
        assert mm(**bad) == _lib.MOE_ERR_ALIGN, bad
    assert mm(M=0, a=None, out=None) == _lib.MOE_OK and mm(N=0, w=None, out=None) == _lib.MOE_OK
    for M, N, K in ((1, 7168, 2048), (16, 256, 256), (4096, 4096, 4096)):
        need = L().moe_matmul_fp8_workspace_bytes(M, N, K)
        assert need % 256 == 0
        if need:
            assert mm(M, N, K, n=need - 1) == _lib.MOE_ERR_WORKSPACE
            assert mm(M, N, K, ws=None, n=0) == _lib.MOE_ERR_NULL
    assert L().moe_matmul_fp8_workspace_bytes(16, 256, 100) == 0


def test_binding_refuses_host_tensors_and_wrong_ones():
    s = shape("fp8")
    x = torch.zeros(16, 256, dtype=torch.bfloat16)
    w = torch.zeros(256)
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_add_rmsnorm(s, x, None, w, 1e-6, None, x.clone(), None, None, None)
    for bad in (x.float(), x[:8], x.t().contiguous().t(), torch.zeros(16, 512, dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError, match="x: needs"):
            moe.moe_add_rmsnorm(s, bad, None, w, 1e-6, None, x.clone(), None, None, None)
    with pytest.raises(ValueError, match="y8_scale"):      # FP8 scales are floats [d/128, T]
        moe.moe_add_rmsnorm(s, x, None, w, 1e-6, None, x.clone(), x.to(torch.uint8), torch.zeros(2, 16, 4, dtype=torch.uint8), None)
    with pytest.raises(ValueError, match="balance"):
        moe.moe_route_scored(s, moe.make_router(), x, torch.zeros(8, 256), None, torch.zeros(7), torch.zeros(16, 2, dtype=torch.int32),
                             torch.zeros(16, 2), torch.zeros(8, dtype=torch.int32), None, None)
    u = torch.zeros(16, 256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="w_scale"):
        moe.moe_matmul_fp8(u, torch.zeros(2, 16), u, torch.zeros(2, 2), x)
    with pytest.raises(ValueError):
        moe.moe_matmul_fp8(u, torch.zeros(2, 16), u, torch.zeros(1, 2), x.half())
    with pytest.raises(ValueError, match="multiple of 128"):
        moe.quantize_fp8(torch.zeros(2, 100, 128, dtype=torch.bfloat16), 128)
    layer = moe.Layer.create(16, 256, 8, 2, 128, dtype="fp8", device="cpu")
    with pytest.raises(ValueError):                          # codes without their scales
        layer.dispatch(u, torch.zeros(16, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="router"):
        layer.route(x, torch.zeros(8, 256), None, None, torch.zeros(8))


DRIVER = r"""
#include <cmath>
#include <cstdio>
#include "moe.h"
static int bad = 0;
static void want(const char* n, long g, long w) { if (g != w) { std::printf("FAIL %s %ld %ld\n", n, g, w); ++bad; } }
int main() {
  unsigned char* b = new unsigned char[64];
  b = (unsigned char*)(((uintptr_t)b + 15) & ~(uintptr_t)15);
  float* F = (float*)b; int32_t* I = (int32_t*)b;
  moe_shape* s = new moe_shape{16, 40, 256, 8, 2, 128, 0, MOE_FP8};
  moe_shape* h = new moe_shape{16, 40, 256, 8, 2, 128, 0, MOE_BF16};
  moe_router* r = new moe_router{MOE_SCORE_SIGMOID, 4, 2, 2, 1, 2.5f};
  moe_router* q = new moe_router{MOE_SCORE_SIGMOID, 4, 2, 2, 1, NAN};
  want("fp8 shape", moe_check_shape(s), MOE_OK);
  for (int op = 0; op <= MOE_OP_ROUTE_BACKWARD; ++op) want("ws", moe_workspace_bytes(s, op) % 256, 0);
  want("norm", moe_add_rmsnorm(s, b, b, F, -1.f, b, b, b, b, F, nullptr), MOE_ERR_SHAPE);
  want("norm y8", moe_add_rmsnorm(h, b, b, F, 0.f, b, b, b, b, F, nullptr), MOE_ERR_DTYPE);
  want("norm bwd", moe_add_rmsnorm_backward(s, b, b, b, F, F, b, F, b, 0, nullptr), MOE_ERR_WORKSPACE);
  want("route", moe_route_scored(s, r, b, F, F, F, I, F, I, F, b, 0, nullptr), MOE_ERR_WORKSPACE);
  want("route nan", moe_route_scored(s, q, b, F, F, F, I, F, I, F, b, 1 << 30, nullptr), MOE_ERR_SHAPE);
  want("route null", moe_route_scored(s, nullptr, b, F, F, F, I, F, I, F, b, 1 << 30, nullptr), MOE_ERR_NULL);
  want("route bwd", moe_route_scored_backward(s, r, F, F, b, F, F, I, b, b, F, F, b, 0, nullptr), MOE_ERR_WORKSPACE);
  want("experts", moe_backward_experts(h, b, I, F, b, I, I, I, 0, b, b, b, b, b, b, b, b, F, b, 0, nullptr), MOE_ERR_WORKSPACE);
  want("dispatch", moe_dispatch_q(s, b, b, I, 40, b, b, I, I, I, b, 1 << 30, nullptr), MOE_ERR_SHAPE);
  want("quantise", moe_quantize_fp8(b, 4, 128, 2, b, F, nullptr), MOE_ERR_SHAPE);
  want("matmul", moe_matmul_fp8(b, F, b, F, 4, 4, 100, MOE_BF16, b, b, 0, nullptr), MOE_ERR_SHAPE);
  want("string", moe_status_string(MOE_ERR_ALIGN)[0] != 0, 1);
  std::printf("ok: %d failure(s)\n", bad);
  return bad != 0;
}
"""


def test_host_code_under_address_sanitizer(tmp_path):
    objs = [os.path.join(libbuild.BUILD, os.path.splitext(s)[0] + ".o") for s in libbuild.SOURCES if s != "api.cpp"]
    if not all(os.path.exists(o) for o in objs):
        libbuild.build()
    src = tmp_path / "driver.cpp"
    src.write_text(DRIVER)
    flags = ["-O1", "-g", "-std=c++17", f"--offload-arch={libbuild.ARCH}", "-I", libbuild.INCLUDE, "-I", libbuild.CSRC,
             "-Wno-unused-command-line-argument", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-fsanitize=address"]
    for name, path, lang in (("api", os.path.join(libbuild.CSRC, "api.cpp"), ["-x", "hip"]), ("driver", str(src), [])):
        subprocess.run([libbuild.HIPCC, *flags, *lang, "-c", path, "-o", str(tmp_path / f"{name}.o")], check=True, timeout=600,
                       capture_output=True)
    exe = str(tmp_path / "driver")
    subprocess.run([libbuild.HIPCC, f"--offload-arch={libbuild.ARCH}", "-Xarch_host", "-fsanitize=address", "-o", exe,
                    str(tmp_path / "driver.o"), str(tmp_path / "api.o"), *objs], check=True, timeout=600, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1"))
    assert r.returncode == 0 and "ok: 0 failure(s)" in r.stdout and "AddressSanitizer" not in r.stderr, r.stdout + r.stderr


def test_dispatch_of_more_tokens_than_a_grid_holds():
    """A workgroup of 256 threads per token, fewer than 2^32 threads: up to 2^24 - 1 tokens."""
    for ty in ("fp8", "mxfp8"):
        for T, want in ((1 << 24, _lib.MOE_ERR_SHAPE), ((1 << 24) - 1, _lib.MOE_ERR_WORKSPACE)):
            s = shape(ty, T=T, d=128, f=128, k=1, C=T)
            assert L().moe_check_shape(s) == _lib.MOE_OK
            assert L().moe_dispatch_q(s, FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, None) == want
            if ty == "fp8":
                assert L().moe_dispatch(s, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, None) == want


def test_quantise_more_blocks_than_a_grid_holds():
    """A workgroup of 256 threads per block of 128 x 128, fewer than 2^32 threads; a short last block of rows counts whole."""
    q = L().moe_quantize_fp8
    assert q(FAKE, 1, 1 << 31, 128, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(FAKE, 129, 1 << 30, 128, FAKE, FAKE, None) == _lib.MOE_ERR_SHAPE
    assert q(FAKE, 1, (1 << 31) - 128, 128, ODD, FAKE, None) == _lib.MOE_ERR_ALIGN
    assert q(FAKE, 1, 1 << 31, 1, ODD, FAKE, None) == _lib.MOE_ERR_ALIGN       # rows: a bounded grid takes them in turn


def test_route_backward_asks_for_what_it_uses():
    """Up to 16 bf16 tokens nothing is kept (256 bytes are asked for all the same); one split of dW_r has no planes."""
    def need(dtype, T):
        return moe.workspace_bytes(shape(dtype, T=T, d=7168, E=512, k=8), moe.OP_ROUTE_BACKWARD)
    for ty in ("bf16", "fp8", "mxfp8"):
        assert [need(ty, T) for T in (1, 4, 5, 16)] == [256] * 4
        turned, plane = 7168 * 2 * 512 * 2, 512 * 7168 * 4      # W_r's parts; a plane of dW_r
        assert turned < need(ty, 17) < turned + (1 << 20) < turned + plane
        assert need(ty, 8192) >= turned + plane
    assert need("f32", 1) < 1 << 20 and need("f32", 0) == need("bf16", 0) == 0


def test_fp8_experts_refuse_misaligned_offsets():
    s = shape("fp8")
    assert L().moe_expert_ffn(s, FAKE, FAKE, FAKE + 2, 0, *([FAKE] * 7), None, FAKE, 1 << 30, None) == _lib.MOE_ERR_ALIGN
