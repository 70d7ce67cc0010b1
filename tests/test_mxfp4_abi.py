"""Refusals of the MXFP4 calls: statuses from the host's checks before any launch (no GPU), the binding's checks of
tensors, and the same host code under AddressSanitizer."""
import os
import subprocess

import pytest
import torch

import mixture_experts_layer_33_amd as moe
from mixture_experts_layer_33_amd import _lib
from mixture_experts_layer_33_amd import build as libbuild

FAKE, ODD = 0x1000, 0x1008
L = _lib.lib
NULL, SHAPE, WORKSPACE, DTYPE, ALIGN, OK = (_lib.MOE_ERR_NULL, _lib.MOE_ERR_SHAPE, _lib.MOE_ERR_WORKSPACE, _lib.MOE_ERR_DTYPE,
                                            _lib.MOE_ERR_ALIGN, _lib.MOE_OK)


def shape(dtype="mxfp4", T=4, d=256, E=8, k=2, f=128, fs=0, C=None):
    return moe.make_shape(T, d, E, k, f, C, fs, dtype)


def test_shapes():
    assert L().moe_check_shape(shape()) == OK
    for bad in (dict(d=192), dict(f=64), dict(d=0), dict(k=9), dict(E=1025), dict(d=1 << 20, f=4096)):
        assert L().moe_check_shape(shape(**bad)) == SHAPE, bad
    for dt in (-1, 5, 99):
        s = shape()
        s.dtype = dt
        assert L().moe_check_shape(s) == DTYPE


def test_quantiser_refusals():
    q = L().moe_quantize_mxfp4
    assert q(FAKE, 4, 96, FAKE, FAKE, None) == SHAPE and q(FAKE, -1, 128, FAKE, FAKE, None) == SHAPE
    assert q(FAKE, 1 << 31, 128, FAKE, FAKE, None) == SHAPE and q(FAKE, 4, 0, FAKE, FAKE, None) == SHAPE
    for a in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert q(a[0], 4, 128, a[1], a[2], None) == NULL
    for a in ((ODD, FAKE, FAKE), (FAKE, ODD, FAKE), (FAKE, FAKE, FAKE + 2)):
        assert q(a[0], 4, 128, a[1], a[2], None) == ALIGN
    assert q(None, 0, 128, None, None, None) == OK


def test_matmul_refusals():
    def mm(M=16, N=256, K=256, ty=_lib.MOE_BF16, x=FAKE, w=FAKE, s=FAKE, out=FAKE, ws=FAKE, n=1 << 40):
        return L().moe_matmul_mxfp4(x, w, s, M, N, K, ty, out, ws, n, None)
    for bad in (dict(K=192), dict(K=0), dict(M=-1), dict(N=-1), dict(M=1 << 25), dict(N=1 << 25), dict(M=1 << 31), dict(M=1 << 22, N=1 << 22, K=128), dict(M=1, N=1, K=1 << 23)):
        assert mm(**bad) == SHAPE, bad
    assert mm(ty=_lib.MOE_MXFP4) == DTYPE
    for bad in (dict(x=None), dict(w=None), dict(s=None), dict(out=None)):
        assert mm(**bad) == NULL, bad
    for bad in (dict(x=ODD), dict(w=ODD), dict(s=FAKE + 2), dict(out=FAKE + 1), dict(out=FAKE + 2, ty=_lib.MOE_F32), dict(ws=ODD)):
        assert mm(**bad) == ALIGN, bad
    assert mm(M=0, x=None, out=None) == OK and mm(N=0, w=None, out=None) == OK
    for M, N, K in ((1, 7168, 2048), (16, 256, 256), (100, 256, 8192), (4096, 4096, 4096)):
        need = L().moe_matmul_mxfp4_workspace_bytes(M, N, K)
        assert need % 256 == 0
        if need:
            assert mm(M, N, K, n=need - 1) == WORKSPACE and mm(M, N, K, ws=None, n=0) == NULL
    assert L().moe_matmul_mxfp4_workspace_bytes(16, 256, 100) == 0


RULE = _lib.MoeRouter(1, 4, 2, 2, 1, 2.5)
NAMES = ("x", "w_r", "b_r", "balance", "wg", "wu", "wd", "sg", "su", "sd", "hg", "hu", "hd", "tg", "tu", "td", "y", "idx", "gate", "ws")


def decode(s, rule=RULE, n=1 << 40, **over):
    return L().moe_decode_mxfp4(s, rule, *(over.get(a, FAKE) for a in NAMES), n, None)


def test_decode_refusals():
    s = shape(fs=128)
    for ty in ("bf16", "mxfp8", "fp8", "f32"):
        assert decode(shape(ty)) == DTYPE
    assert decode(None) == NULL and decode(s, None) == NULL
    assert decode(s, _lib.MoeRouter(2, 4, 2, 2, 1, 2.5)) == SHAPE
    for bad in (dict(T=0), dict(T=17), dict(k=17, E=64), dict(d=8320), dict(f=65664), dict(fs=64), dict(fs=65664), dict(fs=-128),
                dict(E=512, f=16384, d=8192), dict(E=1024, k=4, f=8192, d=8192)):      # scale bytes of 2 GiB
        assert decode(shape(**bad)) == SHAPE, bad
        assert moe.workspace_bytes(shape(**bad), moe.OP_DECODE) == 0
    for a in NAMES:
        want = OK if a in ("b_r", "balance") else NULL
        if want == NULL:
            assert decode(s, **{a: None}) == NULL, a
        odd = {"y": FAKE + 1}.get(a, FAKE + 2 if a in ("b_r", "balance", "sg", "su", "sd", "tg", "tu", "td", "idx", "gate") else ODD)
        assert decode(s, **{a: odd}) == ALIGN, a
    need = moe.workspace_bytes(s, moe.OP_DECODE)
    assert need % 256 == 0 and decode(s, n=need - 1) == WORKSPACE


def test_experts_and_dispatch_refusals():
    s = shape()
    ffn = [s, FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE]
    for i in (1, 2, 3, 5, 6, 7, 8, 9, 10, 11, 13):
        a = list(ffn)
        a[i] = None
        assert L().moe_expert_ffn(*a, 1 << 30, None) == NULL, i
    for i in (1, 5, 6, 7, 11, 13):
        a = list(ffn)
        a[i] = ODD
        assert L().moe_expert_ffn(*a, 1 << 30, None) == ALIGN, i
    for i in (2, 3, 8, 9, 10):
        a = list(ffn)
        a[i] = FAKE + 2
        assert L().moe_expert_ffn(*a, 1 << 30, None) == ALIGN, i
    a = list(ffn)
    a[12] = FAKE                                  # saved A|U: no backward
    assert L().moe_expert_ffn(*a, 1 << 30, None) == DTYPE
    assert L().moe_expert_ffn(*ffn, moe.workspace_bytes(s, moe.OP_EXPERT_FFN) - 1, None) == WORKSPACE
    a = list(ffn)
    a[4] = s.capacity
    assert L().moe_expert_ffn(*a, 1 << 30, None) == SHAPE
    assert L().moe_dispatch(s, FAKE, FAKE, 0, FAKE, None, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == NULL
    for x, ring, scale in ((ODD, FAKE, FAKE), (FAKE, ODD, FAKE), (FAKE, FAKE, FAKE + 2)):
        assert L().moe_dispatch(s, x, FAKE, 0, ring, scale, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == ALIGN
        assert L().moe_dispatch_q(s, x, FAKE, FAKE, 0, ring, scale, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == ALIGN
    big = shape(T=1 << 24, d=128, f=128, k=1, C=1 << 24)
    assert L().moe_dispatch(big, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, None) == SHAPE


def test_what_has_no_mxfp4_form_says_so():
    s = shape()
    assert L().moe_forward(s, *([FAKE] * 6), 0, *([FAKE] * 10), 0, FAKE, 1 << 40, None) == DTYPE
    assert L().moe_decode(s, *([FAKE] * 13), 1 << 40, None) == DTYPE
    assert L().moe_backward(s, *([FAKE] * 9), 0, *([FAKE] * 10), 1 << 40, None) == DTYPE
    assert L().moe_backward_mx(s, *([FAKE] * 8), 0, *([FAKE] * 11), 1 << 40, None) == DTYPE
    assert L().moe_backward_experts(s, *([FAKE] * 7), 0, *([FAKE] * 10), 1 << 40, None) == DTYPE
    assert moe.workspace_bytes(s, moe.OP_BACKWARD) == 0 and moe.workspace_bytes(s, moe.OP_FORWARD) == 0


def test_binding_refuses_host_tensors_and_wrong_ones():
    bf, u8 = torch.bfloat16, torch.uint8
    x, w, s, out = torch.zeros(4, 256, dtype=bf), torch.zeros(32, 128, dtype=u8), torch.zeros(2, 32, 4, dtype=u8), torch.zeros(4, 32)
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_matmul_mxfp4(x, w, s, out)
    for bad, match in (((x.float(), w, s, out), "x"), ((x, w[:, :64].contiguous(), s, out), "w: "), ((x, w, s[:1].contiguous(), out), "w_scale"),
                       ((x, w, s.view(2, 128), out), "w_scale"), ((x, w, s, out.half()), "bfloat16 or float32"), ((x, w, s, out.t()), "out"),
                       ((x[0], w, s, out), "matrix")):
        with pytest.raises(ValueError, match=match):
            moe.moe_matmul_mxfp4(*bad)
    with pytest.raises(ValueError, match="matrices"):
        moe.quantize_mxfp4(x[0])
    sh = shape(fs=128)
    z = torch.zeros
    wide, tall = z(2, 1024, 4, dtype=u8), z(1, 2048, 4, dtype=u8)
    good = [sh, moe.make_router(), x, z(8, 256), None, None, z(8, 128, 128, dtype=u8), z(8, 128, 128, dtype=u8), z(8, 256, 64, dtype=u8), wide, wide, tall,
            z(128, 128, dtype=u8), z(128, 128, dtype=u8), z(256, 64, dtype=u8), z(2, 128, 4, dtype=u8), z(2, 128, 4, dtype=u8), z(1, 256, 4, dtype=u8),
            z(4, 256, dtype=bf), z(4, 2, dtype=torch.int32), z(4, 2), z(1 << 16, dtype=u8)]
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_decode_mxfp4(*good)
    for i in [2, 3] + list(range(6, 21)):
        bad = list(good)
        bad[i] = good[i][..., :-1].contiguous()
        with pytest.raises(ValueError, match="needs"):
            moe.moe_decode_mxfp4(*bad)
    layer = moe.Layer.create(4, 256, 8, 2, 128, dtype="bf16", device="cpu")
    with pytest.raises(ValueError, match="MXFP4"):
        layer.decode(x, None, None, None, None, None, router=moe.make_router())
    with pytest.raises(ValueError, match="MXFP4"):
        layer.decode(x, None, None, None, None, None, scales=(wide, wide, tall))


DRIVER = r"""
#include <cstdio>
#include "moe.h"
static int bad = 0;
static void want(const char* n, long g, long w) { if (g != w) { std::printf("FAIL %s %ld %ld\n", n, g, w); ++bad; } }
int main() {
  unsigned char* b = new unsigned char[64];
  b = (unsigned char*)(((uintptr_t)b + 15) & ~(uintptr_t)15);
  float* F = (float*)b; int32_t* I = (int32_t*)b;
  moe_shape* s = new moe_shape{4, 10, 256, 8, 2, 128, 128, MOE_MXFP4};
  moe_shape* l = new moe_shape{17, 40, 256, 8, 2, 128, 0, MOE_MXFP4};
  moe_router* r = new moe_router{MOE_SCORE_SIGMOID, 4, 2, 2, 1, 2.5f};
  want("shape", moe_check_shape(s), MOE_OK);
  for (int op = 0; op <= MOE_OP_ROUTE_BACKWARD; ++op) { want("ws", moe_workspace_bytes(s, op) % 256, 0); moe_workspace_bytes(l, op); }
  auto decode = [&](moe_shape* q, moe_router* u, size_t n) {
    return moe_decode_mxfp4(q, u, b, F, F, F, b, b, b, b, b, b, b, b, b, b, b, b, b, I, F, b, n, nullptr);
  };
  want("decode", decode(s, r, 0), MOE_ERR_WORKSPACE);
  want("decode rule", decode(s, nullptr, 0), MOE_ERR_NULL);
  want("decode tokens", decode(l, r, 1 << 30), MOE_ERR_SHAPE);
  want("quantise", moe_quantize_mxfp4(b, 4, 64, b, b, nullptr), MOE_ERR_SHAPE);
  want("matmul", moe_matmul_mxfp4(b, b, b, 4, 4, 100, MOE_BF16, b, b, 0, nullptr), MOE_ERR_SHAPE);
  want("matmul ws", moe_matmul_mxfp4_workspace_bytes(100, 1000, 8192) % 256, 0);
  want("experts", moe_expert_ffn(s, b, b, I, 0, b, b, b, b, b, b, b, nullptr, b, 0, nullptr), MOE_ERR_WORKSPACE);
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
