"""Host-side refusals of the expert-grouped calls and of the 4-bit product: every
one is answered before a launch (no device call is made here), and the host
code runs under the sanitizers."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_moe_expert_02_amd", "csrc")
FAKE = ctypes.c_void_p(0x1000)                          # never dereferenced


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_02_amd import _lib
    _lib.lib()
    return _lib


def dims(L, **kw):
    v = dict(n_groups=4, rows=8, x_rows=8, n=32, k=64, src_div=1, type=L.T_BF16, out_type=L.T_BF16, ldx=64, ldy=128,
             ldw=64, w_stride=32 * 64, ld_pre=128)
    v.update(kw)
    return L.GroupDims(**v)


BAD_DIMS = [(dict(n_groups=0), "MOE_ESHAPE"), (dict(n_groups=1025), "MOE_ESHAPE"), (dict(rows=-1), "MOE_EINVAL"),
            (dict(x_rows=-1), "MOE_EINVAL"), (dict(n=0), "MOE_ESHAPE"), (dict(k=0), "MOE_ESHAPE"),
            (dict(src_div=0), "MOE_ESHAPE"), (dict(src_div=9), "MOE_ESHAPE"), (dict(type=0), "MOE_EFORMAT"),
            (dict(type=3), "MOE_EFORMAT"), (dict(out_type=7), "MOE_EFORMAT"), (dict(ldx=31), "MOE_ESHAPE"),
            (dict(ldy=15), "MOE_ESHAPE"), (dict(ldw=63), "MOE_ESHAPE"), (dict(w_stride=-1), "MOE_ESHAPE"),
            (dict(x_rows=7), "MOE_ESHAPE"), (dict(ldx=1 << 60), "MOE_ESHAPE"), (dict(n=1 << 29), "MOE_ESHAPE")]


def calls(L):
    lib = L.lib()
    return {"matmul": lambda d, x=FAKE, off=FAKE, w=FAKE, y=FAKE: lib.moe_group_matmul(d, x, None, off, w, y, None),
            "swiglu": lambda d, x=FAKE, off=FAKE, w=FAKE, y=FAKE: lib.moe_group_swiglu(d, x, None, off, w, y, FAKE, None),
            "matmul_t": lambda d, x=FAKE, off=FAKE, w=FAKE, y=FAKE: lib.moe_group_matmul_t(d, x, None, off, w, y, None),
            "swiglu_grad": lambda d, x=FAKE, off=FAKE, w=FAKE, y=FAKE: lib.moe_group_swiglu_grad(d, x, None, off, w, FAKE,
                                                                                                   y, None),
            "wgrad": lambda d, x=FAKE, off=FAKE, w=FAKE, y=FAKE: lib.moe_group_wgrad(d, w, x, None, off, y, 0, None)}


@pytest.mark.parametrize("call", ["matmul", "swiglu", "matmul_t", "swiglu_grad", "wgrad"])
def test_grouped_products_refuse(L, call):
    f = calls(L)[call]
    for change, status in BAD_DIMS:
        assert f(ctypes.byref(dims(L, **change))) == getattr(L, status), (call, change)
    good = dims(L)
    assert f(None) == L.MOE_EINVAL
    for missing in ("x", "off", "w", "y"):
        assert f(ctypes.byref(good), **{missing: None}) == L.MOE_EINVAL, missing
    if call != "wgrad":                                  # no rows: nothing to do (wgrad writes zeros)
        assert f(ctypes.byref(dims(L, rows=0, x_rows=0))) == L.MOE_OK


def test_grouped_products_refuse_their_own(L):
    f = calls(L)
    assert f["swiglu"](ctypes.byref(dims(L, n=31, ldy=128))) == L.MOE_ESHAPE
    assert f["swiglu"](ctypes.byref(dims(L, ld_pre=31))) == L.MOE_ESHAPE
    assert f["swiglu_grad"](ctypes.byref(dims(L, ld_pre=127))) == L.MOE_ESHAPE
    assert f["swiglu_grad"](ctypes.byref(dims(L, ldy=127))) == L.MOE_ESHAPE
    assert f["wgrad"](ctypes.byref(dims(L, w_stride=32 * 64 - 1))) == L.MOE_ESHAPE
    assert L.lib().moe_group_swiglu_grad(ctypes.byref(dims(L)), FAKE, None, FAKE, FAKE, None, FAKE, None) == L.MOE_EINVAL


def test_plan_refuses(L):
    lib = L.lib()

    def plan(rows=4, top_k=2, groups=8, idx=FAKE, off=FAKE, pairs=FAKE, pos=FAKE, ws=None, n=0):
        return lib.moe_group_plan(idx, rows, top_k, groups, off, pairs, pos, ws, n, None)

    assert plan(rows=-1) == L.MOE_EINVAL
    for kw in (dict(top_k=0), dict(top_k=9), dict(groups=0), dict(groups=1025), dict(rows=2**30, top_k=2)):
        assert plan(**kw) == L.MOE_ESHAPE, kw
    for name in ("idx", "off", "pairs", "pos"):
        assert plan(**{name: None}) == L.MOE_EINVAL, name
    need = L.group_plan_bytes(4096, 2, 8)
    assert need > 0 and L.group_plan_bytes(1024, 2, 8) == 0 and L.group_plan_bytes(-1, 2, 8) == 0
    assert plan(rows=4096, n=need) == L.MOE_EINVAL
    assert plan(rows=4096, ws=FAKE, n=need - 1) == L.MOE_EWORKSPACE
    assert plan(rows=4096, ws=ctypes.c_void_p(0x1002), n=need) == L.MOE_EINVAL


def test_combine_refuses(L):
    lib = L.lib()

    def cd(**kw):
        v = dict(rows=4, top_k=2, n=16, o_rows=8, type=L.T_BF16, out_type=L.T_F32, ldo=16, ldy=16)
        v.update(kw)
        return ctypes.byref(L.CombineDims(**v))

    def fwd(d, o=FAKE, pos=FAKE, y=FAKE):
        return lib.moe_group_combine(d, o, pos, None, y, None)

    def back(d, dy=FAKE, o=FAKE, pos=FAKE, d_o=FAKE, d_w=FAKE):
        return lib.moe_group_combine_grad(d, dy, o, pos, None, d_o, d_w, None)

    for f in (fwd, back):
        for change, status in ((dict(rows=-1), L.MOE_EINVAL), (dict(o_rows=-1), L.MOE_EINVAL), (dict(type=5), L.MOE_EFORMAT),
                               (dict(out_type=-1), L.MOE_EFORMAT), (dict(n=0), L.MOE_ESHAPE), (dict(top_k=0), L.MOE_ESHAPE),
                               (dict(top_k=9), L.MOE_ESHAPE), (dict(ldo=15), L.MOE_ESHAPE), (dict(ldy=15), L.MOE_ESHAPE),
                               (dict(rows=2**30, top_k=4), L.MOE_ESHAPE)):
            assert f(cd(**change)) == status, change
        assert f(None) == L.MOE_EINVAL
        assert f(cd(rows=0)) == L.MOE_OK
        assert f(cd(o_rows=7), pos=None) == L.MOE_ESHAPE
        assert f(cd(), o=None) == L.MOE_EINVAL
    assert fwd(cd(), y=None) == L.MOE_EINVAL
    assert back(cd(), dy=None) == L.MOE_EINVAL
    assert back(cd(), d_o=None, d_w=None) == L.MOE_OK


def test_q4_refuses(L):
    lib = L.lib()

    def qd(**kw):
        v = dict(n=64, k=128, group=32, n_mats=1, rows=2, x_div=1, type=L.T_F16, out_type=L.T_F32, swiglu=0, ldx=128, ldy=64)
        v.update(kw)
        return ctypes.byref(L.Q4Dims(**v))

    def call(d, x=FAKE, c=FAKE, s=FAKE, z=None, y=FAKE):
        return lib.moe_q4_matvec(d, x, None, c, s, z, y, None)

    for change, status in ((dict(rows=-1), L.MOE_EINVAL), (dict(rows=65), L.MOE_ESHAPE), (dict(group=16), L.MOE_ESHAPE),
                           (dict(group=48), L.MOE_ESHAPE), (dict(k=100, ldx=100), L.MOE_ESHAPE), (dict(n=0), L.MOE_ESHAPE),
                           (dict(k=0), L.MOE_ESHAPE), (dict(n_mats=0), L.MOE_ESHAPE), (dict(x_div=0), L.MOE_ESHAPE),
                           (dict(type=0), L.MOE_EFORMAT), (dict(out_type=3), L.MOE_EFORMAT), (dict(swiglu=2), L.MOE_EINVAL),
                           (dict(swiglu=1, n=48), L.MOE_ESHAPE), (dict(ldx=127), L.MOE_ESHAPE), (dict(ldy=63), L.MOE_ESHAPE)):
        assert call(qd(**change)) == status, change
    assert call(None) == L.MOE_EINVAL and call(qd(rows=0)) == L.MOE_OK
    for missing in ("x", "c", "s", "y"):
        assert call(qd(), **{missing: None}) == L.MOE_EINVAL, missing
    odd = ctypes.c_void_p(0x1008)
    for name in ("c", "s", "z"):
        assert call(qd(), **{name: odd}) == L.MOE_EINVAL, name
    with pytest.raises(L.MoeError):
        L.q4_bytes(4, 100, 32)
    w = np.zeros((4, 96), np.float32)
    with pytest.raises(L.MoeError):
        L.q4_pack(w, 64)
    assert lib.moe_q4_pack(None, 4, 96, 32, FAKE, FAKE, None, 1) == L.MOE_EINVAL
    assert lib.moe_q4_unpack(FAKE, None, None, 4, 96, 32, FAKE, 1) == L.MOE_EINVAL
    codes, scales, _ = L.q4_pack(w, 32)
    with pytest.raises(L.MoeError):
        L.q4_unpack(codes[:-1], scales, None, 4, 96, 32)


def test_binding_refuses_host_tensors(L):
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    off, y = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8)
    with pytest.raises(L.MoeError) as e:
        L.moe_group_matmul(x, off, w, y)
    assert e.value.status == L.MOE_EINVAL
    with pytest.raises(L.MoeError):
        L.moe_q4_matvec(x, w, w, None, 32, y)
    with pytest.raises(L.MoeError):
        L.moe_group_combine(x, None, None, y)


HOST_CHECK = r"""
#include <cmath>
#include <cstdio>
#include <vector>
#include "moe.h"
int main() {
  for (int group : {32, 64, 128})
    for (int64_t n : {1, 15, 16, 17, 40})
      for (int64_t k : {1, 2, 3, 5})
        for (int zeros : {0, 1}) {
          const int64_t kk = k * group;
          size_t c, s, z;
          if (moe_q4_bytes(n, kk, group, &c, &s, &z)) return 1;
          std::vector<unsigned char> cb(c), sb(s), zb(z);
          std::vector<float> w(n * kk), v(n * kk);
          for (size_t i = 0; i < w.size(); ++i) w[i] = std::sin(0.37f * i) * (i % 97 == 0 ? 1e6f : 0.02f);
          w[0] = NAN;
          if (moe_q4_pack(w.data(), n, kk, group, cb.data(), sb.data(), zeros ? zb.data() : nullptr, 3)) return 2;
          if (moe_q4_unpack(cb.data(), sb.data(), zeros ? zb.data() : nullptr, n, kk, group, v.data(), 2)) return 3;
        }
  if (moe_group_plan_bytes(4096, 6, 384) != 4u * 384 * 13) return 4;
  std::puts("group host checks ok");
  return 0;
}
"""


def test_host_code_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(HOST_CHECK)
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), str(src),
           os.path.join(CSRC, "group_host.cpp"), os.path.join(CSRC, "pack.cpp"), "-pthread", "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stdout + build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0"))
    assert run.returncode == 0 and "ok" in run.stdout, run.stdout + run.stderr
