"""Host-side checks of the 8-bit head and of sampling (no GPU): argument
errors come back before any device work, workspace sizes, struct layouts as a
C client sees them, the host layer under sanitizers, and pins of the oracle
against exact rational arithmetic and worked examples."""

import ctypes
import math
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

import output_projection_kl_amd as fkl
from oracle import decode_oracle as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EWORKSPACE, EUNSUPPORTED = 1, 2, 5
vp, sz = ctypes.c_void_p, ctypes.c_size_t


def _quantize(rows=4, cols=64, type=1, x=4096, ldx=64, q=8192, ldq=64, scale=256):
    return fkl.lib().fkl_quantize(rows, cols, type, vp(x), ldx, vp(q), ldq, vp(scale), vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL), (dict(type=3), EINVAL), (dict(type=9), EINVAL),
    (dict(ldx=63), EINVAL), (dict(ldq=63), EINVAL), (dict(x=0), EINVAL), (dict(q=0), EINVAL), (dict(scale=0), EINVAL),
    (dict(x=4097), EINVAL), (dict(type=0, x=4098), EINVAL), (dict(scale=2), EINVAL),
    (dict(rows=1 << 31), EUNSUPPORTED), (dict(cols=1 << 31, ldx=1 << 31, ldq=1 << 31), EUNSUPPORTED),
    (dict(ldx=1 << 41), EUNSUPPORTED), (dict(rows=0), 0),
])
def test_quantize_argument_errors(kw, status):
    assert _quantize(**kw) == status
    assert status == 0 or fkl.lib().fkl_last_error()


def _project(M=4, N=64, K=64, lda=64, ldb=64, ldo=64, a_type=3, out_type=1, flags=0, a=4096, sa=256, b=8192, sb=256,
             bias=0, out=512, ws=1 << 20, ws_bytes=1 << 30):
    s = fkl.ProjectShape(M, N, K, lda, ldb, ldo, a_type, out_type, flags)
    return fkl.lib().fkl_project(ctypes.byref(s), vp(a), vp(sa), vp(b), vp(sb), vp(bias), vp(out), vp(ws), sz(ws_bytes),
                                 vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(lda=63), EINVAL), (dict(ldb=63), EINVAL),
    (dict(ldo=63), EINVAL), (dict(a_type=7), EINVAL), (dict(out_type=3), EINVAL), (dict(flags=4), EINVAL),
    (dict(a=0), EINVAL), (dict(b=0), EINVAL), (dict(sb=0), EINVAL), (dict(out=0), EINVAL), (dict(sa=0), EINVAL),
    (dict(a_type=1), EINVAL),  # floating rows come without a_scale
    (dict(a=4100), EINVAL), (dict(b=8200), EINVAL), (dict(out=513), EINVAL), (dict(out_type=0, out=514), EINVAL),
    (dict(sb=258), EINVAL), (dict(bias=257), EINVAL),
    (dict(K=131072, lda=131072, ldb=131072), EUNSUPPORTED), (dict(N=1 << 31, ldo=1 << 31), EUNSUPPORTED),
    (dict(M=1 << 20, N=1 << 21, ldo=1 << 21), EUNSUPPORTED), (dict(ldb=1 << 41), EUNSUPPORTED),
    # a copied operand and quantised rows need room
    (dict(ldb=72, ws=0), EWORKSPACE), (dict(ldb=72, ws=(1 << 20) + 16), EWORKSPACE), (dict(ldb=72, ws_bytes=4095), EWORKSPACE),
    (dict(a_type=1, sa=0, ws=0), EWORKSPACE), (dict(a_type=1, sa=0, ws_bytes=255), EWORKSPACE),
    (dict(M=0), 0),
])
def test_project_argument_errors(kw, status):
    assert _project(**kw) == status
    assert status == 0 or fkl.lib().fkl_last_error()


def _sample(N=4, V=100, ld=100, ld_ids=0, type=0, T=1.0, k=0, p=1.0, q=0.0, T_rows=0, k_rows=0, p_rows=0, q_rows=0,
            logits=4096, ids=0, u=256, token=512, logprob=0, ws=1 << 20, ws_bytes=1 << 30, params=True):
    s = fkl.SampleShape(N, V, ld, ld_ids, type)
    pr = fkl.SampleParams(T_rows, k_rows, p_rows, q_rows, T, k, p, q)
    return fkl.lib().fkl_sample(ctypes.byref(s), ctypes.byref(pr) if params else None, vp(logits), vp(ids), vp(u),
                                vp(token), vp(logprob), vp(ws), sz(ws_bytes), vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), EINVAL), (dict(V=0), EINVAL), (dict(ld=99), EINVAL), (dict(type=3), EINVAL), (dict(ld_ids=-1), EINVAL),
    (dict(T=-0.5), EINVAL), (dict(T=math.nan), EINVAL), (dict(T=math.inf), EINVAL), (dict(p=math.nan), EINVAL),
    (dict(q=math.nan), EINVAL), (dict(params=False), EINVAL), (dict(T_rows=2), EINVAL), (dict(k_rows=3), EINVAL),
    (dict(logits=0), EINVAL), (dict(u=0), EINVAL), (dict(token=0), EINVAL), (dict(logits=4098), EINVAL),
    (dict(type=1, logits=4097), EINVAL), (dict(ids=1024, ld_ids=99), EINVAL), (dict(ids=1026, ld_ids=100), EINVAL),
    (dict(logprob=3), EINVAL), (dict(V=1 << 31, ld=1 << 31), EUNSUPPORTED), (dict(ld=1 << 41), EUNSUPPORTED),
    (dict(V=5000, ld=5000, ws=0), EWORKSPACE), (dict(V=5000, ld=5000, ws=(1 << 20) + 128), EWORKSPACE),
    (dict(V=5000, ld=5000, ws_bytes=100), EWORKSPACE), (dict(N=0), 0),
])
def test_sample_argument_errors(kw, status):
    assert _sample(**kw) == status
    assert status == 0 or fkl.lib().fkl_last_error()


def test_workspace_sizes_hold_what_they_are_for():
    row = 2896  # 2887 bytes rounded up to 16
    base = fkl.project_workspace_size(10, 100, 2887, lda=row, ldb=row)
    assert base < 100 * row
    assert fkl.project_workspace_size(10, 100, 2887, lda=row) >= base + 100 * row
    assert fkl.project_workspace_size(10, 100, 2887, lda=row, ldb=row, flags=fkl.PROJECT_COPY_A) >= base + 10 * row
    assert fkl.project_workspace_size(10, 100, 2887, torch.bfloat16, ldb=row) >= base + 10 * row + 40
    # nothing to hold: the workspace may be NULL
    if "debug" not in os.path.basename(fkl.library_path()):
        assert fkl.project_workspace_size(5, 1024, 1024) == 0 and fkl.sample_workspace_size(10, 1024) == 0
    for N, V in ((3, 5000), (512, 201088), (64, 128256), (1, 262136), (2, 1048568)):
        assert 0 < fkl.sample_workspace_size(N, V) <= N * (V // 4096 + 2) * 5200 + 4096


def test_binding_refuses_what_is_not_a_gpu_matrix():
    x = torch.zeros((2, 64))
    for call in (lambda: fkl.quantize(x), lambda: fkl.project(x, x, x[0]), lambda: fkl.sample(x, x[:, 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        fkl.quantize([[1.0]])


_C_CLIENT = r"""
#include <stddef.h>
#include <stdio.h>
#include "fkl.h"
#define F(T, f) printf(" %s=%zu", #f, offsetof(T, f))
int main(void) {
  printf("ProjectShape %zu", sizeof(fkl_project_shape));
  F(fkl_project_shape, M); F(fkl_project_shape, N); F(fkl_project_shape, K); F(fkl_project_shape, lda);
  F(fkl_project_shape, ldb); F(fkl_project_shape, ldo); F(fkl_project_shape, a_type);
  F(fkl_project_shape, out_type); F(fkl_project_shape, flags);
  printf("\nSampleShape %zu", sizeof(fkl_sample_shape));
  F(fkl_sample_shape, N); F(fkl_sample_shape, V); F(fkl_sample_shape, ld); F(fkl_sample_shape, ld_ids);
  F(fkl_sample_shape, type);
  printf("\nSampleParams %zu", sizeof(fkl_sample_params));
  F(fkl_sample_params, temperature_rows); F(fkl_sample_params, top_k_rows); F(fkl_sample_params, top_p_rows);
  F(fkl_sample_params, min_p_rows); F(fkl_sample_params, temperature); F(fkl_sample_params, top_k);
  F(fkl_sample_params, top_p); F(fkl_sample_params, min_p);
  printf("\ntypes %d %d %d %d", FKL_F32, FKL_BF16, FKL_F16, FKL_I8);
  printf("\nrefused %d %d\n", (int)fkl_quantize(1, 0, FKL_F32, NULL, 1, NULL, 1, NULL, NULL),
         (int)fkl_sample(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL));
  return 0;
}
"""


def test_c_client_sees_the_bindings_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None or not os.path.exists(fkl.library_path()):
        pytest.skip("needs a C compiler and the built library")
    src, exe, lib = tmp_path / "client.c", tmp_path / "client", os.path.abspath(fkl.library_path())
    src.write_text(_C_CLIENT)
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe), lib, f"-Wl,-rpath,{os.path.dirname(lib)}"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout
    lines = {ln.split()[0]: ln.split()[1:] for ln in out.splitlines()}
    for name in ("ProjectShape", "SampleShape", "SampleParams"):
        t = getattr(fkl, name)
        want = [str(ctypes.sizeof(t))] + [f"{f}={getattr(t, f).offset}" for f, _ in t._fields_]
        assert lines[name] == want
    assert lines["types"] == ["0", "1", "2", "3"] and lines["refused"] == ["1", "1"]


def test_host_layer_under_sanitizers(tmp_path):
    """csrc/fkl_decode_api.cpp with g++ under AddressSanitizer and
    UndefinedBehaviorSanitizer; stub launchers check the plans they are handed."""
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = tmp_path / "decode_plan_check"
    csrc = os.path.join(ROOT, "output_projection_kl_amd", "csrc")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(ROOT, "tests", "host_sanitize", "decode_plan_check.cpp"),
           os.path.join(csrc, "fkl_decode_api.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "failures 0" in r.stdout, (r.stdout + r.stderr)[-4000:]


def _nearest(x):
    """Fraction -> nearest integer, ties to even."""
    f = x.numerator // x.denominator
    d = x - f
    return f + (d > Fraction(1, 2) or (d == Fraction(1, 2) and f % 2 != 0))


def test_oracle_levels_are_those_of_rational_arithmetic():
    rng = np.random.default_rng(0)
    rows = [rng.standard_normal(200).astype(np.float32), (rng.integers(-254, 255, 200) / 2).astype(np.float32),
            rng.standard_normal(200).astype(np.float16).astype(np.float32)]
    rows[1][0] = 127.0
    for x in rows:
        q, s = oracle.quantize(x[None])
        a = max(abs(Fraction(float(v))) for v in x)
        assert [int(v) for v in q[0]] == [_nearest(127 * Fraction(float(v)) / a) for v in x]
        assert s[0] == np.float32(float(a)) / np.float32(127)


def test_oracle_draws_of_worked_examples():
    x = np.log(np.array([[0.1, 0.4, 0.2, 0.3]]))
    at = lambda u, **kw: oracle.sample(x, [u], **kw)[0][0]  # noqa: E731
    assert [at(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [at(u, k=2) for u in (0.0, 0.57, 0.58)] == [1, 1, 3]            # 0.4 and 0.3 remain
    assert [at(u, p=0.65) for u in (0.0, 0.57, 0.58, 0.99)] == [1, 1, 3, 3]  # 0.4 + 0.3 >= 0.65
    assert [at(u, p=0.75) for u in (0.0, 0.45, 0.6, 0.99)] == [1, 2, 2, 3]   # 0.2 joins in its position
    assert [at(u, q=0.6) for u in (0.0, 0.57, 0.58)] == [1, 1, 3]          # at least 0.6 * 0.4
    assert at(0.999, T=0.0) == 1
    assert abs(oracle.sample(x, [0.0], k=2)[1][0] - math.log(4 / 7)) < 1e-7
    tie = np.zeros((1, 4))
    assert [oracle.sample(tie, [u], k=2)[0][0] for u in (0.0, 0.49, 0.51, 0.99)] == [0, 0, 1, 1]
    none = np.full((1, 3), -np.inf)
    assert oracle.sample(none, [0.5])[0][0] == -1 and np.isneginf(oracle.sample(none, [0.5])[1][0])
