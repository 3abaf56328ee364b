"""The C ABI of the clipping, AdamW and RMS norm entries on the CPU: structure
sizes and the refusals that the host makes before anything is launched."""

import ctypes as C
import os
import shutil
import subprocess

import pytest

import memory_reduced_muon_gb300 as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000   # never dereferenced
INV, UNS, SMALL = q.QMUON_ERR_INVALID_ARGUMENT, q.QMUON_ERR_UNSUPPORTED, q.QMUON_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q.LIB_PATH):
        from memory_reduced_muon_gb300 import build
        build.build()
    return q.lib()


_C_CALLER = r"""
#include <stddef.h>
#include "qmuon.h"
int main(void) {
  if (sizeof(qmuon_grad) != 24 || sizeof(qmuon_adamw_tensor) != 80 || sizeof(qmuon_rmsnorm) != 112 ||
      sizeof(qmuon_rmsnorm_grad) != 104)
    return 1;
  qmuon_clip_plan* c = (qmuon_clip_plan*)0x1;
  qmuon_adamw_plan* a = (qmuon_adamw_plan*)0x1;
  if (qmuon_clip_plan_create(NULL, 1, &c) != QMUON_ERR_INVALID_ARGUMENT || c != NULL) return 2;
  if (qmuon_adamw_plan_create(NULL, 1, QMUON_STATE_F32, &a) != QMUON_ERR_INVALID_ARGUMENT || a != NULL) return 3;
  qmuon_clip_plan_destroy(NULL);
  qmuon_adamw_plan_destroy(NULL);
  return 0;
}
"""


def test_header_compiles_as_c_and_sizes_agree(L, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text(_C_CALLER)
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                        "-o", str(exe), q.LIB_PATH, "-Wl,-rpath," + os.path.dirname(q.LIB_PATH)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0
    assert [C.sizeof(t) for t in (q.qmuon_grad, q.qmuon_adamw_tensor, q.qmuon_rmsnorm, q.qmuon_rmsnorm_grad)] == [24, 80, 112, 104]


def _clip(L, grads, n=None):
    arr = (q.qmuon_grad * max(1, len(grads)))(*grads)
    out = C.c_void_p(1)
    st = L.qmuon_clip_plan_create(arr, len(grads) if n is None else n, C.byref(out))
    assert out.value is None or st == q.QMUON_OK
    return st


def test_clip_refusals(L):
    assert _clip(L, []) == INV
    assert _clip(L, [q.qmuon_grad(FAKE, 8, 5, 0)]) == INV          # dtype
    assert _clip(L, [q.qmuon_grad(FAKE, -1, 0, 0)]) == INV
    assert _clip(L, [q.qmuon_grad(FAKE, (1 << 40) + 1, 0, 0)]) == INV
    assert _clip(L, [q.qmuon_grad(0, 8, 0, 0)]) == INV
    assert _clip(L, [q.qmuon_grad(FAKE + 1, 8, 0, 0)]) == INV      # not on a bf16 boundary
    assert _clip(L, [q.qmuon_grad(FAKE + 2, 8, 2, 0)]) == INV      # not on an fp32 boundary
    assert _clip(L, [q.qmuon_grad(0, 0, 0, 0)]) == INV             # no element at all
    assert L.qmuon_clip_plan_create((q.qmuon_grad * 1)(q.qmuon_grad(FAKE, 8, 0, 0)), 1, None) == INV
    assert L.qmuon_clip_workspace_size(None) == 0
    assert L.qmuon_grad_clip(None, 1.0, 0, FAKE, FAKE, 1 << 20, None) == INV


def _adamw(L, state=q.QMUON_STATE_F32, **kw):
    t = q.qmuon_adamw_tensor(FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 64, 1.0, 0.0, q.QMUON_BF16, q.QMUON_BF16)
    for k, v in kw.items():
        setattr(t, k, v)
    out = C.c_void_p(1)
    st = L.qmuon_adamw_plan_create((q.qmuon_adamw_tensor * 1)(t), 1, state, C.byref(out))
    assert out.value is None or st == q.QMUON_OK
    return st


def test_adamw_refusals(L):
    E = q.QMUON_STATE_E4M3
    assert _adamw(L, state=2) == INV
    for kw in (dict(numel=-1), dict(numel=(1 << 40) + 1), dict(numel=0), dict(param=0), dict(grad=0), dict(m=0), dict(v=0),
               dict(param=FAKE + 2), dict(grad=FAKE + 1), dict(m=FAKE + 2), dict(v=FAKE + 1), dict(grad_dtype=3),
               dict(copy=FAKE + 1), dict(copy=FAKE, copy_dtype=q.QMUON_FP32), dict(lr_scale=float("nan")),
               dict(weight_decay=float("inf"))):
        assert _adamw(L, **kw) == INV, kw
    for kw in (dict(m=FAKE + 4), dict(v=FAKE + 8), dict(m_absmax=0), dict(v_absmax=0), dict(m_absmax=FAKE + 2)):
        assert _adamw(L, state=E, **kw) == INV, kw
    assert L.qmuon_adamw_step(None, 1, 1e-3, 0.9, 0.99, 1e-8, None, None) == INV
    assert L.qmuon_adamw_step_sr(None, 1, 1e-3, 0.9, 0.99, 1e-8, 1, None, None) == INV


def _norm(**kw):
    n = q.qmuon_rmsnorm(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, 4, 64, 64, 64, 64, 64, 1e-5, q.QMUON_BF16)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def test_rmsnorm_forward_refusals(L):
    call = lambda **kw: L.qmuon_rmsnorm_forward(C.byref(_norm(**kw)), None)   # noqa: E731
    assert L.qmuon_rmsnorm_forward(None, None) == INV
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=(1 << 30) + 1), dict(rows=1 << 40), dict(dtype=3), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=0), dict(gain=0), dict(gain=FAKE + 2), dict(x=FAKE + 1), dict(ld_x=63),
               dict(ld_residual=63), dict(ld_sum=0), dict(ld_y=-64), dict(y=0), dict(payload=FAKE), dict(scale_inv=FAKE),
               dict(x=FAKE + 2, dtype=q.QMUON_FP32)):
        assert call(**kw) == INV, kw
    assert call(payload=FAKE, scale_inv=FAKE, cols=48) == UNS
    assert call(rows=0) == q.QMUON_OK      # nothing to do, nothing launched


def test_rmsnorm_backward_refusals(L):
    def call(ws=FAKE, ws_bytes=1 << 30, **kw):
        n = q.qmuon_rmsnorm_grad(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 64, 64, 64, 64, 1e-5, q.QMUON_BF16)
        for k, v in kw.items():
            setattr(n, k, v)
        return L.qmuon_rmsnorm_backward(C.byref(n), ws, ws_bytes, None)
    assert L.qmuon_rmsnorm_backward(None, FAKE, 1 << 20, None) == INV
    for kw in (dict(rows=-1), dict(cols=0), dict(dtype=-1), dict(eps=float("inf")), dict(dy=0), dict(h=0), dict(dx=0),
               dict(gain=0), dict(dgain=0), dict(dgain=FAKE + 1), dict(ld_dy=1), dict(ld_h=1), dict(ld_dsum=1), dict(ld_dx=1),
               dict(dsum=FAKE + 1), dict(ws=0), dict(ws=FAKE + 128)):
        assert call(**kw) == INV, kw
    assert q.qmuon_rmsnorm_workspace_size(-1, 64) == 0
    assert q.qmuon_rmsnorm_workspace_size(4, 0) == 0
    assert q.qmuon_rmsnorm_workspace_size(4, 64) >= 64 * 4
