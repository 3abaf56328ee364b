"""The C ABI of the embedding, checkpoint and feed-forward entries on the CPU:
structure sizes and the refusals that the host makes before anything is
launched."""

import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

import memory_reduced_muon_gb300 as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000   # never dereferenced
INV, UNS = q.QMUON_ERR_INVALID_ARGUMENT, q.QMUON_ERR_UNSUPPORTED


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
  if (sizeof(qmuon_embedding) != 80 || sizeof(qmuon_embedding_grad) != 88 || sizeof(qmuon_mxfp8) != 56 ||
      sizeof(qmuon_gated_ffn) != 152 || sizeof(qmuon_gated_ffn_grad) != 232)
    return 1;
  if (qmuon_embedding_forward(NULL, NULL) != QMUON_ERR_INVALID_ARGUMENT) return 2;
  if (qmuon_gated_ffn_workspace_size(NULL) != 0 || qmuon_gated_ffn_backward_workspace_size(NULL) != 0) return 3;
  if (qmuon_embedding_workspace_size(1, 0, 1) != 0) return 4;
  return QMUON_ACT_GELU_TANH == 2 && QMUON_SAVE_MXFP8 == 2 ? 0 : 5;
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
    assert [C.sizeof(t) for t in (q.qmuon_embedding, q.qmuon_embedding_grad, q.qmuon_mxfp8, q.qmuon_gated_ffn,
                                  q.qmuon_gated_ffn_grad)] == [80, 88, 56, 152, 232]


def _with(struct, kw):
    for k, v in kw.items():
        setattr(struct, k, v)
    return struct


def test_embedding_forward_refusals(L):
    call = lambda **kw: L.qmuon_embedding_forward(   # noqa: E731
        C.byref(_with(q.qmuon_embedding(FAKE, FAKE, FAKE, 4, 16, 64, 64, 64, 1.0, q.QMUON_BF16, 64, 0), kw)), None)
    for kw in (dict(n_tokens=-1), dict(n_tokens=(1 << 28) + 1), dict(vocab=0), dict(vocab=(1 << 31) - 1), dict(cols=0),
               dict(cols=(1 << 22) + 1), dict(vocab=1 << 30, cols=1 << 20), dict(dtype=3), dict(dtype=-1), dict(token_bits=16),
               dict(table=0), dict(tokens=0), dict(out=0), dict(table=FAKE + 1), dict(out=FAKE + 2, dtype=q.QMUON_FP32),
               dict(tokens=FAKE + 4), dict(ld_table=63), dict(ld_out=63), dict(ld_out=1 << 41)):
        assert call(**kw) == INV, kw
    assert call(n_tokens=0) == q.QMUON_OK


def test_embedding_backward_refusals(L):
    def call(ws=FAKE, ws_bytes=1 << 40, **kw):
        c = q.qmuon_embedding_grad(FAKE, FAKE, FAKE, 4, 16, 64, 64, 64, 1.0, q.QMUON_BF16, q.QMUON_BF16, 64, 0, 0)
        return L.qmuon_embedding_backward(C.byref(_with(c, kw)), ws, ws_bytes, None)
    assert L.qmuon_embedding_backward(None, FAKE, 1 << 20, None) == INV
    for kw in (dict(n_tokens=-1), dict(vocab=0), dict(cols=0), dict(dtype=7), dict(grad_dtype=q.QMUON_FP16), dict(grad_dtype=5),
               dict(dout=0), dict(tokens=0), dict(dtable=0), dict(dtable=FAKE + 2, grad_dtype=q.QMUON_FP32), dict(token_bits=0),
               dict(tokens=FAKE + 2, token_bits=32), dict(ld_dout=63), dict(ld_dtable=63), dict(ws=0), dict(ws=FAKE + 128)):
        assert call(**kw) == INV, kw
    need = q.qmuon_embedding_workspace_size(4, 16, 64)
    assert need > 0 and call(ws_bytes=need - 1) == q.QMUON_ERR_WORKSPACE_TOO_SMALL
    assert call(n_tokens=0, accumulate=1) == q.QMUON_OK           # nothing to do, nothing launched
    for sizes in ((-1, 16, 64), (4, 0, 64), (4, 16, 0), (1 << 29, 16, 64), (4, 1 << 31, 64)):
        assert q.qmuon_embedding_workspace_size(*sizes) == 0


@pytest.mark.parametrize("name", ["qmuon_mxfp8_encode", "qmuon_mxfp8_decode"])
def test_mxfp8_refusals(L, name):
    fn = getattr(L, name)
    call = lambda **kw: fn(C.byref(_with(q.qmuon_mxfp8(FAKE, FAKE, FAKE, 4, 64, 64, q.QMUON_BF16, 0), kw)), None)   # noqa: E731
    assert fn(None, None) == INV
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=1 << 31), dict(rows=1 << 40), dict(dtype=3), dict(x=0), dict(payload=0),
               dict(scale_inv=0), dict(x=FAKE + 1), dict(x=FAKE + 2, dtype=q.QMUON_FP32), dict(payload=FAKE + 8), dict(ld_x=63)):
        assert call(**kw) == INV, kw
    assert call(cols=48) == UNS
    assert call(rows=0) == q.QMUON_OK


def _ffn(**kw):
    return _with(q.qmuon_gated_ffn(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 96, 64, 64, 64, 96, 96, 96, q.QMUON_ACT_SILU,
                                   q.QMUON_BF16, q.QMUON_SAVE_NONE, 0), kw)


def test_gated_ffn_forward_refusals(L):
    def call(ws=FAKE, ws_bytes=1 << 40, **kw):
        return L.qmuon_gated_ffn_forward(C.byref(_ffn(**kw)), ws, ws_bytes, None)
    S, M = q.QMUON_SAVE_SAME, q.QMUON_SAVE_MXFP8
    assert L.qmuon_gated_ffn_forward(None, FAKE, 1 << 20, None) == INV
    bad = (dict(rows=-1), dict(width=0), dict(inner=0), dict(rows=(1 << 28) + 1), dict(inner=1 << 28, width=1 << 20),
           dict(rows=1 << 28, inner=1 << 20), dict(act=3), dict(act=-1), dict(dtype=3), dict(saved=3), dict(saved=-1), dict(x=0),
           dict(w_gate=0), dict(w_up=0), dict(h=0), dict(x=FAKE + 1), dict(h=FAKE + 1), dict(ld_x=63), dict(ld_w_gate=63),
           dict(ld_w_up=63), dict(ld_h=95), dict(saved=S, gate=0), dict(saved=S, up=0), dict(saved=S, ld_gate=95),
           dict(saved=S, ld_up=95), dict(saved=M, gate=FAKE + 8), dict(saved=M, up=FAKE + 8), dict(saved=M, gate_scale=0),
           dict(saved=M, up_scale=0))
    for kw in bad:
        assert call(**kw) == INV, kw
        assert L.qmuon_gated_ffn_workspace_size(C.byref(_ffn(**kw))) == 0, kw
    assert call(ws=0) == INV and call(ws=FAKE + 128) == INV
    assert call(dtype=q.QMUON_FP32) == UNS and call(saved=M, inner=97, ld_h=97) == UNS
    assert call(rows=0) == q.QMUON_OK
    # rows that do not start on 16 bytes are copied, but for small products: the workspace says so
    big = dict(rows=300, width=1024, inner=2048, ld_x=1024, ld_w_gate=1024, ld_w_up=1024, ld_h=2048)
    size = lambda **kw: L.qmuon_gated_ffn_workspace_size(C.byref(_ffn(**kw)))   # noqa: E731
    assert size(**big) > 0 and size(**{**big, "x": FAKE + 2}) >= size(**big) + 300 * 1024 * 2
    assert size(**{**big, "ld_w_up": 1025}) >= size(**big) + 2048 * 1024 * 2
    assert size(ld_w_up=65) == size() > 0


def _grad(**kw):
    return _with(q.qmuon_gated_ffn_grad(*[FAKE] * 2, None, *[FAKE] * 10, 4, 64, 96, 96, 64, 64, 64, 96, 96, 64, 64, 64, 96,
                                        q.QMUON_ACT_SILU, q.QMUON_BF16, q.QMUON_SAVE_NONE, q.QMUON_BF16, 0, 0), kw)


def test_gated_ffn_backward_refusals(L):
    def call(ws=FAKE, ws_bytes=1 << 40, **kw):
        return L.qmuon_gated_ffn_backward(C.byref(_grad(**kw)), ws, ws_bytes, None)
    S, M = q.QMUON_SAVE_SAME, q.QMUON_SAVE_MXFP8
    assert L.qmuon_gated_ffn_backward(None, FAKE, 1 << 20, None) == INV
    bad = (dict(rows=-1), dict(width=0), dict(inner=0), dict(act=3), dict(dtype=3), dict(saved=3), dict(grad_dtype=q.QMUON_FP16),
           dict(dh=0), dict(x=0), dict(w_gate=0), dict(w_up=0), dict(dw_gate=0), dict(dw_up=0), dict(dx=0, dw_gate=0, dw_up=0, h=0),
           dict(dh=FAKE + 1), dict(dx=FAKE + 1), dict(dw_up=FAKE + 2, grad_dtype=q.QMUON_FP32), dict(ld_dh=95), dict(ld_x=63),
           dict(ld_w_gate=63), dict(ld_dx=63), dict(ld_dw_gate=63), dict(ld_dw_up=63), dict(ld_h=95), dict(saved=S, gate=0),
           dict(saved=S, ld_up=95), dict(saved=M, gate=FAKE + 8), dict(saved=M, up_scale=0), dict(x_scale=FAKE, x=FAKE + 8))
    for kw in bad:
        assert call(**kw) == INV, kw
        assert L.qmuon_gated_ffn_backward_workspace_size(C.byref(_grad(**kw))) == 0, kw
    assert call(ws=0) == INV and call(ws=FAKE + 128) == INV
    assert call(dtype=q.QMUON_FP32) == UNS and call(saved=M, inner=97, ld_dh=97, ld_h=97) == UNS
    assert call(x_scale=FAKE, width=65, **{"ld_" + k: 65 for k in ("w_gate", "w_up", "dx", "dw_gate", "dw_up")}) == UNS
    assert call(rows=0, accumulate=1) == q.QMUON_OK and call(rows=0, dw_gate=0, dw_up=0) == q.QMUON_OK
    # what a call does not read may be missing
    size = lambda **kw: L.qmuon_gated_ffn_backward_workspace_size(C.byref(_grad(**kw)))   # noqa: E731
    assert size(saved=S, dw_gate=0, dw_up=0, x=0) > 0 and size(saved=S, dx=0, w_gate=0, w_up=0) > 0
    assert size(saved=S, x=FAKE + 2) >= size(saved=S) + 4 * 64 * 2


def test_binding_refuses_other_tensors():
    def refused(call, *words):
        with pytest.raises(q.QmuonError) as e:
            call()
        assert e.value.status == INV
        for w in words:
            assert w in str(e.value), (w, str(e.value))
    x, t = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    p = FAKE
    refused(lambda: q.qmuon_embedding_forward(x, t, x, 4, 4, 64, "bf16", stream=0), "tokens has to be", "cpu")
    refused(lambda: q.qmuon_embedding_forward(p, x, p, 4, 4, 64, "bf16", stream=0), "tokens has to be", "int32 or int64")
    refused(lambda: q.qmuon_embedding_forward(x, p, p, 4, 4, 64, "bf16", stream=0), "table has to be")
    refused(lambda: q.qmuon_embedding_forward(p, p, p, 4, 4, 64, "e4m3", stream=0))
    refused(lambda: q.qmuon_embedding_backward(x, p, p, 4, 4, 64, "bf16", p, ws_bytes=1, stream=0), "dout has to be")
    refused(lambda: q.qmuon_mxfp8_encode(x, p, p, 4, 64, "bf16", stream=0), "x has to be")
    refused(lambda: q.qmuon_mxfp8_decode(x, p, p, 4, 64, "bf16", stream=0), "payload has to be", "one byte")
    refused(lambda: q.gated_ffn(x, p, p, p, 4, 64, 96, "bf16"), "x has to be", "cpu")
    refused(lambda: q.gated_ffn(p, p, p, p, 4, 64, 96, "bf16", saved="mxfp8", gate=x, up=p), "gate has to be", "one byte")
    refused(lambda: q.gated_ffn(p, p, p, p, 4, 64, 96, "bf16", act="relu"))
    refused(lambda: q.gated_ffn_grad(x, p, p, p, p, p, p, 4, 64, 96, "bf16"), "dh has to be", "cpu")
    for rows in (1 << 70, 1.5):
        refused(lambda: q.qmuon_embedding_forward(p, p, p, rows, 4, 64, "bf16", stream=0))
        refused(lambda: q.qmuon_mxfp8_encode(p, p, p, rows, 64, "bf16", stream=0))
        refused(lambda: q.gated_ffn(p, p, p, p, rows, 64, 96, "bf16"))
        refused(lambda: q.gated_ffn_grad(p, p, p, p, p, p, p, rows, 64, 96, "bf16"))
