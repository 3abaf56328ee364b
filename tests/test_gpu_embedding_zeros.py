"""The zeros that the embedding's gradient writes to rows without a token: those
of the table's last 64 MB while the tokens are sorted, by as many threads as a
row has vectors, and the others' behind it.  Whole numbers, compared exactly."""

import pytest
import torch

import memory_reduced_muon_gb300 as q

from test_gpu_embedding import DT, Matrix

pytestmark = pytest.mark.gpu


# rows of one vector, of a number that is no power of two, of a whole CTA's threads and one more; tables of less and of more
# than 64 MB, and one whose last rows begin in the middle of what a CTA writes
@pytest.mark.parametrize("vocab,cols,pad,dtype", [(5000011, 8, 0, "bf16"), (3000001, 4, 8, "f32"), (700001, 24, 8, "f16"), (70001, 1000, 0, "bf16"),
                                                  (9001, 4096, 8, "bf16"), (9001, 4104, 0, "f16"), (1, 2048, 0, "f32"), (3, 8, 8, "bf16"),
                                                  (40, 2056, 0, "f32")])
@pytest.mark.parametrize("n", [1, 700, 20000])
def test_rows_without_a_token(vocab, cols, pad, dtype, n):
    gen = torch.Generator("cuda").manual_seed(vocab + n)
    tokens = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    tokens[torch.rand(n, generator=gen, device="cuda") < 0.1] = -1
    tokens[0] = vocab - 1
    if n > 1:
        tokens[1] = 0
    dout = torch.randint(-1, 2, (n, cols), generator=gen, device="cuda").to(DT[dtype])
    grad = Matrix(vocab, cols, pad, DT[dtype], 0)
    grad.t.fill_(float("nan"))
    ws = torch.empty(q.qmuon_embedding_workspace_size(n, vocab, cols), dtype=torch.uint8, device="cuda")
    q.qmuon_embedding_backward(dout, tokens, grad.t, n, vocab, cols, dtype, ws, ld_dtable=grad.ld)
    grad.check()
    there = tokens >= 0
    want = torch.zeros(vocab, cols, device="cuda").index_add_(0, tokens[there], dout[there].float())
    assert torch.equal(grad.t, want.to(DT[dtype]))
