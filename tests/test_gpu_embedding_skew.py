"""The embedding's gradient where some tokens are most of the batch: which rows
have no token is found by searches there instead of a look at every token of
the rows.  Bounds as in the tests of ordinary tokens, but sums of whole numbers
up to 2^24, which fp32 holds, are compared exactly."""

import pytest
import torch

import memory_reduced_muon_gb300 as q

from test_gpu_embedding import DT, Matrix

pytestmark = pytest.mark.gpu


def _frequent(n, vocab, rows, share, gen):
    """Tokens of which `share` are one of `rows`, the others any but none just beside these rows."""
    other = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    near = torch.tensor([r + d for r in rows for d in (-1, 1)], device="cuda")
    other = torch.where(torch.isin(other, near), torch.full_like(other, rows[0]), other)
    pick = torch.tensor(rows, device="cuda")[torch.randint(0, len(rows), (n,), generator=gen, device="cuda")]
    return torch.where(torch.rand(n, generator=gen, device="cuda") < share, pick, other)


# columns of one and of eight warps, by vectors and by elements; rows at both ends of a CTA's 16 and of the table; sorted by
# one cluster (elements only: else it writes these rows' zeros itself) and by several kernels
@pytest.mark.parametrize("n,vocab,cols,pad,dtype", [(65536, 1000, 33, 0, "f32"), (65536, 5003, 301, 2, "bf16"), (200000, 1000, 64, 0, "bf16"),
                                                    (200000, 5003, 2048, 0, "f32"), (70000, 17, 8, 0, "f16"), (1 << 20, 102400, 16, 0, "f32")])
@pytest.mark.parametrize("rows,share", [((7,), 0.95), ((0, 15, 16), 0.9), ((3, 11), 1.0)])
def test_frequent_tokens(n, vocab, cols, pad, dtype, rows, share):
    gen = torch.Generator("cuda").manual_seed(n + vocab)
    tokens = _frequent(n, vocab, rows, share, gen)
    top = 3 if dtype == "f32" else 1
    dout = Matrix(n, cols, pad, DT[dtype], 0, torch.randint(-top, top + 1, (n, cols), generator=gen, device="cuda").float())
    grad = Matrix(vocab, cols, pad, torch.float32, 0, torch.full((vocab, cols), 7.0, device="cuda"))
    ws = torch.empty(q.qmuon_embedding_workspace_size(n, vocab, cols), dtype=torch.uint8, device="cuda")
    q.qmuon_embedding_backward(dout.t, tokens, grad.t, n, vocab, cols, dtype, ws, grad_dtype="f32", ld_dout=dout.ld, ld_dtable=grad.ld)
    want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, tokens, dout.t.double())
    assert torch.equal(grad.t.double(), want)
    grad.check()
    dout.check()
