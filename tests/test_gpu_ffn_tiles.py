"""The gated block's projections on the tensor cores, by the tiles that a call
takes: 128 or 64 columns of gate and of up, forward and computed again in the
backward pass, finished by the product's own epilogue or through partial sums,
in one piece of K or several.  Which of them a size goes to is the library's
choice, so each test looks at the kernels that ran.  Bounds as in the tests of
the small sizes, whose projections go through the cores' registers."""

import re
import warnings

import pytest
import torch

import memory_reduced_muon_gb300 as q

from test_gpu_ffn import _backward, _check_forward

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh"]
TYPES = ["bf16", "f16"]
FWD, BWD = 0, 1
FROM_PART = 0
_profiles = False


def _ran(f):
    """(the call's result, [(kernel, its numbers)] of the gated block's kernels that it launched)."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        r = f()
        torch.cuda.synchronize()
    found = [re.search(r"::(ffn_kernel|elem_kernel|few_kernel)<([^>]*)>", e.name) for e in p.events()]
    return r, [(m.group(1), [{"true": 1, "false": 0}.get(v.strip()) if v.strip() in ("true", "false") else int(re.sub(r"\(.*?\)", "", v))
                             for v in m.group(2).split(",")]) for m in found if m]


@pytest.fixture(scope="module", autouse=True)
def _profiler_has_run():
    """A process's first profile shows torch's launches only.  Where no profile shows any kernel, because another tool holds the
    GPU's counters, the values are tested and the kernels are not looked at."""
    global _profiles
    x, w, h = (torch.ones(n, 8, dtype=torch.bfloat16, device="cuda") for n in (4, 8, 4))
    call = q.gated_ffn(x, w, w, h, 4, 8, 8, "bf16")
    ws = torch.empty(q.qmuon_gated_ffn_workspace_size(call), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        _, kernels = _ran(lambda: q.qmuon_gated_ffn_forward(call, ws))
    _profiles = bool(kernels)
    if not _profiles:
        warnings.warn("torch.profiler shows no kernels here: which of them ran is not tested")


def _went(kernels, kind, dtype, name, columns, joined):
    """The projections went by tiles of `columns` columns; `joined`: and through partial sums, not straight to the results."""
    if not _profiles:
        return
    tiles = [k for n, k in kernels if n == "ffn_kernel" and k[0] == kind]
    assert tiles == [[kind, TYPES.index(dtype), ACTS.index(name), columns]], kernels
    assert any(n == "elem_kernel" and k[2] == FROM_PART for n, k in kernels) == joined, kernels
    assert not any(n == "few_kernel" for n, _ in kernels)


# shape (rows, width, inner, pad, off), columns of a tile, through partial sums.  Of either width: more tiles than pairs or
# ragged in every size; K round the ring of shared memory; K in pieces; rows that leave by elements
TILES = [((513, 136, 5984, 0, 0), 128, False), ((600, 1032, 3008, 0, 8), 128, False), ((1000, 4104, 224, 0, 0), 128, True),
         ((3001, 64, 2016, 3, 1), 128, True), ((257, 1100, 416, 0, 0), 64, False), ((1000, 520, 224, 8, 0), 64, False),
         ((260, 2056, 192, 0, 0), 64, True), ((129, 2001, 320, 3, 1), 64, True)]
BOTH = [("bf16", "silu"), ("f16", "gelu"), ("bf16", "gelu_tanh"), ("f16", "silu"), ("bf16", "gelu"), ("f16", "gelu_tanh")]


@pytest.mark.parametrize("shape,columns,joined", TILES, ids=str)
@pytest.mark.parametrize("i", range(6), ids=lambda k: "-".join(BOTH[k]))
def test_forward(shape, columns, joined, i):
    dtype, name = BOTH[i]
    saved = ("mxfp8", "same", "none", "none", "same", "mxfp8")[i]
    _, kernels = _ran(lambda: _check_forward(shape, dtype, name, saved))
    _went(kernels, FWD, dtype, name, columns, joined)


@pytest.mark.parametrize("shape,columns,joined", TILES, ids=str)
@pytest.mark.parametrize("i", range(6), ids=lambda k: "-".join(BOTH[k]))
def test_backward_from_nothing_kept(shape, columns, joined, i):
    dtype, name = BOTH[i]
    _, kernels = _ran(lambda: _backward(shape, dtype, name, "none", again=i % 2 == 0))
    _went(kernels, BWD, dtype, name, columns, joined)


@pytest.mark.parametrize("shape", [(513, 160, 5984, 0, 0), (257, 1120, 416, 0, 0)], ids=str)
def test_backward_from_a_carrier_of_x(shape):
    _, kernels = _ran(lambda: _backward(shape, "bf16", "silu", "none", x_mxfp8=True))
    _went(kernels, BWD, "bf16", "silu", 128 if shape[0] == 513 else 64, False)
