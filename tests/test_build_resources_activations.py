"""Register and spill budgets of the embedding's, the gated block's and the
checkpoints' kernels, from ptxas's report (CPU only).

The gated block's tensor-core kernel runs one CTA of 320 threads per SM, the
kernel of few rows three of 256 (80 registers), the embedding's sums four of
256 (64).  None of them spills but the kernel of few rows for rows that do not
start on 16 bytes and one product at a time: 4 bytes as it stands, and no more."""

import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from memory_reduced_muon_gb300 import build
from test_build_resources import _report, pytestmark  # noqa: F401

# kernel: registers at most
CAPS = {"ffn_kernel": 168, "few_kernel": 80, "elem_kernel": 128, "dh_max_kernel": 64, "11join_kernelE": 64, "clear_kernel": 32,
        "lookup_kernel": 64, "cluster_sort_kernel": 128, "count_kernel": 64, "offsets_kernel": 128, "scatter_kernel": 128, "sum_kernel": 64,
        "11join_kernelI": 64, "encode": 64, "decode": 64, "repack_kernel": 64}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("ptxas")
    with ThreadPoolExecutor(3) as ex:
        reports = ex.map(lambda f: _report(os.path.join(build.CSRC, f), tmp), ("ffn.cu", "embedding.cu", "mxfp8.cu"))
    return {n: v for r in reports for n, v in r.items()}


def test_every_kernel_has_its_budget(kernels):
    for key in CAPS:
        assert any(key in n for n in kernels), key
    for n, v in kernels.items():
        caps = [cap for key, cap in CAPS.items() if key in n]
        assert len(caps) == 1, (n, caps)
        assert v["regs"] <= caps[0], (n, v)


def test_no_kernel_spills_but_one(kernels):
    for n, v in kernels.items():
        small = "few_kernel" in n and "Li1ELb0E" in n        # one product of 8 rows at a time, rows off 16 bytes
        assert v["spill"] <= (8 if small else 0), (n, v)
