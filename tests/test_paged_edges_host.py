"""Host-side edges of the paged-cache calls (no GPU needed)."""
import ctypes

import pytest
import torch

import causal_kernelized_sequence_b200 as la


@pytest.fixture(scope="module")
def lib():
    from causal_kernelized_sequence_b200 import build
    build.build()
    return la.load_library()


def test_kept_workspace_sizes_are_bounded(lib):
    """A run that meets ever new batch sizes and widths keeps a bounded number of sizes, and they stay right."""
    cpu = torch.device("cpu")
    for i in range(1, 5001):
        _, have, _ = la._paged_workspace("la_paged_evict_workspace_bytes", None, cpu, 1 + i % 7, 2, 16, i, 8)
        assert have >= la.la_paged_evict_workspace_bytes(1 + i % 7, 2, 16, i, 8)
    assert len(la._paged_sizes) <= 1024
