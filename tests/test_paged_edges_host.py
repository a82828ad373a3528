"""Host-side edges of the paged-cache calls (no GPU needed)."""
import pytest
import torch

import causal_kernelized_sequence_b200 as la
from test_paged_host import _state, _z


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


F, I, H = torch.float32, torch.int32, torch.bfloat16


def _fill(k=None, v=None, state=None, **kw):
    return lambda: la.la_paged_cache_fill(_z(3, 2, 5, 64) if k is None else k, _z(3, 2, 5, 32) if v is None else v,
                                          *(state or _state()), **kw)


def _step(q=None, k=None, v=None, state=None, **kw):
    return lambda: la.la_paged_decode_step(_z(3, 4, 64) if q is None else q, k, v, *(state or _state()), **kw)


def _evict(w=None, state=None, budget=32, **kw):
    return lambda: la.la_paged_evict(*(state or _state()), _z(3, 2, 64, dtype=F) if w is None else w, budget, **kw)


SLOTS, LONG = _z(3, 2, 64, dtype=F), torch.int64


@pytest.mark.parametrize("call,name", [
    (_fill(k=_z(3, 2, 5, 63)), "k"), (_fill(k=_z(3, 2, 5, 64, dtype=F)), "k"), (_fill(v=_z(3, 2, 4, 32)), "v"),
    (_fill(state=_state(lens=_z(2, dtype=I))), "lens"), (_fill(state=_state(lens=_z(3, dtype=LONG))), "lens"),
    (_fill(state=_state(block_table=_z(3, 4, dtype=LONG))), "block_table"),
    (_fill(state=_state(v_pages=_z(15, 2, 16, 32))), "v_pages"), (_fill(n_new=_z(3, dtype=LONG)), "n_new"),
    (_fill(weights=_z(3, 2, 63, dtype=F)), "weights"), (_fill(weights=_z(3, 2, 64)), "weights"),
    (_fill(positions=_z(3, 2, 64, dtype=LONG), pos=_z(3, dtype=I)), "positions"),
    (_fill(positions=_z(3, 2, 64, dtype=I), pos=_z(2, dtype=I)), "pos"),
    (_step(q=_z(2, 4, 64)), "q"), (_step(q=_z(3, 4, 64, dtype=F)), "q"), (_step(k=_z(3, 1, 64), v=_z(3, 2, 32)), "k"),
    (_step(k=_z(3, 2, 64), v=_z(3, 2, 64)), "v"), (_step(y=_z(3, 4, 64)), "y"), (_step(lse=_z(3, 4)), "lse"),
    (_step(lse=_z(3, 2, dtype=F)), "lse"), (_step(weights=_z(3, 2, 63, dtype=F)), "weights"),
    (_step(weights=SLOTS, weights_out=_z(3, 2, 64)), "weights_out"),
    (_step(state=_state(v_pages=_z(16, 2, 8, 32))), "v_pages"),
    (_evict(w=_z(3, 2, 64)), "weights"), (_evict(w=_z(3, 2, 48, dtype=F)), "weights"),
    (_evict(weights_out=_z(3, 1, 64, dtype=F)), "weights_out"), (_evict(lens_out=_z(3, dtype=LONG)), "lens_out"),
    (_evict(positions=_z(3, 2, 64)), "positions"),
    (_evict(recent=1, positions=_z(3, 2, 64, dtype=I), pos=_z(1, dtype=I)), "pos"),
    (_evict(positions=_z(3, 2, 64, dtype=I), positions_out=_z(3, 2, 64)), "positions_out"),
])
def test_refusal_names_its_tensor(lib, call, name):
    """One tensor of a call is wrong, and the refusal names that one."""
    with pytest.raises(ValueError, match=f"^{name}: expected"):
        call()


@pytest.mark.parametrize("call,text", [
    (_fill(positions=_z(3, 2, 64, dtype=I)), "^positions and pos go together$"),
    (_fill(pos=_z(3, dtype=I)), "^positions and pos go together$"),
    (_step(k=_z(3, 2, 64)), "^k and v go together$"), (_step(v=_z(3, 2, 32)), "^k and v go together$"),
    (_step(pos=_z(3, dtype=I)), "^positions and pos go together$"),
    (_step(positions=_z(3, 2, 64, dtype=I), pos=_z(3, dtype=I)), "^positions need a new token"),
    (_step(weights_out=SLOTS), "^weights_out needs weights$"),
    (_evict(recent=4), "^recent > 0 needs positions and pos$"),
    (_evict(recent=4, positions=_z(3, 2, 64, dtype=I)), "^recent > 0 needs positions and pos$"),
    (_evict(positions_out=_z(3, 2, 64, dtype=I)), "^positions_out needs positions$"),
])
def test_refusal_of_arguments_that_go_together(lib, call, text):
    with pytest.raises(ValueError, match=text):
        call()
