"""Host-side checks of the paged-cache calls (no GPU needed): the C entry points refuse bad arguments before any
launch, the binding refuses tensors that disagree, and the oracle's step agrees with itself on simple cases."""
import ctypes
import math

import pytest
import torch

import causal_kernelized_sequence_b200 as la
from oracle import paged as orc

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from causal_kernelized_sequence_b200 import build
    build.build()
    return la.load_library()


def _fill(lib, k=0x1000, v=0x2000, kp=0x3000, vp=0x4000, tab=0x5000, lens=0x6000, nn=None, w=None, ps=None, pos=None,
          B=2, Hkv=2, N=8, dqk=64, dv=64, num=16, page=16, mp=4, dt=1):
    return lib.la_paged_cache_fill(P(k), P(v), P(kp), P(vp), P(tab), P(lens), P(nn), P(w), P(ps), P(pos), B, Hkv, N,
                                   dqk, dv, num, page, mp, dt, None)


def _step(lib, q=0x1000, k=0x2000, v=0x3000, y=0x4000, lse=None, kp=0x5000, vp=0x6000, tab=0x7000, lens=0x8000,
          wi=None, wo=None, ps=None, pos=None, ws=0x100000, wsb=1 << 40, B=2, Hq=4, Hkv=2, dqk=64, dv=64, num=16,
          page=16, mp=4, dt=1):
    return lib.la_paged_decode_step(P(q), P(k), P(v), P(y), P(lse), P(kp), P(vp), P(tab), P(lens), P(wi), P(wo), P(ps),
                                    P(pos), P(ws), wsb, B, Hq, Hkv, dqk, dv, num, page, mp, dt, None)


def _evict(lib, kp=0x1000, vp=0x2000, tab=0x3000, lens=0x4000, lo=0x4000, wi=0x10000, wo=0x10000, pi=0x20000,
           po=0x20000, pos=0x5000, ws=0x100000, wsb=1 << 40, B=2, Hkv=2, dqk=64, dv=64, num=16, page=16, mp=4,
           budget=32, recent=8, dt=1):
    return lib.la_paged_evict(P(kp), P(vp), P(tab), P(lens), P(lo), P(wi), P(wo), P(pi), P(po), P(pos), P(ws), wsb, B,
                              Hkv, dqk, dv, num, page, mp, budget, recent, dt, None)


SIZES = [dict(B=0), dict(Hkv=0), dict(dqk=0), dict(dv=-1), dict(num=0), dict(page=0), dict(mp=0), dict(dt=2),
         dict(num=1 << 20, page=1 << 11, Hkv=2, Hq=2), dict(page=1 << 16, mp=1 << 15, num=1),
         dict(page=1 << 15, mp=1 << 15, num=1)]
MISALIGNED = [dict(kp=0x5008), dict(vp=0x6004), dict(tab=0x7002), dict(lens=0x8001), dict(kp=None), dict(vp=None),
              dict(tab=None), dict(lens=None)]


def _only(call, kw):
    names = call.__code__.co_varnames[:call.__code__.co_argcount]
    return {k: v for k, v in kw.items() if k in names}


@pytest.mark.parametrize("call", [_fill, _step, _evict])
def test_sizes_and_cache_pointers_refused(lib, call):
    for kw in SIZES + MISALIGNED:
        assert call(lib, **_only(call, kw)) == 1, kw
    for kw in (dict(dqk=129), dict(dv=256)):
        assert call(lib, **kw) == 2, kw            # LA_ERR_UNSUPPORTED


def test_fill_arguments_refused(lib):
    for kw in (dict(k=None), dict(v=None), dict(N=0), dict(N=-1), dict(k=0x1008), dict(nn=0x9002), dict(w=0x9001),
               dict(ps=0x9000), dict(pos=0x9000), dict(ps=0x9002, pos=0x9000)):
        assert _fill(lib, **kw) == 1, kw


def test_step_arguments_refused(lib):
    for kw in (dict(q=None), dict(y=None), dict(k=None), dict(v=None), dict(q=0x1004), dict(y=0x4002), dict(lse=0x9002),
               dict(Hq=3), dict(Hq=0), dict(wi=0x9000), dict(wo=0x9000), dict(ps=0x9000), dict(pos=0x9000),
               dict(k=None, v=None, ps=0x9000, pos=0xa000),          # positions without a new token
               dict(wi=0x10000, wo=0x10010),                         # overlapping, not the same
               dict(wi=0x10002, wo=0x20000)):
        assert _step(lib, **kw) == 1, kw
    assert _step(lib, Hq=258) == 2                 # 129 query heads on one key/value head
    need = la.la_paged_decode_workspace_bytes(2, 4, 2, 64, 64, 16, 4, True, la.LA_BF16)
    w = dict(wi=0x10000, wo=0x10000)
    assert _step(lib, wsb=need - 1, **w) == 1 and _step(lib, ws=None, **w) == 1 and _step(lib, ws=0x100004, **w) == 1
    assert la.la_paged_decode_workspace_bytes(2, 4, 2, 64, 64, 16, 4, False, la.LA_BF16) < need


def test_evict_arguments_refused(lib):
    for kw in (dict(budget=0), dict(recent=-1), dict(recent=33), dict(lo=None), dict(wi=None), dict(wo=None),
               dict(pi=None), dict(po=None), dict(pos=None), dict(pi=None, po=None), dict(lo=0x4004), dict(wo=0x10010),
               dict(po=0x20020), dict(ws=None), dict(ws=0x100008), dict(wsb=4)):
        assert _evict(lib, **kw) == 1, kw


def test_workspace_bytes(lib):
    f = la.la_paged_evict_workspace_bytes
    assert f(2, 3, 16, 4, 32) == (6 * 2 * 32 + 2) * 4                # 64 slots, half of them move at most
    assert f(2, 3, 16, 4, 60) == (6 * 2 * 4 + 2) * 4
    assert f(2, 3, 16, 4, 100) == 2 * 4                              # nothing can move
    assert f(0, 3, 16, 4, 32) == 0 and f(2, 3, 16, 4, 0) == 0
    assert la.la_paged_decode_workspace_bytes(2, 3, 2, 64, 64, 16, 4, False, la.LA_BF16) == 0      # 3 heads over 2


def test_kernel_plan(lib):
    assert la.la_paged_kernel_plan(0, 2, 0, 2, 64, 64, 16, 4, False, la.LA_F32) == (1, ["paged_fill_kernel"])
    assert la.la_paged_kernel_plan(2, 2, 0, 2, 64, 64, 16, 4, False, la.LA_BF16)[0] == 2
    assert la.la_paged_kernel_plan(1, 2, 3, 2, 64, 64, 16, 4, False, la.LA_BF16)[0] == -1
    assert la.la_paged_kernel_plan(3, 2, 2, 2, 64, 64, 16, 4, False, la.LA_BF16)[0] == -1
    n, names = la.la_paged_kernel_plan(1, 2, 4, 2, 64, 64, 16, 4, True, la.LA_BF16)
    assert n == len(names) >= 1


def _state(**kw):
    s = {"k_pages": torch.zeros(16, 2, 16, 64, dtype=torch.bfloat16), "v_pages": torch.zeros(16, 2, 16, 32, dtype=torch.bfloat16),
         "block_table": torch.zeros(3, 4, dtype=torch.int32), "lens": torch.zeros(3, dtype=torch.int32)}
    s.update(kw)
    return list(s.values())


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


F, I = torch.float32, torch.int32


@pytest.mark.parametrize("call,what", [
    (lambda: la.la_paged_cache_fill(_z(3, 2, 5, 64), _z(3, 2, 5, 32), *_state()), "CUDA"),
    (lambda: la.la_paged_cache_fill(_z(3, 2, 5, 64), _z(3, 2, 4, 32), *_state()), "v"),
    (lambda: la.la_paged_cache_fill(_z(3, 2, 5, 64, dtype=F), _z(3, 2, 5, 32), *_state()), "k"),
    (lambda: la.la_paged_cache_fill(_z(3, 2, 5, 64), _z(3, 2, 5, 32), *_state(lens=_z(2, dtype=I))), "lens"),
    (lambda: la.la_paged_cache_fill(_z(3, 2, 5, 64), _z(3, 2, 5, 32), *_state(), n_new=_z(3, dtype=torch.int64)), "n_new"),
    (lambda: la.la_paged_cache_fill(_z(3, 2, 5, 64), _z(3, 2, 5, 32), *_state(), positions=_z(3, 2, 64, dtype=I)), "pos"),
    (lambda: la.la_paged_decode_step(_z(3, 4, 64), _z(3, 2, 64), _z(3, 2, 32), *_state()), "CUDA"),
    (lambda: la.la_paged_decode_step(_z(3, 4, 64), None, None, *_state(), weights=_z(3, 2, 64, dtype=F),
                                     weights_out=_z(3, 2, 64, dtype=F), lse=_z(3, 4, dtype=F)), "CUDA"),
    (lambda: la.la_paged_decode_step(_z(3, 4, 64), _z(3, 2, 64), None, *_state()), "together"),
    (lambda: la.la_paged_decode_step(_z(3, 4, 64), None, None, *_state(), positions=_z(3, 2, 64, dtype=I),
                                     pos=_z(3, dtype=I)), "new token"),
    (lambda: la.la_paged_decode_step(_z(3, 4, 64), None, None, *_state(), weights_out=_z(3, 2, 64, dtype=F)), "weights"),
    (lambda: la.la_paged_decode_step(_z(2, 4, 64), None, None, *_state()), "q"),
    (lambda: la.la_paged_decode_step(_z(3, 4, 64), None, None, *_state(), weights=_z(3, 2, 63, dtype=F)), "weights"),
    (lambda: la.la_paged_decode_step(_z(3, 4, 64), None, None, *_state(v_pages=_z(15, 2, 16, 32))), "v_pages"),
    (lambda: la.la_paged_evict(*_state(), _z(3, 2, 64, dtype=F), 32), "CUDA"),
    (lambda: la.la_paged_evict(*_state(), _z(3, 2, 64, dtype=F), 32, recent=4), "positions"),
    (lambda: la.la_paged_evict(*_state(), _z(3, 2, 64), 32), "weights"),
    (lambda: la.la_paged_evict(*_state(), _z(3, 2, 64, dtype=F), 32, positions_out=_z(3, 2, 64, dtype=I)), "positions"),
])
def test_binding_refuses(lib, call, what):
    with pytest.raises(ValueError, match=what):
        call()


def test_oracle_step_closed_forms():
    """Equal keys give the mean of the values; one token gives its value; the weights of a head sum to one."""
    kp, vp = torch.ones(3, 1, 4, 8), torch.arange(3 * 4 * 2, dtype=torch.float64).view(3, 1, 4, 2)
    table, lens = torch.tensor([[2, 0], [1, -1], [0, 0]], dtype=torch.int32), torch.tensor([6, 1, 0], dtype=torch.int32)
    q = torch.randn(3, 2, 8, generator=torch.Generator().manual_seed(0))
    y, lse, w, size, spread = orc.decode(q, None, None, kp, vp, table, lens, torch.zeros(3, 1, 8))
    rows = torch.cat([vp[2, 0], vp[0, 0, :2]])
    assert torch.allclose(y[0], rows.mean(0).expand(2, 2)) and torch.equal(y[1], vp[1, 0, 0].expand(2, 2))
    assert torch.equal(y[2], torch.zeros(2, 2).double()) and (lse[2] == -math.inf).all()
    assert torch.allclose(w.sum(-1)[:, 0], torch.tensor([2.0, 2.0, 0.0]).double())
    assert torch.allclose(lse[0], q[0].double().sum(1) / math.sqrt(8) + math.log(6))


def test_oracle_evict_example():
    """Five slots, budget three: the recent one and the two heaviest stay; slot 4 fills the lowest hole."""
    kp = torch.arange(6.0).view(2, 1, 3, 1)
    table, lens = torch.tensor([[1, 0]], dtype=torch.int32), torch.tensor([5], dtype=torch.int32)
    w = torch.tensor([[[0.5, 0.1, 0.5, 0.5, 0.2, 9.0]]])
    posn = torch.tensor([[[0, 1, 2, 3, 4, 7]]], dtype=torch.int32)
    k2, _, l2, w2, p2 = orc.evict(kp, kp, table, lens, w, 3, 1, posn, torch.tensor([5], dtype=torch.int32))
    # kept: slot 4 (recent), then 0 and 2 (0.5, ties to the lowest slots); slot 1 is dropped, 4 takes its place
    assert l2.tolist() == [3] and p2[0, 0, :3].tolist() == [0, 4, 2] and w2[0, 0, :3].tolist() == pytest.approx([0.5, 0.2, 0.5])
    assert k2[1, 0, :, 0].tolist() == [3.0, 1.0, 5.0] and k2[0, 0].equal(kp[0, 0])


def test_every_dependent_paged_launch_waits_and_releases():
    """The paged kernels are launched as programmatic dependents: each waits for the kernel before it and releases the
    one after it."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(la.__file__), "csrc")
    src = open(os.path.join(csrc, "la_paged.cuh")).read()
    api = open(os.path.join(csrc, "la_api.cu")).read()
    names = re.findall(r"\b(paged_\w+_kernel)\s*\(const", src)
    assert len(names) == 6, names
    for name in names:
        body = src[src.index(name + "(const"):]
        body = body[:body.index("\n}\n")]
        assert "grid_dependency_wait()" in body and "launch_dependents()" in body, name
        assert re.search(r"launch_pdl(_cluster)?\(" + name, api), name
        assert not re.search(name + r"[^;(]*<<<", api), name
