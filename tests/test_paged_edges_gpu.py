"""The paged key/value cache on the GPU where it is easily wrong: infinite values, and what the calls must leave
alone.  Caches, the oracle's comparison and its tolerances are those of test_paged_gpu.py."""
import math

import pytest
import torch

import causal_kernelized_sequence_b200 as la
import test_paged_gpu as base
from oracle import paged as orc
from test_paged_gpu import BF16, DEV, F32, U, cache, check_step, sync, to_dev

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- infinite values

def _pools_with(kp, vp, table, page, lens):
    """Infinities and NaN in the first five columns of the held values."""
    for b, n in enumerate(lens):
        def put(t, col, x):
            pg, r = orc.slot(table, page, b, t)
            vp[pg, :, r, col] = x
        if n == 0:
            continue
        put(0, 0, math.inf)
        put(n - 1, 1, -math.inf)
        put(0, 2, math.inf)
        put(n // 2, 2, -math.inf)
        put(n // 3, 3, math.nan)
        for t in range(0, n, 3):
            put(t, 4, -math.inf)


def _same_class(got, want):
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf])


@pytest.mark.parametrize("dtype,Hq,Hkv,dqk,dv,page", [
    (BF16, 4, 4, 64, 64, 16), (BF16, 8, 2, 128, 128, 64), (BF16, 8, 1, 64, 128, 32), (BF16, 16, 1, 128, 64, 64),
    (BF16, 9, 1, 128, 128, 8), (BF16, 20, 1, 64, 64, 64), (BF16, 16, 1, 64, 128, 12), (BF16, 40, 1, 128, 128, 24),
    (BF16, 14, 2, 72, 40, 24), (BF16, 5, 1, 33, 20, 10), (F32, 8, 2, 128, 128, 64), (F32, 5, 1, 33, 20, 7)])
def test_infinite_values(dtype, Hq, Hkv, dqk, dv, page):
    """An infinite value with a weight above 0 gives that infinity, values of both signs or a NaN give NaN, and the
    other columns are what they are without them.  One block per unit and ranges with a join."""
    lens_list = [0, 1, 2, 31, 32, 33, 127, 128, 129, 257]
    B, mp = len(lens_list), -(-300 // page)
    kp, vp, table, lens = cache(17, dtype, B, Hkv, dqk, dv, page, mp, lens_list)
    _pools_with(kp, vp, table, page, lens_list)
    q = torch.randn(B, Hq, dqk, generator=torch.Generator().manual_seed(3)).to(dtype)
    w = torch.zeros(B, Hkv, mp * page)
    ref = orc.decode(q, None, None, kp, vp, table, lens, w)
    qd, kpd, vpd, td, ld = to_dev(q, kp, vp, table, lens)
    for weights in (False, True):
        lse = torch.empty(B, Hq, device=DEV)
        wd = w.to(DEV)
        y = la.la_paged_decode_step(qd, None, None, kpd, vpd, td, ld, lse=lse, **({"weights": wd} if weights else {}))
        sync()
        _same_class(y.double().cpu()[..., :5], ref[0][..., :5])
        check_step(dtype, 257, dqk, (y[..., 5:], lse, wd.cpu() if weights else None),
                   (ref[0][..., 5:], ref[1], ref[2] if weights else None, ref[3][..., 5:], ref[4]))


@pytest.mark.parametrize("Hq", [1, 8, 9, 16])
def test_infinite_value_of_the_new_token(Hq):
    """The new token's own value, alone and behind others; a long sequence whose parts are joined."""
    d, page, lens_list = 64, 16, [0, 1, 40, 5000]
    B, mp = len(lens_list), 320
    kp, vp, table, lens = cache(23, BF16, B, 1, d, d, page, mp, lens_list)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(B, h, d, generator=g).to(BF16) for h in (Hq, 1, 1))
    v[..., 0], v[..., 1] = math.inf, -math.inf
    ref = orc.decode(q, k, v, kp, vp, table, lens)
    qd, kd, vd, kpd, vpd, td, ld = to_dev(q, k, v, kp, vp, table, lens)
    lse = torch.empty(B, Hq, device=DEV)
    y = la.la_paged_decode_step(qd, kd, vd, kpd, vpd, td, ld, lse=lse)
    sync()
    assert (y[..., 0] == math.inf).all() and (y[..., 1] == -math.inf).all()
    check_step(BF16, 5001, d, (y[..., 2:], lse, None), (ref[0][..., 2:], ref[1], None, ref[3][..., 2:], ref[4]))


# ---------------------------------------------------- what a call leaves alone

def test_append_from_the_longest_padded_batch():
    """N = 2^31 - 1 tokens of padding, of which n_new count: both heads' first tokens are stored and nothing else."""
    N, Hkv, page, held, new = (1 << 31) - 1, 2, 16, 5, 70
    k = torch.empty(1, Hkv, N, 1, dtype=BF16, device=DEV)
    v = torch.empty(1, Hkv, N, 1, dtype=BF16, device=DEV)
    for i, t in enumerate((k, v)):
        t[:, :, :new] = torch.randn(1, Hkv, new, 1, generator=torch.Generator().manual_seed(i)).to(BF16).to(DEV)
    kp, vp = (torch.randn(8, Hkv, page, 1, generator=torch.Generator().manual_seed(9 + i)).to(BF16) for i in range(2))
    table = torch.tensor([[3, 0, 6, 1, 5, -1]], dtype=torch.int32)
    lens, n_new = torch.tensor([held], dtype=torch.int32), torch.tensor([new], dtype=torch.int32)
    kr, vr, _, _ = orc.fill(k[:, :, :new].cpu(), v[:, :, :new].cpu(), kp, vp, table, lens, n_new)
    kpd, vpd, td, ld, nd = to_dev(kp, vp, table, lens, n_new)
    la.la_paged_cache_fill(k, v, kpd, vpd, td, ld, n_new=nd)
    sync()
    assert torch.equal(kpd.cpu(), kr) and torch.equal(vpd.cpu(), vr)


# ------------------------------------------------------------------- evictions

@pytest.mark.parametrize("B,Hkv,n,budget,recent,ties", [
    (20, 8, 20000, 3000, 100, True),        # more clusters of 2 than run at once
    (9, 8, 26000, 2000, 0, False),          # more clusters of 4
    (152, 1, 9000, 8000, 500, True),        # single blocks with long slices
    (8, 5, 9000, 4500, 64, False)])         # clusters of 4 for tables that could take 8
def test_evict_by_blocks_and_clusters(B, Hkv, n, budget, recent, ties):
    """The same answer whatever number of blocks shares a head."""
    base.test_evict_long(B, Hkv, n, budget, recent, ties)
