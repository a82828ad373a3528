"""The paged key/value cache on the GPU where it is easily wrong: infinite values, the weights that long sequences
receive, evictions by any number of blocks, and what the calls must leave alone.  Caches, the oracle's comparison and
its tolerances are those of test_paged_gpu.py."""
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


# -------------------------------------------------------- accumulated weights

@pytest.mark.parametrize("dtype,B,Hq,Hkv,dqk,dv,page,lens", [
    (BF16, 1, 8, 2, 128, 128, 64, [20000]), (BF16, 3, 4, 4, 64, 64, 24, [5000, 3, 9001]),
    (BF16, 1, 1, 1, 64, 64, 16, [30011]), (BF16, 1, 24, 1, 80, 48, 50, [6007]), (BF16, 2, 16, 2, 128, 128, 64, [12000, 1]),
    (BF16, 2, 128, 1, 64, 64, 32, [3000, 4097]), (BF16, 1, 5, 1, 33, 20, 10, [4099]),
    (BF16, 300, 2, 1, 64, 64, 16, [i % 37 for i in range(300)]), (F32, 2, 4, 2, 64, 64, 64, [7001, 640]),
    (F32, 1, 20, 1, 96, 64, 16, [5003])])
def test_weights_of_long_sequences(dtype, B, Hq, Hkv, dqk, dv, page, lens):
    """The weight that each slot receives, to a fraction of itself: units that cross ranges, groups of several units,
    the join's shares of the tiles; added to what is there, in place and apart.

    A head's weight is ex2(s - L), L = log2 of the row's sum.  s is off by (dqk + 6) u_s spread (the product, the scale
    and its rounding), and so is L, which adds (n + 16) u for the sum and u |L| for its own rounding; the difference is
    rounded, and ex2 is off by 4 u.  So a weight is off by rel times itself,
        rel = 2 (dqk + 6) u_s spread + u (n + 24 + 4 |lse| + 2 spread),
    and the sum over the group's g heads and what was there by (g + 1) u of what is added and u of the result."""
    mp, g, us = -(-max(lens) // page) + 1, Hq // Hkv, 4 * U if dtype == BF16 else U
    gen = torch.Generator(device=DEV).manual_seed(15)
    used = [-(-(n + 1) // page) for n in lens]
    table = torch.full((B, mp), -1, dtype=torch.int32)
    order = torch.randperm(sum(used), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    for b in range(B):
        table[b, :used[b]] = order[sum(used[:b]):sum(used[:b + 1])]
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dtype)
    kp, vp = rnd(sum(used), Hkv, page, dqk), rnd(sum(used), Hkv, page, dv)
    q, k, v = rnd(B, Hq, dqk), rnd(B, Hkv, dqk), rnd(B, Hkv, dv)
    w0 = torch.rand(B, Hkv, mp * page, generator=gen, device=DEV) * 0.01
    td, ld = to_dev(table, torch.tensor(lens, dtype=torch.int32))
    wo, w = torch.full_like(w0, -7.0), w0.clone()
    la.la_paged_decode_step(q, k, v, kp, vp, td, ld, weights=w0, weights_out=wo)
    la.la_paged_decode_step(q, k, v, kp, vp, td, ld, weights=w)
    sync()
    scale = 1 / math.sqrt(dqk)
    for b, n in enumerate(lens):
        t = torch.arange(n + 1, device=DEV)
        K = kp[td[b].long()[t // page], :, t % page].double().transpose(0, 1)
        qq = q[b].double().view(Hkv, g, dqk)
        s = qq @ K.transpose(1, 2) * scale
        lse = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - lse)
        spread = (qq.abs() @ K.abs().transpose(1, 2) * scale).amax(-1, keepdim=True)
        rel = 2 * (dqk + 6) * us * spread + U * (n + 1 + 24 + 4 * lse.abs() + 2 * spread)
        assert rel.max() < 0.02                       # so that weights which were never added fail
        old = w0[b].double()[:, :n + 1].clone()
        old[:, n] = 0
        added = p.sum(1)
        tol = (rel * p).sum(1) + (g + 1) * U * added + U * (old + added) + 1e-30
        got = wo[b].double()[:, :n + 1]
        assert ((got - old - added).abs() <= tol).all(), ((got - old - added).abs() / tol).max()
        assert (((got - old).sum(1) - g).abs() <= tol.sum(1)).all()
        assert torch.equal(wo[b, :, :n + 1], w[b, :, :n + 1])
        assert (wo[b, :, n + 1:] == -7).all() and torch.equal(w[b, :, n + 1:], w0[b, :, n + 1:])


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


def _int(t):
    return t.cpu().view(torch.int16 if t.dtype == BF16 else torch.int32)


@pytest.mark.parametrize("dtype,Hq,d", [(BF16, 4, 64), (BF16, 24, 128), (F32, 4, 40), (BF16, 6, 33)])
def test_new_token_on_a_bad_page_is_nowhere(dtype, Hq, d):
    """The pools, bit for bit, hold the other sequences' new tokens and nothing else new; the new slot's weight starts
    at 0 and receives none, and its position stays."""
    kp, vp, table, lens = cache(52, dtype, 3, 2, d, d, 16, 6, [40, 50, 60], used=[6] * 3)
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(3, h, d, generator=g).to(dtype) for h in (Hq, 2, 2))
    w = torch.rand(3, 2, 96, generator=g)
    posn = torch.randint(0, 99, (3, 2, 96), generator=g, dtype=torch.int32)
    pos = lens + 7
    own = table.clone()
    for bad in (-1, kp.shape[0], (1 << 31) - 1):
        table[2, 3] = bad                             # sequence 2 holds 60: its new token's page
        qd, kd, vd, kpd, vpd, td, ld, wd, pd, posd = to_dev(q, k, v, kp, vp, table, lens, w, posn, pos)
        y = la.la_paged_decode_step(qd, kd, vd, kpd, vpd, td, ld, weights=wd, positions=pd, pos=posd)
        base._reported()
        kr, vr, _, pr = orc.fill(k[:2, :, None], v[:2, :, None], kp, vp, own, lens, None, None, posn, pos)
        assert torch.equal(_int(kpd), _int(kr)) and torch.equal(_int(vpd), _int(vr))
        assert torch.equal(pd.cpu(), pr)
        l2 = lens.clone()
        l2[2] = 48
        ref = orc.decode(q[2:], None, None, kp, vp, own[2:], l2[2:], w[2:])
        got, want = wd.cpu()[2:].clone(), ref[2].clone()
        assert (got[..., 60] == 0).all() and torch.equal(got[..., 61:], w[2:, :, 61:])
        assert torch.equal(got[..., 48:60], w[2:, :, 48:60])
        want[..., 60] = 0
        check_step(dtype, 61, d, (y[2:], None, got), (ref[0], ref[1], want, *ref[3:]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_evict_more_recent_tokens_than_the_budget_moves_their_rows(dtype):
    """Positions that are not distinct, so that the recent tokens alone exceed the budget: rows, weights, positions and
    lens all follow the weights."""
    kp, vp, table, lens = cache(2, dtype, 2, 2, 24, 8, 16, 8, [64, 100], used=[8, 8])
    g = torch.Generator().manual_seed(3)
    w = torch.rand(2, 2, 128, generator=g)
    posn = torch.full((2, 2, 128), 9, dtype=torch.int32)
    posn[..., :5] = 0
    posn[..., 70:73] = 0
    pos = torch.tensor([10, 10], dtype=torch.int32)
    kr, vr, lr, wr, pr = orc.evict(kp, vp, table, lens, w, 20, 20, posn, pos)
    kpd, vpd, td, ld, wd, pd, posd = to_dev(kp, vp, table, lens, w, posn, pos)
    la.la_paged_evict(kpd, vpd, td, ld, wd, 20, recent=20, positions=pd, pos=posd)
    sync()
    assert torch.equal(_int(kpd), _int(kr)) and torch.equal(_int(vpd), _int(vr)) and ld.cpu().tolist() == [20, 20]
    assert torch.equal(wd.cpu()[..., :20], wr[..., :20]) and torch.equal(pd.cpu()[..., :20], pr[..., :20])
    assert torch.equal(wd.cpu()[..., 20:], w[..., 20:])


@pytest.mark.parametrize("bad", [-1, 101, 47, -(1 << 31), (1 << 31) - 1])
def test_bad_n_new_leaves_the_sequence_alone(bad):
    """n_new below 0, above N or past the table's room (96 slots, 50 held): that sequence stores nothing, the others
    are served."""
    kp, vp, table, lens = cache(53, BF16, 3, 2, 64, 64, 16, 6, [40, 50, 60], used=[6] * 3)
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(3, 2, 100, 64, generator=g).to(BF16) for _ in range(2))
    w = torch.rand(3, 2, 96, generator=g)
    posn = torch.randint(0, 99, (3, 2, 96), generator=g, dtype=torch.int32)
    pos = lens + 3
    kr, vr, wr, pr = orc.fill(k, v, kp, vp, table, lens, torch.tensor([30, 0, 36]), w, posn, pos)
    n_new = torch.tensor([30, bad, 36], dtype=torch.int32)
    kd, vd, kpd, vpd, td, ld, nd, wd, pd, posd = to_dev(k, v, kp, vp, table, lens, n_new, w, posn, pos)
    la.la_paged_cache_fill(kd, vd, kpd, vpd, td, ld, n_new=nd, weights=wd, positions=pd, pos=posd)
    base._reported()
    assert torch.equal(_int(kpd), _int(kr)) and torch.equal(_int(vpd), _int(vr))
    assert torch.equal(wd.cpu(), wr) and torch.equal(pd.cpu(), pr)


# ------------------------------------------------------------------- evictions

@pytest.mark.parametrize("B,Hkv,n,budget,recent,ties", [
    (20, 8, 20000, 3000, 100, True),        # more clusters of 2 than run at once
    (9, 8, 26000, 2000, 0, False),          # more clusters of 4
    (152, 1, 9000, 8000, 500, True),        # single blocks with long slices
    (8, 5, 9000, 4500, 64, False)])         # clusters of 4 for tables that could take 8
def test_evict_by_blocks_and_clusters(B, Hkv, n, budget, recent, ties):
    """The same answer whatever number of blocks shares a head."""
    base.test_evict_long(B, Hkv, n, budget, recent, ties)
