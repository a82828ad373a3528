"""The paged key/value cache on the GPU against the fp64 oracle: appending
tokens, one-token attention over any length, eviction, and the three together
as a generation loop uses them.

Tolerances.  u = 2^-24 is half a step of fp32.  A score is a sum of dqk
products whose fp32 error is at most (dqk + 4) u_s * spread, spread = sum_i
|q_i k_i| / sqrt(dqk), with u_s = u for fp32 FMA and 4 u where a tensor core
adds the products (it may truncate, and align a block of them to the largest).
With that error ds, a softmax weight is off by a factor within 1 +- 2 ds, plus
(n + 16) u for the sum and the exponentials; where weights enter a tensor core
as two bf16 halves, each is off by at most 2^-16 more.  y adds the rounding to
its own type, eps / 2.
"""
import math

import pytest
import torch

import causal_kernelized_sequence_b200 as la
from oracle import paged as orc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def cache(seed, dtype, B, Hkv, dqk, dv, page, max_pages, lens, used=None):
    """A cache whose sequences hold `lens` slots, in shuffled pages; every row that
    no slot below lens uses holds NaN, and unused table entries -1."""
    g = torch.Generator().manual_seed(seed)
    used = [max(1, -(-(n + 1) // page)) for n in lens] if used is None else used
    P = sum(used) + 2
    order = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    at = 0
    kp = torch.full((P, Hkv, page, dqk), float("nan"), dtype=dtype)
    vp = torch.full((P, Hkv, page, dv), float("nan"), dtype=dtype)
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        for t in range(lens[b]):
            pg, r = orc.slot(table, page, b, t)
            kp[pg, :, r] = torch.randn(Hkv, dqk, generator=g).to(dtype)
            vp[pg, :, r] = torch.randn(Hkv, dv, generator=g).to(dtype)
    return kp, vp, table, torch.tensor(lens, dtype=torch.int32)


def to_dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def check_step(dtype, n_max, dqk, got, ref):
    y, lse, w = got
    yr, lser, wr, size, spread = ref
    tc = dtype == BF16
    ds = (dqk + 4) * (4 * U if tc else U) * spread
    rel = 2 * ds + (n_max + 16) * U + (2.0 ** -15 if tc else 0)
    half = torch.finfo(dtype).eps / 2
    tol = half * yr.abs() * (1 + half) + rel[..., None] * size + 1e-30
    bad = (y.double().cpu() - yr).abs() - tol
    assert bad.max() <= 0, (bad.max(), (y.double().cpu() - yr).abs().max())
    if lse is not None:
        fin = torch.isfinite(lser)
        l = lse.double().cpu()
        assert torch.equal(torch.isfinite(l), fin) and torch.equal(l[~fin], lser[~fin])
        assert ((l - lser).abs()[fin] <= (ds + (n_max + 16) * U + 2 * U * lser.abs())[fin]).all()
    if w is not None:
        g = y.shape[1] // wr.shape[1]
        r = rel.view(y.shape[0], wr.shape[1], g).amax(2)[..., None]
        assert ((w.double().cpu() - wr).abs() <= (r + 4 * U) * (g + wr.abs()) * 1.0).all()


def sync():
    torch.cuda.synchronize()
    la.la_get_device_status()


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 130, 257]
SHAPES = [  # dtype, Hq, Hkv, dqk, dv, page
    (BF16, 4, 4, 64, 64, 16), (BF16, 8, 2, 128, 128, 64), (BF16, 8, 1, 64, 128, 32), (BF16, 16, 1, 128, 64, 64),
    (BF16, 9, 1, 128, 128, 8), (BF16, 20, 1, 64, 64, 64), (BF16, 40, 1, 128, 128, 24), (BF16, 3, 3, 80, 96, 7),
    (BF16, 14, 2, 72, 40, 24), (BF16, 6, 2, 16, 64, 1), (BF16, 5, 1, 33, 20, 10), (BF16, 2, 2, 1, 1, 3),
    (BF16, 7, 1, 8, 8, 100), (BF16, 1, 1, 127, 5, 16),
    (F32, 4, 4, 64, 64, 16), (F32, 8, 2, 128, 128, 64), (F32, 20, 1, 64, 32, 8), (F32, 6, 3, 24, 40, 10),
    (F32, 5, 1, 33, 20, 7), (F32, 1, 1, 1, 128, 1), (F32, 17, 1, 128, 128, 128),
    (BF16, 128, 1, 64, 64, 16), (F32, 65, 1, 32, 40, 4), (BF16, 6, 2, 65, 127, 48), (F32, 9, 3, 127, 66, 2),
    (F32, 2, 1, 4, 8, 16), (F32, 14, 2, 128, 64, 256), (F32, 5, 1, 64, 64, 12), (BF16, 12, 1, 96, 24, 128),
    (F32, 8, 1, 65, 33, 32), (BF16, 10, 1, 128, 127, 5), (BF16, 64, 8, 64, 64, 200),
]


@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("dtype,Hq,Hkv,dqk,dv,page", SHAPES)
def test_decode_step(dtype, Hq, Hkv, dqk, dv, page, new):
    """Lengths around every tile border in one batch, the empty cache among them, with NaN in every slot that is
    not held; with and without weights; the new token lands in its slot and nothing else changes."""
    B, mp = len(LENS), -(-300 // page)
    kp, vp, table, lens = cache(7, dtype, B, Hkv, dqk, dv, page, mp, LENS)
    g = torch.Generator().manual_seed(11)
    q = torch.randn(B, Hq, dqk, generator=g).to(dtype)
    k, v = (torch.randn(B, Hkv, d, generator=g).to(dtype) if new else None for d in (dqk, dv))
    cap = mp * page
    w = torch.rand(B, Hkv, cap, generator=g)
    posn = torch.randint(0, 99, (B, Hkv, cap), generator=g, dtype=torch.int32)
    pos = lens + 5
    ref = orc.decode(q, k, v, kp, vp, table, lens, w)
    for weights in (False, True):
        qd, kd, vd, kpd, vpd, td, ld, wd, pd, posd = to_dev(q, k, v, kp, vp, table, lens, w, posn, pos)
        lse = torch.full((B, Hq), 3.0, device=DEV)
        wo = torch.full_like(wd, -7.0)
        more = {"weights": wd, "weights_out": wo} if weights else {}
        if new:
            more.update(positions=pd, pos=posd)
        y = la.la_paged_decode_step(qd, kd, vd, kpd, vpd, td, ld, lse=lse, **more)
        sync()
        got_w = None
        if weights:
            n = (lens + (1 if new else 0))[:, None, None]
            held = (torch.arange(cap) < n).expand(B, Hkv, cap)
            assert (wo.cpu()[~held] == -7.0).all() and torch.equal(wd.cpu(), w)
            got_w = torch.where(held, wo.cpu(), w)
            ref_w = torch.where(held, ref[2], w.double())
        check_step(dtype, 258, dqk, (y, lse, got_w), (ref[0], ref[1], ref_w if weights else None, ref[3], ref[4]))
        # pages: the new token and nothing else; bit for bit, NaN included
        kr, vr, _, pr = (kp, vp, None, posn) if not new else orc.fill(
            k[:, :, None], v[:, :, None], kp, vp, table, lens, positions=posn, pos=pos)
        as_int = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(kpd.cpu().view(as_int), kr.view(as_int)) and torch.equal(vpd.cpu().view(as_int), vr.view(as_int))
        assert torch.equal(pd.cpu(), pr)
        if weights:   # in place gives the same bits
            wd2 = w.to(DEV)
            y2 = la.la_paged_decode_step(qd, kd, vd, kpd, vpd, td, ld, weights=wd2)
            sync()
            assert torch.equal(y2, y) and torch.equal(wd2.cpu()[held], wo.cpu()[held])
            assert torch.equal(wd2.cpu()[~held], w[~held])


@pytest.mark.parametrize("dtype,B,Hq,Hkv,dqk,dv,page,lens", [
    (BF16, 1, 8, 2, 128, 128, 64, [20000]), (BF16, 3, 4, 4, 64, 64, 24, [5000, 3, 9001]),
    (BF16, 1, 1, 1, 64, 64, 16, [30011]), (F32, 2, 4, 2, 64, 64, 64, [7001, 640]), (BF16, 1, 24, 1, 80, 48, 50, [6007]),
    (BF16, 300, 2, 1, 64, 64, 16, [i % 37 for i in range(300)])])
def test_decode_long(dtype, B, Hq, Hkv, dqk, dv, page, lens):
    """Long sequences, split across many blocks and joined, and more sequences than threads in a block."""
    mp = -(-max(lens) // page) + 1
    g = torch.Generator(device=DEV).manual_seed(5)
    used = [-(-(n + 1) // page) for n in lens]
    table = torch.full((B, mp), -1, dtype=torch.int32)
    order = torch.randperm(sum(used), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    for b in range(B):
        table[b, :used[b]] = order[sum(used[:b]):sum(used[:b + 1])]
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)
    kp, vp = rnd(sum(used), Hkv, page, dqk), rnd(sum(used), Hkv, page, dv)
    q, k, v = rnd(B, Hq, dqk), rnd(B, Hkv, dqk), rnd(B, Hkv, dv)
    w = torch.zeros(B, Hkv, mp * page, device=DEV)
    td, ld = to_dev(table, torch.tensor(lens, dtype=torch.int32))
    lse = torch.empty(B, Hq, device=DEV)
    y = la.la_paged_decode_step(q, k, v, kp, vp, td, ld, lse=lse, weights=w)
    sync()
    # the formulas in fp64, sequence by sequence
    scale = 1 / math.sqrt(dqk)
    for b, n in enumerate(lens):
        t = torch.arange(n + 1, device=DEV)
        pg = td[b].long()[t // page]
        K, V = kp[pg, :, t % page].double().transpose(0, 1), vp[pg, :, t % page].double().transpose(0, 1)
        qq = q[b].double().view(Hkv, Hq // Hkv, dqk)
        s = qq @ K.transpose(1, 2) * scale
        p = torch.softmax(s, -1)
        spread = (qq.abs() @ K.abs().transpose(1, 2) * scale).amax(-1).view(1, Hq)
        ref = ((p @ V).view(1, Hq, dv), torch.logsumexp(s, -1).view(1, Hq), p.sum(1)[None],
               (p @ V.abs()).view(1, Hq, dv), spread)
        check_step(dtype, n + 1, dqk, (y[b:b + 1], lse[b:b + 1], w[b:b + 1, :, :n + 1]), [r.cpu() for r in ref])
        assert (w[b, :, n + 1:] == 0).all()


def test_decode_extreme_scores():
    """Scores of -inf and +-large beside ordinary ones: rows stay finite where softmax is, NaN where it is not."""
    for dtype, d in ((BF16, 64), (F32, 48)):
        n = 200
        kp, vp, table, lens = cache(3, dtype, 1, 1, d, d, 16, 13, [n])
        kp = torch.nan_to_num(kp)
        for t in range(0, 190):                    # a whole first block of -inf scores
            pg, r = orc.slot(table, 16, 0, t)
            kp[pg, 0, r] = 0
            kp[pg, 0, r, 0] = -math.inf
        q = torch.zeros(1, 2, d, dtype=dtype)
        q[0, :, 0] = 1.0                           # scores -inf for t < 190, k_0 / sqrt(d) after
        q[0, 1, 1] = 300.0
        ref = orc.decode(q, None, None, torch.nan_to_num(kp, neginf=-1e30), vp, table, lens)
        qd, kpd, vpd, td, ld = to_dev(q, kp, vp, table, lens)
        # (0 * -inf is NaN for the other coordinates only if q has zeros there: they multiply zeros, not the inf)
        lse = torch.empty(1, 2, device=DEV)
        y = la.la_paged_decode_step(qd, None, None, kpd, vpd, td, ld, lse=lse)
        sync()
        assert torch.isfinite(y.float()).all() and torch.isfinite(lse).all()
        # two products per score, |s| < 150: the score's error is below 8 * 2^-22 * 150 < 2^-11.7, a weight's below 2^-10
        tol = torch.finfo(dtype).eps / 2 * ref[0].abs() + (2 ** -10) * ref[3]
        assert ((y.double().cpu() - ref[0]).abs() <= tol).all()
        # a NaN key reaches every output of its head and nothing else
        pg, r = orc.slot(table, 16, 0, 195)
        kp[pg, 0, r, 3] = math.nan
        y = la.la_paged_decode_step(qd, None, None, kp.to(DEV), vpd, td, ld)
        sync()
        assert torch.isnan(y.float()).all()


def test_shared_pages_and_steps_on_shared_prefix():
    """Two sequences whose tables share pages read the same rows."""
    kp, vp, table, lens = cache(4, BF16, 2, 2, 64, 64, 16, 8, [64, 64])
    table[1, :3] = table[0, :3]
    q = torch.randn(1, 4, 64).to(BF16).expand(2, 4, 64).contiguous()
    ref = orc.decode(q, None, None, kp, vp, table, lens)
    y = la.la_paged_decode_step(*to_dev(q), None, None, *to_dev(kp, vp, table, lens))
    sync()
    check_step(BF16, 64, 64, (y, None, None), (*ref[:2], None, *ref[3:]))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the last pages are read and written."""
    P, Hkv, page, d = 4200, 64, 64, 128            # 2.2e9 elements each
    kp = torch.empty(P, Hkv, page, d, dtype=BF16, device=DEV)
    vp = torch.empty(P, Hkv, page, d, dtype=BF16, device=DEV)
    table = torch.tensor([[P - 1, 0, P - 2, -1]], dtype=torch.int32)
    N = 150
    k, v = (torch.randn(1, Hkv, N, d, device=DEV).to(BF16) for _ in range(2))
    td, ld = to_dev(table, torch.zeros(1, dtype=torch.int32))
    la.la_paged_cache_fill(k, v, kp, vp, td, ld)
    q = torch.randn(1, Hkv, d, device=DEV).to(BF16)
    ld += N - 1
    y = la.la_paged_decode_step(q, k[:, :, -1].contiguous(), v[:, :, -1].contiguous(), kp, vp, td, ld)
    sync()
    assert torch.equal(kp[P - 1, :, :64], k[0, :, :64]) and torch.equal(vp[P - 2, :, :22], v[0, :, 128:])
    s = (q[0].double()[:, None] * k[0].double()).sum(-1) / math.sqrt(d)
    p = torch.softmax(s, -1)
    ref = (p[..., None] * v[0].double()).sum(1)
    size = (p[..., None] * v[0].double().abs()).sum(1)
    assert ((y[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -9 * size).all()


@pytest.mark.parametrize("dtype,Hkv,N,dqk,dv,page", [
    (BF16, 2, 200, 64, 64, 16), (F32, 3, 77, 33, 20, 7), (BF16, 1, 1, 8, 128, 1), (BF16, 4, 65, 72, 5, 100),
    (F32, 1, 64, 4, 4, 64), (BF16, 2, 129, 128, 128, 64)])
def test_cache_fill(dtype, Hkv, N, dqk, dv, page):
    """Padded batches appended to empty and part-filled caches; nothing else changes, bit for bit."""
    held = [0, 3, 40, 0]
    mp = -(-(N + 41) // page)
    kp, vp, table, lens = cache(9, dtype, 4, Hkv, dqk, dv, page, mp, held, used=[mp] * 4)
    g = torch.Generator().manual_seed(2)
    k, v = torch.randn(4, Hkv, N, dqk, generator=g).to(dtype), torch.randn(4, Hkv, N, dv, generator=g).to(dtype)
    w = torch.rand(4, Hkv, mp * page, generator=g)
    posn = torch.randint(0, 99, w.shape, generator=g, dtype=torch.int32)
    pos = lens + 11
    as_int = torch.int16 if dtype == BF16 else torch.int32
    for n_new in (None, torch.tensor([N, 1, N // 2, 0], dtype=torch.int32)):
        kr, vr, wr, pr = orc.fill(k, v, kp, vp, table, lens, n_new, w, posn, pos)
        kd, vd, kpd, vpd, td, ld, nd, wd, pd, posd = to_dev(k, v, kp, vp, table, lens, n_new, w, posn, pos)
        la.la_paged_cache_fill(kd, vd, kpd, vpd, td, ld, n_new=nd, weights=wd, positions=pd, pos=posd)
        sync()
        assert torch.equal(kpd.cpu().view(as_int), kr.view(as_int)) and torch.equal(vpd.cpu().view(as_int), vr.view(as_int))
        assert torch.equal(wd.cpu(), wr) and torch.equal(pd.cpu(), pr)


EVICT = [  # dtype, Hkv, dqk, dv, page, lens, budget, recent
    (BF16, 2, 64, 64, 16, [100, 64, 65, 0, 1], 64, 16), (F32, 3, 24, 40, 10, [90, 33, 34, 70, 5], 33, 7),
    (BF16, 1, 33, 20, 7, [600, 100, 1], 1, 0), (BF16, 1, 8, 8, 1, [50, 49], 48, 48), (F32, 1, 4, 4, 64, [1500, 20], 700, 0),
    (BF16, 2, 128, 128, 64, [2500, 3], 512, 100), (BF16, 4, 16, 64, 100, [300, 250], 299, 20)]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("dtype,Hkv,dqk,dv,page,lens,budget,recent", EVICT)
def test_evict(dtype, Hkv, dqk, dv, page, lens, budget, recent, ties):
    """Exact agreement with the oracle: which slots stay and where they go, in place and into other buffers; with
    equal, negative, infinite and NaN weights."""
    B = len(lens)
    mp = -(-max(lens) // page)
    kp, vp, table, lens = cache(21, dtype, B, Hkv, dqk, dv, page, mp, lens, used=[mp] * B)
    g = torch.Generator().manual_seed(8)
    cap = mp * page
    w = torch.rand(B, Hkv, cap, generator=g) ** 3
    if ties:
        w = (w * 4).floor() - 1.0
        w[..., ::13] = -0.0
        w[..., 1::13] = math.inf
        w[..., 2::13] = math.nan
        w[..., 3::13] = -math.inf
    posn = torch.stack([torch.randperm(cap, generator=g) for _ in range(B * Hkv)]).view(B, Hkv, cap).int() + 3
    pos = torch.full((B,), cap + 3, dtype=torch.int32)
    more = {"recent": recent, "positions": posn, "pos": pos}
    kr, vr, lr, wr, pr = orc.evict(kp, vp, table, lens, w, budget, **more)
    as_int = torch.int16 if dtype == BF16 else torch.int32
    held = (torch.arange(cap) < lr[:, None, None]).expand(B, Hkv, cap)
    bits = lambda t: t.view(torch.int32)
    for place in (True, False):
        kpd, vpd, td, ld, wd, pd, posd = to_dev(kp, vp, table, lens, w, posn, pos)
        out = {} if place else {"lens_out": torch.full_like(ld, -9), "weights_out": torch.full_like(wd, -9),
                                "positions_out": torch.full_like(pd, -9)}
        lo = la.la_paged_evict(kpd, vpd, td, ld, wd, budget, recent=recent, positions=pd, pos=posd, **out)
        sync()
        wo, po = out.get("weights_out", wd).cpu(), out.get("positions_out", pd).cpu()
        assert torch.equal(lo.cpu(), lr)
        assert torch.equal(bits(wo)[held], bits(wr)[held]) and torch.equal(po[held], pr[held])
        if place:
            assert lo is ld and torch.equal(bits(wo)[~held], bits(w)[~held])
        else:
            assert (wo[~held] == -9).all() and torch.equal(ld.cpu(), lens) and torch.equal(bits(wd.cpu()), bits(w))
        assert torch.equal(kpd.cpu().view(as_int), kr.view(as_int)) and torch.equal(vpd.cpu().view(as_int), vr.view(as_int))
    if not recent:   # without the positions
        kpd, vpd, td, ld, wd = to_dev(kp, vp, table, lens, w)
        la.la_paged_evict(kpd, vpd, td, ld, wd, budget)
        sync()
        assert torch.equal(kpd.cpu().view(as_int), kr.view(as_int)) and torch.equal(ld.cpu(), lr)


@pytest.mark.parametrize("B,Hkv,n,budget,recent,ties", [
    (1, 1, 110000, 30000, 1000, False),     # a cluster whose slices are too long for the keys to be kept
    (300, 1, 13000, 500, 64, True),         # the same for single blocks; more warps' rounds than one
    (40, 4, 3000, 2900, 0, True), (5, 3, 9000, 4000, 4000, False)])
def test_evict_long(B, Hkv, n, budget, recent, ties):
    """Against a stable sort of every head's slots."""
    page, d = 64, 8
    mp = -(-n // page)
    g = torch.Generator(device=DEV).manual_seed(6)
    kp, vp = (torch.randn(B * mp, Hkv, page, d, generator=g, device=DEV).to(BF16) for _ in range(2))
    table = torch.randperm(B * mp, generator=g, device=DEV).view(B, mp).int()
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    lens[1:][-1:] = budget + 1
    w = torch.rand(B, Hkv, mp * page, generator=g, device=DEV)
    if ties:
        w = (w * 9).floor()
    posn = torch.rand(B, Hkv, mp * page, generator=g, device=DEV).argsort(-1).int()
    pos = torch.full((B,), mp * page, dtype=torch.int32, device=DEV)
    t = torch.arange(n, device=DEV).expand(B, Hkv, n)
    live = t < lens[:, None, None]
    key = torch.where(posn[..., :n] >= mp * page - recent, math.inf, w[..., :n]) if recent else w[..., :n]
    order = torch.where(live, key, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(live).scatter_(2, order[..., :budget], True) & live
    # the slot that each one below the budget takes: itself, or the next mover
    src = t[..., :budget].clone()
    hole, mover = (~keep & live)[..., :budget], keep & (t >= budget)
    src[hole] = t[mover]                    # both in (b, h, ascending slot) order, equally many per head
    assert torch.equal(hole.sum(-1), mover.sum(-1))
    flat = lambda slots: ((table.long()[:, None].expand(B, Hkv, mp).gather(2, slots // page) * Hkv
                           + torch.arange(Hkv, device=DEV)[None, :, None]) * page + slots % page)
    to, frm = flat(t[..., :budget].contiguous()), flat(src)
    kr, vr = kp.clone(), vp.clone()
    kr.view(-1, d)[to], vr.view(-1, d)[to] = kp.view(-1, d)[frm], vp.view(-1, d)[frm]
    w0, p0 = w.clone(), posn.clone()
    la.la_paged_evict(kp, vp, table, lens, w, budget, recent=recent, positions=posn, pos=pos)
    sync()
    assert (lens == budget).all()
    assert torch.equal(w[..., :budget], w0.gather(2, src)) and torch.equal(posn[..., :budget], p0.gather(2, src))
    assert torch.equal(w[..., budget:], w0[..., budget:])
    assert torch.equal(kp, kr) and torch.equal(vp, vr)


def test_evict_recent_alone_exceed_the_budget():
    """Every token recent (positions not distinct): the weights decide among them."""
    kp, vp, table, lens = cache(2, BF16, 1, 1, 8, 8, 16, 4, [64], used=[4])
    w = torch.rand(1, 1, 64, generator=torch.Generator().manual_seed(3))
    posn = torch.full((1, 1, 64), 9, dtype=torch.int32)
    posn[..., :5] = 0
    pos = torch.tensor([10], dtype=torch.int32)
    ref = orc.evict(kp, vp, table, lens, w, 20, 20, posn, pos)
    kpd, vpd, td, ld, wd, pd, posd = to_dev(kp, vp, table, lens, w, posn, pos)
    la.la_paged_evict(kpd, vpd, td, ld, wd, 20, recent=20, positions=pd, pos=posd)
    sync()
    assert torch.equal(wd.cpu()[..., :20], ref[3][..., :20]) and torch.equal(pd.cpu()[..., :20], ref[4][..., :20])


@pytest.mark.parametrize("dtype,Hq,Hkv,d,page", [(BF16, 8, 2, 64, 16), (F32, 3, 3, 40, 10)])
def test_generation_with_a_bounded_cache(dtype, Hq, Hkv, d, page):
    """The operators as a generation loop uses them: prompts of different lengths are appended, steps add tokens and
    weights, and every time a sequence may pass the budget the cache is cut back.  Every step against the oracle, whose
    state is carried along; an eviction is decided on the library's own weights and then compared exactly."""
    B, budget, recent, steps, prompt = 3, 64, 16, 40, [50, 7, 61]
    mp = -(-(budget + 16) // page)
    kp, vp, table, lens = cache(31, dtype, B, Hkv, d, d, page, mp, [0] * B, used=[mp] * B)
    g = torch.Generator().manual_seed(77)
    k, v = (torch.randn(B, Hkv, max(prompt), d, generator=g).to(dtype) for _ in range(2))
    w = torch.full((B, Hkv, mp * page), math.nan)
    posn = torch.full((B, Hkv, mp * page), -1, dtype=torch.int32)
    pos, n_new = lens.clone(), torch.tensor(prompt, dtype=torch.int32)
    kd, vd, kpd, vpd, td, ld, wd, pd, posd, nd = to_dev(k, v, kp, vp, table, lens, w, posn, pos, n_new)
    la.la_paged_cache_fill(kd, vd, kpd, vpd, td, ld, n_new=nd, weights=wd, positions=pd, pos=posd)
    ld += nd
    posd += nd
    kp, vp, w, posn = orc.fill(k, v, kp, vp, table, lens, n_new, w, posn, pos)
    lens, pos = lens + n_new, pos + n_new
    evicted = 0
    for s in range(steps):
        q, kn, vn = (torch.randn(B, h, d, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        q = q * 3
        ref = orc.decode(q, kn, vn, kp, vp, table, lens, w)
        qd, kd, vd = to_dev(q, kn, vn)
        lse = torch.empty(B, Hq, device=DEV)
        y = la.la_paged_decode_step(qd, kd, vd, kpd, vpd, td, ld, lse=lse, weights=wd, positions=pd, pos=posd)
        sync()
        kp, vp, _, posn = orc.fill(kn[:, :, None], vn[:, :, None], kp, vp, table, lens, None, None, posn, pos)
        held = (torch.arange(mp * page) <= lens[:, None, None]).expand_as(w)
        got_w, ref_w = (torch.where(held, t.cpu().double(), 0.0) for t in (wd, ref[2]))
        check_step(dtype, int(lens.max()) + 1, d, (y, lse, got_w), (*ref[:2], ref_w, *ref[3:]))
        w = wd.cpu()                                # carried on as the library has them
        lens, pos = lens + 1, pos + 1
        ld += 1
        posd += 1
        if int(lens.max()) >= budget + 8:
            kp, vp, lens, w, posn = orc.evict(kp, vp, table, lens, w, budget, recent, posn, pos)
            la.la_paged_evict(kpd, vpd, td, ld, wd, budget, recent=recent, positions=pd, pos=posd)
            sync()
            held = (torch.arange(mp * page) < lens[:, None, None]).expand_as(w)
            assert torch.equal(ld.cpu(), lens) and torch.equal(pd.cpu()[held], posn[held])
            assert torch.equal(wd.cpu()[held], w[held])
            evicted += 1
    assert evicted >= 3


def test_captured_step_follows_the_lengths():
    """A captured step replayed while lens advances gives the eager steps' bits (the grid does not depend on lens)."""
    B, Hq, Hkv, d, page, mp = 3, 8, 2, 64, 16, 40
    start = [0, 100, 500]
    kp, vp, table, lens = cache(41, BF16, B, Hkv, d, d, page, mp, start, used=[mp] * B)
    g = torch.Generator().manual_seed(4)
    toks = [[torch.randn(B, h, d, generator=g).to(BF16).to(DEV) for h in (Hq, Hkv, Hkv)] for _ in range(6)]
    runs = []
    for captured in (False, True):
        kpd, vpd, td, ld = to_dev(kp, vp, table, lens)
        wd = torch.zeros(B, Hkv, mp * page, device=DEV)
        ws = torch.empty(la.la_paged_decode_workspace_bytes(B, Hq, Hkv, d, d, page, mp, True, la.LA_BF16) + 16,
                         dtype=torch.uint8, device=DEV)
        q, k, v = (t.clone() for t in toks[0])
        y = torch.empty(B, Hq, d, dtype=BF16, device=DEV)

        def step():
            la.la_paged_decode_step(q, k, v, kpd, vpd, td, ld, y=y, weights=wd, workspace=ws)
            ld.add_(1)
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()                              # warm-up
            torch.cuda.current_stream().wait_stream(side)
            sync()
            kpd.copy_(kp.to(DEV)); vpd.copy_(vp.to(DEV)); ld.copy_(lens.to(DEV)); wd.zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        out = []
        for t in toks:
            for dst, src in zip((q, k, v), t):
                dst.copy_(src)
            graph.replay() if captured else step()
            out.append(y.clone())
        sync()
        runs.append((out, wd, ld))
    for a, b in zip(runs[0][0], runs[1][0]):
        assert torch.equal(a, b)
    assert torch.equal(runs[0][1], runs[1][1]) and torch.equal(runs[0][2], runs[1][2])


def test_captured_append_step_and_evict():
    """One graph of an append, a step and an eviction in place, replayed: the eager calls' bits."""
    B, Hq, Hkv, d, page, mp, budget = 2, 4, 2, 64, 16, 30, 300
    g = torch.Generator().manual_seed(14)
    kp, vp, table, lens = cache(43, BF16, B, Hkv, d, d, page, mp, [290, 20], used=[mp] * B)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF16).to(DEV)
    kf, vf = rnd(B, Hkv, 40, d), rnd(B, Hkv, 40, d)
    q, k, v = rnd(B, Hq, d), rnd(B, Hkv, d), rnd(B, Hkv, d)
    res = []
    for captured in (False, True):
        kpd, vpd, td, ld = to_dev(kp, vp, table, lens)
        w = torch.rand(B, Hkv, mp * page, generator=torch.Generator().manual_seed(1)).to(DEV)
        ps = torch.arange(mp * page, dtype=torch.int32, device=DEV).expand(B, Hkv, -1).contiguous()
        pos, y = ld.clone(), torch.empty(B, Hq, d, dtype=BF16, device=DEV)

        def steps():
            la.la_paged_cache_fill(kf, vf, kpd, vpd, td, ld, weights=w, positions=ps, pos=pos)
            ld.add_(40)
            pos.add_(40)
            la.la_paged_decode_step(q, k, v, kpd, vpd, td, ld, y=y, weights=w, positions=ps, pos=pos)
            ld.add_(1)
            pos.add_(1)
            la.la_paged_evict(kpd, vpd, td, ld, w, budget, recent=32, positions=ps, pos=pos)
        if captured:
            keep = [x.clone() for x in (kpd, vpd, ld, w, ps, pos)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                steps()
            torch.cuda.current_stream().wait_stream(side)
            sync()
            for x, c in zip((kpd, vpd, ld, w, ps, pos), keep):
                x.copy_(c)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                steps()
        for _ in range(8):
            graph.replay() if captured else steps()
        sync()
        res.append([x.cpu() for x in (kpd.view(torch.int16), vpd.view(torch.int16), ld, w, ps, pos, y)])
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert res[0][2].tolist() == [300, 300]


def test_steps_on_two_streams_with_their_own_workspaces():
    """Two steps in flight at once on different caches give what they give alone."""
    d, page, mp, Hq, Hkv = 64, 16, 260, 4, 2
    st = []
    for seed in (1, 2):
        kp, vp, table, lens = to_dev(*cache(seed, BF16, 2, Hkv, d, d, page, mp, [4000, 900]))
        q = torch.randn(2, Hq, d, generator=torch.Generator().manual_seed(seed)).to(BF16).to(DEV)
        st.append((q, None, None, kp, vp, table, lens))
    alone = [la.la_paged_decode_step(*a) for a in st]
    sync()
    streams = [torch.cuda.Stream() for _ in st]
    outs = [[], []]
    for _ in range(10):
        for i, (s, a) in enumerate(zip(streams, st)):
            with torch.cuda.stream(s):
                outs[i].append(la.la_paged_decode_step(*a))
    sync()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


def _bad_state():
    kp, vp, table, lens = cache(51, BF16, 3, 2, 64, 64, 16, 6, [40, 50, 60], used=[6] * 3)
    return to_dev(torch.nan_to_num(kp), torch.nan_to_num(vp), table, lens)


def _reported():
    with pytest.raises(la.LAError) as e:
        la.la_get_device_status()
    assert e.value.status == 5
    la.la_get_device_status()


@pytest.mark.parametrize("bad", [-1, 96, 97, 1 << 30, (1 << 31) - 1, -(1 << 31)])
def test_bad_length_leaves_the_sequence_alone(bad):
    """A length below zero or without room for the new token: that sequence writes nothing, the others are served."""
    kp, vp, table, lens = _bad_state()
    q, k, v = (torch.randn(3, h, 64, device=DEV).to(BF16) for h in (4, 2, 2))
    w = torch.rand(3, 2, 96, device=DEV)
    good = la.la_paged_decode_step(q, k, v, kp.clone(), vp.clone(), table, lens)
    lens[1] = bad
    for call in ("decode", "fill", "evict"):
        kp2, vp2, w2, l2 = kp.clone(), vp.clone(), w.clone(), lens.clone()
        if call == "decode":
            y = torch.full((3, 4, 64), 7.0, dtype=BF16, device=DEV)
            lse = torch.full((3, 4), 7.0, device=DEV)
            la.la_paged_decode_step(q, k, v, kp2, vp2, table, l2, y=y, lse=lse, weights=w2)
            torch.cuda.synchronize()
            assert (y[1] == 7).all() and (lse[1] == 7).all()
            assert torch.equal(y[::2], good[::2])
        elif call == "fill":
            la.la_paged_cache_fill(k[:, :, None].contiguous(), v[:, :, None].contiguous(), kp2, vp2, table, l2,
                                   weights=w2)
        elif bad != 96:
            la.la_paged_evict(kp2, vp2, table, l2, w2, 30)
            torch.cuda.synchronize()
            assert l2.tolist() == [30, bad, 30]
        else:
            continue
        _reported()
        own = table[1].long()
        assert torch.equal(kp2[own], kp[own]) and torch.equal(vp2[own], vp[own]) and torch.equal(w2[1], w[1])


def test_narrow_and_wide_tables_agree():
    """The same short sequences behind a table of few pages (one block per unit) and of many (ranges and a join)."""
    for dtype, Hq, Hkv, d in ((BF16, 8, 2, 64), (BF16, 24, 2, 128), (F32, 4, 4, 64), (BF16, 3, 1, 33)):
        lens = [0, 1, 31, 128, 129, 200]
        kp, vp, table, ln = to_dev(*cache(71, dtype, len(lens), Hkv, d, d, 16, 13, lens))
        wide = torch.full((len(lens), 4000), -1, dtype=torch.int32, device=DEV)
        wide[:, :13] = table
        q = torch.randn(len(lens), Hq, d, device=DEV).to(dtype)
        n1 = la.la_paged_kernel_plan(1, len(lens), Hq, Hkv, d, d, 16, 13, False, la._dtype_code(q))[0]
        n2 = la.la_paged_kernel_plan(1, len(lens), Hq, Hkv, d, d, 16, 4000, False, la._dtype_code(q))[0]
        assert (n1, n2) == (1, 2)
        ref = orc.decode(*(t.cpu() for t in (q,)), None, None, *(t.cpu() for t in (kp, vp, table, ln)))
        for tab in (table, wide):
            lse = torch.empty(len(lens), Hq, device=DEV)
            y = la.la_paged_decode_step(q, None, None, kp, vp, tab, ln, lse=lse)
            sync()
            check_step(dtype, 200, d, (y, lse, None), (*ref[:2], None, *ref[3:]))


@pytest.mark.parametrize("bad", [-1, 20, 1 << 30, -(1 << 31)])
def test_bad_page_is_left_out_and_reported(bad):
    """A table entry outside the pool: its tokens are not attended to and not written."""
    kp, vp, table, lens = _bad_state()
    assert kp.shape[0] == 20
    q, k, v = (torch.randn(3, h, 64, device=DEV).to(BF16) for h in (4, 2, 2))
    broken = table.clone()
    broken[0, 1] = bad                               # slots 16..31 of sequence 0
    y = la.la_paged_decode_step(q, k, v, kp.clone(), vp.clone(), broken, lens)
    _reported()
    short = table.clone()                            # the same sequence without those slots
    short[0, 1], short[0, 2] = table[0, 2], table[0, 5]
    kp2, vp2 = kp.clone(), vp.clone()
    l2 = lens.clone()
    l2[0] -= 16
    ref = orc.decode(*(t.cpu() for t in (q, k, v, kp2, vp2, short, l2)))
    check_step(BF16, 61, 64, (y, None, None), (*ref[:2], None, *ref[3:]))
    # an eviction that would move rows leaves the sequence as it was
    w = torch.rand(3, 2, 96, device=DEV)
    kp2, vp2, w2, l2 = kp.clone(), vp.clone(), w.clone(), lens.clone()
    la.la_paged_evict(kp2, vp2, broken, l2, w2, 30)
    _reported()
    own = table[0].long()
    assert l2.tolist() == [40, 30, 30] and torch.equal(w2[0], w[0])
    assert torch.equal(kp2[own], kp[own]) and torch.equal(vp2[own], vp[own])
    # an append skips the tokens of that page and stores the others
    kk, vv = (torch.randn(3, 2, 30, 64, device=DEV).to(BF16) for _ in range(2))
    kp2, vp2, l2 = kp.clone(), vp.clone(), torch.zeros_like(lens)
    la.la_paged_cache_fill(kk, vv, kp2, vp2, broken, l2)
    _reported()
    assert torch.equal(kp2[table[0, 0].long()], kk[0, :, :16])
    assert torch.equal(kp2[table[0, 1].long()], kp[table[0, 1].long()])


def test_new_token_on_a_bad_page():
    """The new token's own page is out of range: it is not stored and not attended to."""
    kp, vp, table, lens = _bad_state()
    q, k, v = (torch.randn(3, h, 64, device=DEV).to(BF16) for h in (4, 2, 2))
    table[2, 3] = 1000                               # sequence 2 holds 60: slots 48..63
    kp2, vp2 = kp.clone(), vp.clone()
    y = la.la_paged_decode_step(q, k, v, kp2, vp2, table, lens)
    _reported()
    l2 = lens.clone().cpu()
    l2[2] = 48
    ref = orc.decode(q.cpu(), None, None, kp.cpu(), vp.cpu(), table.cpu(), l2)
    check_step(BF16, 61, 64, (y[2:], None, None), (ref[0][2:], ref[1][2:], None, ref[3][2:], ref[4][2:]))


def test_negative_pos_reported():
    kp, vp, table, lens = _bad_state()
    k, v = (torch.randn(3, 2, 1, 64, device=DEV).to(BF16) for _ in range(2))
    posn = torch.zeros(3, 2, 96, dtype=torch.int32, device=DEV)
    pos = torch.tensor([50, -1, 70], dtype=torch.int32, device=DEV)
    kp2 = kp.clone()
    la.la_paged_cache_fill(k, v, kp2, vp.clone(), table, lens, positions=posn, pos=pos)
    _reported()
    assert torch.equal(kp2[table[1].long()], kp[table[1].long()]) and posn[0, 0, 40] == 50 and (posn[1] == 0).all()


def test_deterministic():
    kp, vp, table, lens = to_dev(*cache(61, BF16, 2, 2, 64, 64, 16, 200, [3000, 1000]))
    q = torch.randn(2, 8, 64, device=DEV).to(BF16)
    ys = [la.la_paged_decode_step(q, None, None, kp, vp, table, lens) for _ in range(5)]
    sync()
    assert all(torch.equal(y, ys[0]) for y in ys)
