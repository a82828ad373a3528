"""Cases of the paged key/value cache: writing prompts into it, the attention of one new token over it, and
eviction by accumulated attention weight.

With ``own`` false ``run`` computes each operator from elementary torch operations in fp32; with ``own`` true it
makes the library's calls.  The cache of one layer:

  k_pages [P, Hkv, page, dqk], v_pages [P, Hkv, page, dv]; table [B, max_pages]; lens [B]: tokens held
  weights, positions [B, Hkv, max_pages * page]: per slot, the attention weight it has received and its token's
  position; pos [B]: tokens seen so far

Slot t of sequence b lies in page table[b, t // page], row t % page.  Where an operator has separate outputs for
the bookkeeping (weights_out, lens_out) they are used here, so that a pass can be repeated on the same state.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(name, op, dtype, B, Hq, Hkv, dqk, dv, page, longest, **more):
    c = {"name": name, "op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "dqk": dqk, "dv": dv, "page": page,
         "longest": longest, "ragged": False, "new": False, "weights": False, "budget": 0, "recent": 0}
    c.update(more)
    return c


def listed():
    return [
        # one user, a short context: latency
        _case("decode_alone_short", "decode", "bf16", 1, 8, 8, 64, 64, 16, 200, new=True),
        # one user, a very long context: one sequence has to fill the GPU
        _case("decode_alone_long", "decode", "bf16", 1, 32, 8, 128, 128, 64, 131072, new=True),
        # a serving batch of mixed context lengths, four query heads on each key/value head
        _case("decode_batch_ragged", "decode", "bf16", 64, 32, 8, 128, 128, 64, 8192, ragged=True, new=True),
        # many sequences with short contexts
        _case("decode_many_short", "decode", "bf16", 256, 16, 4, 64, 64, 64, 512, ragged=True, new=True),
        # attention over stored states that do not grow (an encoder's), fp32, a head of keys for each query head
        _case("decode_states_f32", "decode", "f32", 16, 16, 16, 64, 64, 128, 4096, ragged=True),
        # dimensions and pages that are no powers of two
        _case("decode_odd", "decode", "bf16", 17, 14, 2, 72, 40, 24, 1500, ragged=True, new=True),
        # the step of a bounded cache: the weights that each slot receives are summed up
        _case("decode_weights", "decode", "bf16", 64, 32, 8, 128, 128, 64, 2112, new=True, weights=True),
        # prompts written into the pages
        _case("fill_prompts", "fill", "bf16", 8, 8, 8, 128, 128, 64, 4096),
        # a padded batch of short prompts, odd sizes, fp32
        _case("fill_ragged_odd", "fill", "f32", 5, 3, 3, 33, 20, 7, 777, ragged=True, weights=True),
        # the steady state of a bounded cache: one page over budget
        _case("evict_step", "evict", "bf16", 64, 8, 8, 128, 128, 64, 2112, weights=True, budget=2048, recent=256),
        # long prompts cut down once, after they were read
        _case("evict_long", "evict", "bf16", 4, 8, 8, 128, 128, 64, 32768, weights=True, budget=4096, recent=512),
        # small, odd sizes, some sequences within their budget
        _case("evict_odd", "evict", "f32", 3, 3, 3, 24, 40, 10, 1000, ragged=True, weights=True, budget=333, recent=17),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "fill", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = _log(rng, 1, 16)
    g = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 20]) if op == "decode" else 1
    dqk, dv = (8 * rng.randint(2, 16) for _ in range(2))
    if rng.random() < 0.4:
        dqk = dv = rng.choice([64, 128])
    elif rng.random() < 0.2:
        dqk, dv = rng.randint(5, 127), rng.randint(5, 127)
    page = rng.choice([1, 8, 16, 24, 32, 64, 64, 100, 128, 256])
    B = _log(rng, 1, 256)
    longest = _log(rng, 16, 65536)
    # elements of the keys and values held: up to 1 GB to read, or to read and write
    most = 1 << (29 - (dtype == "f32") - (op != "decode"))
    while B * Hkv * longest * (dqk + dv) > most:
        if B > 1 and rng.random() < 0.5:
            B = (B + 1) // 2
        else:
            longest = max(16, longest // 2 + 1)
    c = _case("", op, dtype, B, Hkv * g, Hkv, dqk, dv, page, longest, ragged=rng.random() < 0.6,
              new=op == "decode" and rng.random() < 0.7, weights=op == "evict" or rng.random() < 0.3)
    if op == "evict":
        c["budget"] = max(1, int(longest * rng.uniform(0.1, 1.0)))
        c["recent"] = int(c["budget"] * rng.choice([0, 0.125, 0.5]))
    del c["name"]
    return c


def _lengths(c):
    """Tokens of each sequence after the pass (before it, for an eviction): a draw that depends on the case alone, so
    that the work is known; the longest is always there."""
    if not c["ragged"]:
        return [c["longest"]] * c["B"]
    r = random.Random("%(op)s %(B)d %(longest)d %(page)d" % c)
    return [c["longest"]] + [r.randint(1, c["longest"]) for _ in range(c["B"] - 1)]


def prepare(c, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    dt = _DT[c["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, Hq, Hkv, dqk, dv, page = c["B"], c["Hq"], c["Hkv"], c["dqk"], c["dv"], c["page"]
    n = torch.tensor(_lengths(c), dtype=torch.int32)
    max_pages = -(-c["longest"] // page)
    cap = max_pages * page
    used = torch.clamp(-(-n // page), min=1)
    if c["op"] == "evict":
        used = torch.full_like(used, max_pages)
    P = int(used.sum()) + 3
    # pages in the order in which a server hands them out: shuffled; unused entries hold -1
    order = torch.randperm(P, generator=torch.Generator().manual_seed(seed))[:P - 3].to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    table[torch.arange(max_pages)[None, :] < used[:, None]] = order
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32).to(dt)
    st = {"case": c, "longest": c["longest"], "table": table.to(dev),
          "k_pages": rnd(P, Hkv, page, dqk), "v_pages": rnd(P, Hkv, page, dv)}
    if c["op"] == "decode":
        st["q"] = rnd(B, Hq, dqk)
        if c["new"]:
            st["k"], st["v"] = rnd(B, Hkv, dqk), rnd(B, Hkv, dv)
            n = n - 1
    elif c["op"] == "fill":
        st["k"], st["v"] = rnd(B, Hkv, c["longest"], dqk), rnd(B, Hkv, c["longest"], dv)
        st["n_new"] = n.to(dev)
        n = torch.zeros_like(n)
    st["lens"] = n.to(dev)
    if c["weights"]:
        u = torch.rand(B, Hkv, cap, generator=gen, device=dev)
        st["weights"] = u / (1.0 - 0.999 * u)          # many small, few large
        st["weights_out"] = torch.zeros_like(st["weights"])
        # slots filled in order; every fourth swapped with its neighbour, as after earlier evictions
        p = torch.arange(cap, dtype=torch.int32, device=dev)
        p = torch.where(p % 4 == 1, p + 1, torch.where(p % 4 == 2, p - 1, p))
        st["positions"] = (p + 100).expand(B, Hkv, cap).contiguous()
        st["positions_out"] = torch.zeros_like(st["positions"])
        st["pos"] = st["lens"] + 100
        st["lens_out"] = torch.zeros_like(st["lens"])
    return st


# ------------------------------------------------------------------ plain forms

def _rows(st, L):
    """Row of every slot t < L in the pages seen as [P * Hkv * page, d]: [B, Hkv, L]."""
    Hkv, page = st["k_pages"].shape[1:3]
    t = torch.arange(L, device=st["table"].device)
    pg = st["table"].long().clamp(min=0)[:, t // page]
    h = torch.arange(Hkv, device=t.device)
    return (pg[:, None, :] * Hkv + h[None, :, None]) * page + (t % page)


def _plain_decode(st):
    q, kp, vp, lens = st["q"], st["k_pages"], st["v_pages"], st["lens"].long()
    B, Hq, dqk = q.shape
    Hkv, dv = kp.shape[1], vp.shape[3]
    L = st["longest"]
    rows = _rows(st, L)
    kf, vf = kp.view(-1, dqk), vp.view(-1, dv)
    n = lens
    if "k" in st:
        at = rows.gather(2, lens[:, None, None].expand(B, Hkv, 1))[:, :, 0]
        kf[at], vf[at] = st["k"], st["v"]
        n = lens + 1
    t = torch.arange(L, device=q.device)
    live = (t < n[:, None])[:, None, :, None]
    K = torch.where(live, kf[rows].float(), 0.0)
    V = torch.where(live, vf[rows].float(), 0.0)
    s = q.float().view(B, Hkv, Hq // Hkv, dqk) @ K.transpose(2, 3) * dqk ** -0.5
    s = torch.where(live.transpose(2, 3), s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    p = e / z
    out = {"y": (p @ V).view(B, Hq, dv).to(q.dtype), "lse": (m + torch.log(z)).view(B, Hq)}
    if "k" in st:
        out["k_pages"], out["v_pages"] = kp, vp
    if "weights" in st:
        w, wo = st["weights"][..., :L], st["weights_out"][..., :L]
        old = torch.where(t < lens[:, None, None], w, 0.0)
        wo.copy_(torch.where(t < n[:, None, None], old + p.sum(2), wo))
        out["weights"] = st["weights_out"]
        if "k" in st:
            st["positions"].scatter_(2, lens[:, None, None].expand(B, Hkv, 1),
                                     st["pos"][:, None, None].expand(B, Hkv, 1))
            out["positions"] = st["positions"]
    return out


def _plain_fill(st):
    k, v, kp, vp = st["k"], st["v"], st["k_pages"], st["v_pages"]
    B, Hkv, N, dqk = k.shape
    # tokens past a sequence's own repeat its last one
    i = torch.minimum(torch.arange(N, device=k.device), st["n_new"].long()[:, None] - 1)
    rows = _rows(st, N).gather(2, (st["lens"].long()[:, None] + i)[:, None, :].expand(B, Hkv, N))
    at = i[:, None, :, None]
    kp.view(-1, dqk)[rows] = k.gather(2, at.expand(B, Hkv, N, dqk))
    vp.view(-1, v.shape[3])[rows] = v.gather(2, at.expand(B, Hkv, N, v.shape[3]))
    out = {"k_pages": kp, "v_pages": vp}
    if "weights" in st:
        slot = (st["lens"].long()[:, None] + i)[:, None, :].expand(B, Hkv, N)
        st["weights"].scatter_(2, slot, 0.0)
        st["positions"].scatter_(2, slot, (st["pos"][:, None] + i).int()[:, None, :].expand(B, Hkv, N))
        out["weights"], out["positions"] = st["weights"], st["positions"]
    return out


def _plain_evict(st):
    c = st["case"]
    kp, vp, budget = st["k_pages"], st["v_pages"], c["budget"]
    B, Hkv = st["weights"].shape[:2]
    L = st["longest"]
    n = st["lens"].long()[:, None, None]
    t = torch.arange(L, device=n.device).expand(B, Hkv, L)
    w, pos = st["weights"][..., :L], st["positions"][..., :L]
    key = torch.where(pos >= st["pos"][:, None, None] - c["recent"], math.inf, w) if c["recent"] else w
    key = torch.where(t < n, key, -math.inf)
    ranked = torch.sort(key, dim=2, descending=True, stable=True).indices
    kept = torch.zeros_like(t, dtype=torch.bool).scatter_(2, ranked[..., :budget], True) & (t < n)
    mover, hole = kept & (t >= budget), ~kept & (t < budget) & (t < n)
    # the i-th dropped slot below the budget takes the i-th kept one above it
    nth = torch.where(mover, mover.cumsum(2) - 1, L)
    source = torch.zeros(B, Hkv, L + 1, dtype=torch.long, device=n.device).scatter_(2, nth, t)
    src = torch.where(hole, source.gather(2, (hole.cumsum(2) - 1).clamp(min=0)), t)[..., :budget]
    rows = _rows(st, L)
    to, frm = rows[..., :budget], rows.gather(2, src)
    kf, vf = kp.view(-1, kp.shape[3]), vp.view(-1, vp.shape[3])
    kf[to], vf[to] = kf[frm], vf[frm]
    live = t[..., :budget] < n
    wo, po = st["weights_out"][..., :budget], st["positions_out"][..., :budget]
    wo.copy_(torch.where(live, w.gather(2, src), wo))
    po.copy_(torch.where(live, pos.gather(2, src), po))
    st["lens_out"].copy_(st["lens"].clamp(max=budget))
    return {"lens": st["lens_out"], "weights": st["weights_out"], "positions": st["positions_out"],
            "k_pages": kp, "v_pages": vp}


# ------------------------------------------------------------------ the library's calls

def _own_decode(st):
    import causal_kernelized_sequence_b200 as la
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=st["q"].device)
    more = {}
    if "weights" in st:
        more = {"weights": st["weights"], "weights_out": st["weights_out"]}
        if "k" in st:
            more.update(positions=st["positions"], pos=st["pos"])
    y = la.la_paged_decode_step(st["q"], st.get("k"), st.get("v"), st["k_pages"], st["v_pages"], st["table"],
                                st["lens"], lse=lse, **more)
    out = {"y": y, "lse": lse}
    if "k" in st:
        out["k_pages"], out["v_pages"] = st["k_pages"], st["v_pages"]
    if "weights" in st:
        out["weights"] = st["weights_out"]
        if "k" in st:
            out["positions"] = st["positions"]
    return out


def _own_fill(st):
    import causal_kernelized_sequence_b200 as la
    more = {x: st[x] for x in ("weights", "positions", "pos") if x in st}
    la.la_paged_cache_fill(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                           n_new=st["n_new"], **more)
    out = {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    if "weights" in st:
        out["weights"], out["positions"] = st["weights"], st["positions"]
    return out


def _own_evict(st):
    import causal_kernelized_sequence_b200 as la
    c = st["case"]
    la.la_paged_evict(st["k_pages"], st["v_pages"], st["table"], st["lens"], st["weights"], c["budget"],
                      recent=c["recent"], positions=st["positions"], pos=st["pos"], lens_out=st["lens_out"],
                      weights_out=st["weights_out"], positions_out=st["positions_out"])
    return {"lens": st["lens_out"], "weights": st["weights_out"], "positions": st["positions_out"],
            "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def run(st):
    op = st["case"]["op"]
    if own:
        return {"decode": _own_decode, "fill": _own_fill, "evict": _own_evict}[op](st)
    return {"decode": _plain_decode, "fill": _plain_fill, "evict": _plain_evict}[op](st)


def work(c):
    el = 4 if c["dtype"] == "f32" else 2
    d = c["dqk"] + c["dv"]
    n = _lengths(c)
    tokens = sum(n) * c["Hkv"]
    if c["op"] == "decode":
        small = c["B"] * (c["Hq"] * (d * el + 4) + (2 * c["Hkv"] * d * el if c["new"] else 0) + 4)
        return {"bytes": tokens * d * el + small + (8 * tokens if c["weights"] else 0),
                "flops": 2 * sum(n) * c["Hq"] * d}
    if c["op"] == "fill":
        return {"bytes": 2 * tokens * d * el + (8 * tokens if c["weights"] else 0), "flops": 0}
    # weights and positions of every slot read, those kept written; of a sequence's dropped tokens, a share
    # budget / length lies below the budget, and as many rows move
    over = sum((x - c["budget"]) * c["budget"] // x for x in n if x > c["budget"]) * c["Hkv"]
    kept = sum(min(x, c["budget"]) for x in n) * c["Hkv"]
    return {"bytes": 2 * over * d * el + 8 * tokens + 8 * kept, "flops": 0}


# ------------------------------------------------------------------ 64 bits

def _slots(st, b, h, n):
    """Rows (page, row) of the first n slots of sequence b."""
    page = st["k_pages"].shape[2]
    t = torch.arange(n, device=st["table"].device)
    return st["table"][b].long()[t // page], t % page


def exact(c, seed):
    st = prepare(c, seed)
    B, Hq, Hkv, dqk = c["B"], c["Hq"], c["Hkv"], c["dqk"]
    kp, vp = st["k_pages"], st["v_pages"]
    lens = st["lens"].tolist()
    if c["op"] == "decode":
        y = torch.zeros(B, Hq, c["dv"], dtype=torch.float64, device=kp.device)
        lse = torch.zeros(B, Hq, dtype=torch.float64, device=kp.device)
        wo = st["weights_out"].double() if c["weights"] else None
        for b in range(B):
            pg, r = _slots(st, b, 0, lens[b] + (1 if c["new"] else 0))
            if c["new"]:
                kp[pg[-1], :, r[-1]], vp[pg[-1], :, r[-1]] = st["k"][b], st["v"][b]
            for h in range(Hkv):
                K, V = kp[pg, h, r].double(), vp[pg, h, r].double()
                heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                s = K @ st["q"][b, heads].double().T / math.sqrt(dqk)
                lse[b, heads] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                y[b, heads] = p.T @ V
                if c["weights"]:
                    got = p.sum(1)
                    got[:lens[b]] += st["weights"][b, h, :lens[b]].double()
                    wo[b, h, :got.numel()] = got
        out = {"y": y, "lse": lse}
        if c["new"]:
            out["k_pages"], out["v_pages"] = kp, vp
        if c["weights"]:
            out["weights"] = wo
            if c["new"]:
                for b in range(B):
                    st["positions"][b, :, lens[b]] = st["pos"][b]
                out["positions"] = st["positions"]
        return out
    if c["op"] == "fill":
        for b, n in enumerate(st["n_new"].tolist()):
            pg, r = _slots(st, b, 0, lens[b] + n)
            kp[pg[lens[b]:], :, r[lens[b]:]] = st["k"][b, :, :n].transpose(0, 1)
            vp[pg[lens[b]:], :, r[lens[b]:]] = st["v"][b, :, :n].transpose(0, 1)
            if c["weights"]:
                st["weights"][b, :, lens[b]:lens[b] + n] = 0
                st["positions"][b, :, lens[b]:lens[b] + n] = st["pos"][b] + torch.arange(n, device=kp.device)
        out = {"k_pages": kp, "v_pages": vp}
        if c["weights"]:
            out["weights"], out["positions"] = st["weights"].double(), st["positions"]
        return out
    wo, po, lo = st["weights_out"], st["positions_out"], st["lens_out"]
    for b in range(B):
        n, budget = lens[b], c["budget"]
        lo[b] = min(n, budget)
        for h in range(Hkv):
            w, p = st["weights"][b, h, :n], st["positions"][b, h, :n]
            keep = torch.arange(n, device=w.device)
            if n > budget:
                recent = p >= int(st["pos"][b]) - c["recent"] if c["recent"] else torch.zeros_like(p, dtype=torch.bool)
                first = keep[recent][:budget]
                rest = keep[~recent]
                rest = rest[torch.argsort(w[rest], descending=True, stable=True)[:budget - first.numel()]]
                keep = torch.cat([first, rest]).sort().values
                into = torch.ones(budget, dtype=torch.bool, device=w.device)
                into[keep[keep < budget]] = False
                into, frm = into.nonzero()[:, 0], keep[keep >= budget]
                keep = torch.arange(budget, device=w.device)
                keep[into] = frm
                pg, r = _slots(st, b, h, n)
                kp[pg[into], h, r[into]] = kp[pg[frm], h, r[frm]]
                vp[pg[into], h, r[into]] = vp[pg[frm], h, r[frm]]
            wo[b, h, :keep.numel()], po[b, h, :keep.numel()] = w[keep], p[keep]
    return {"lens": lo, "weights": wo.double(), "positions": po, "k_pages": kp, "v_pages": vp}
