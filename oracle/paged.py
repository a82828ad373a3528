"""fp64 CPU oracle of the paged key/value cache: appending tokens, the attention
of one new token over the cache, and eviction by accumulated weight.

TEST INFRASTRUCTURE ONLY, written from the definitions in include/la.h, one
sequence, head and token at a time.  Floating inputs may be tensors of any
type; results are float64 (moved rows keep their type).  The functions return
new tensors and leave their arguments alone.
"""
from __future__ import annotations

import math

import torch


def slot(table, page, b, t):
    """(page, row) of slot t of sequence b."""
    return int(table[b, t // page]), t % page


def fill(k, v, k_pages, v_pages, table, lens, n_new=None, weights=None, positions=None, pos=None):
    """(k_pages, v_pages, weights, positions) after the append."""
    kp, vp = k_pages.clone(), v_pages.clone()
    w = None if weights is None else weights.clone()
    p = None if positions is None else positions.clone()
    for b in range(k.shape[0]):
        for i in range(k.shape[2] if n_new is None else int(n_new[b])):
            t = int(lens[b]) + i
            pg, r = slot(table, k_pages.shape[2], b, t)
            kp[pg, :, r], vp[pg, :, r] = k[b, :, i], v[b, :, i]
            if w is not None:
                w[b, :, t] = 0
            if p is not None:
                p[b, :, t] = int(pos[b]) + i
    return kp, vp, w, p


def decode(q, k, v, k_pages, v_pages, table, lens, weights=None):
    """(y [B,Hq,dv], lse [B,Hq], weights, size [B,Hq,dv], spread [B,Hq]):
    size = sum_t p_t |v_t| and spread = max_t sum_i |q_i k_ti| / sqrt(dqk), which
    bound what fp32 sums of these terms may lose."""
    B, Hq, dqk = q.shape
    Hkv, page, dv = k_pages.shape[1], k_pages.shape[2], v_pages.shape[3]
    g = Hq // Hkv
    y = torch.zeros(B, Hq, dv, dtype=torch.float64)
    size = torch.zeros_like(y)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    spread = torch.zeros(B, Hq, dtype=torch.float64)
    w = None if weights is None else weights.double().clone()
    for b in range(B):
        n = int(lens[b])
        at = [slot(table, page, b, t) for t in range(n)]
        for h in range(Hkv):
            K = [k_pages[pg, h, r].double() for pg, r in at]
            V = [v_pages[pg, h, r].double() for pg, r in at]
            if k is not None:
                K.append(k[b, h].double())
                V.append(v[b, h].double())
                if w is not None:
                    w[b, h, n] = 0
            if not K:
                continue
            K, V = torch.stack(K), torch.stack(V)
            for hq in range(h * g, (h + 1) * g):
                qq = q[b, hq].double()
                s = (K * qq).sum(1) / math.sqrt(dqk)
                e = torch.exp(s - s.max())
                p = e / e.sum()
                y[b, hq] = (p[:, None] * V).sum(0)
                size[b, hq] = (p[:, None] * V.abs()).sum(0)
                lse[b, hq] = s.max() + torch.log(e.sum())
                spread[b, hq] = (K * qq).abs().sum(1).max() / math.sqrt(dqk)
                if w is not None:
                    w[b, h, :len(p)] += p
    return y, lse, w, size, spread


def evict(k_pages, v_pages, table, lens, weights, budget, recent=0, positions=None, pos=None):
    """(k_pages, v_pages, lens, weights, positions); weights and positions hold
    the kept slots' entries below the new length and are unchanged above it."""
    kp, vp, w, new = k_pages.clone(), v_pages.clone(), weights.clone(), lens.clone()
    p = None if positions is None else positions.clone()
    page = k_pages.shape[2]
    for b in range(lens.numel()):
        n = int(lens[b])
        if n <= budget:
            continue
        new[b] = budget
        for h in range(k_pages.shape[1]):
            def rank(t):
                x = float(weights[b, h, t])
                x = -math.inf if math.isnan(x) else x
                late = recent > 0 and int(positions[b, h, t]) >= int(pos[b]) - recent
                return (not late, -x, t)
            keep = set(sorted(range(n), key=rank)[:budget])
            into = [t for t in range(budget) if t not in keep]
            frm = [t for t in range(budget, n) if t in keep]
            assert len(into) == len(frm)
            for a, z in zip(into, frm):
                (pa, ra), (pz, rz) = slot(table, page, b, a), slot(table, page, b, z)
                kp[pa, h, ra], vp[pa, h, ra] = k_pages[pz, h, rz], v_pages[pz, h, rz]
                w[b, h, a] = weights[b, h, z]
                if p is not None:
                    p[b, h, a] = positions[b, h, z]
    return kp, vp, new, w, p
