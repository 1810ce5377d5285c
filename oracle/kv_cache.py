"""The paged key-value cache in fp64 numpy: append, attention, eviction.

A cache is a dict of numpy arrays named as in include/sta.h (sta_kv_cache):
k_pages, v_pages [num_pages, kv_heads, 64, d] in fp64; page_table
[B, max_pages]; lens, seen [B, kv_heads]; slot_pos, weight
[B, kv_heads, 64 * max_pages]. Calls change it in place, slot by slot.
"""
import numpy as np

PAGE = 64


def where(c, b, slot):
    """(page, row in it) of a slot of sequence b."""
    return int(c["page_table"][b, slot // PAGE]), slot % PAGE


def append(c, k_new, v_new, counts=None):
    B, n, kv, _ = k_new.shape
    for b in range(B):
        m = n if counts is None else int(counts[b])
        for h in range(kv):
            for i in range(m):
                slot = int(c["lens"][b, h]) - m + i
                page, row = where(c, b, slot)
                c["k_pages"][page, h, row] = k_new[b, i, h]
                c["v_pages"][page, h, row] = v_new[b, i, h]
                if c.get("slot_pos") is not None:
                    c["slot_pos"][b, h, slot] = int(c["seen"][b, h]) - m + i
                if c.get("weight") is not None:
                    c["weight"][b, h, slot] = 0.0


def attend(c, q, scale, lists=None, accumulate=False, by_position=False):
    """(o, lse, sigma, terms): o [B, n_q, q_heads, d], lse [B, q_heads, n_q];
    for the tests' error bounds, sigma (like o) = sum_j p_j |v_j| and terms
    (like lse) = max_j of scale * sum_i |q_i k_ji|. lists[b][h]: the page
    columns of a head, None: all. Query i of n_q does not see the n_q - 1 - i
    newest tokens: the last slots or, by position, those at seen - (n_q - 1 - i)
    and later (the newest query sees every slot)."""
    B, n_q, hq, d = q.shape
    kv = c["lens"].shape[1]
    group = hq // kv
    o, sigma = np.zeros((B, n_q, hq, d)), np.zeros((B, n_q, hq, d))
    lse, terms = np.full((B, hq, n_q), -np.inf), np.zeros((B, hq, n_q))
    for b in range(B):
        for h in range(kv):
            n = int(c["lens"][b, h])
            cols = range(-(-n // PAGE)) if lists is None else lists[b][h]
            for i in range(n_q):
                end = n if by_position else n - (n_q - 1 - i)
                slots = [j for p in cols for j in range(p * PAGE, min(end, p * PAGE + PAGE))]
                if by_position and i < n_q - 1:
                    slots = [j for j in slots if c["slot_pos"][b, h, j] < c["seen"][b, h] - (n_q - 1 - i)]
                if not slots:
                    continue
                at = [where(c, b, j) for j in slots]
                k = np.stack([c["k_pages"][p, h, r] for p, r in at])
                v = np.stack([c["v_pages"][p, h, r] for p, r in at])
                for g in range(group):
                    x = q[b, i, h * group + g]
                    s = scale * (k @ x)
                    top = s.max()
                    e = np.exp(s - top)
                    z = e.sum()
                    o[b, i, h * group + g] = (e / z) @ v
                    sigma[b, i, h * group + g] = (e / z) @ np.abs(v)
                    lse[b, h * group + g, i] = top + np.log(z)
                    terms[b, h * group + g, i] = scale * (np.abs(k) @ np.abs(x)).max()
                    if accumulate:
                        c["weight"][b, h, slots] += e / z
    return o, lse, sigma, terms


def evict(c, budget, recent, sinks):
    B, kv = c["lens"].shape
    for b in range(B):
        for h in range(kv):
            n = int(c["lens"][b, h])
            if n <= budget:
                continue

            def rank(j):
                p, w = int(c["slot_pos"][b, h, j]), float(c["weight"][b, h, j])
                if p < sinks or p >= int(c["seen"][b, h]) - recent:
                    return (0, 0.0, j)
                return (2, 0.0, j) if np.isnan(w) else (1, -w, j)

            stay = sorted(sorted(range(n), key=rank)[:budget])
            given_up = [j for j in range(budget) if j not in set(stay)]
            for to, of in zip(given_up, [j for j in stay if j >= budget]):
                (pt, rt), (pf, rf) = where(c, b, to), where(c, b, of)
                c["k_pages"][pt, h, rt] = c["k_pages"][pf, h, rf]
                c["v_pages"][pt, h, rt] = c["v_pages"][pf, h, rf]
                c["slot_pos"][b, h, to] = c["slot_pos"][b, h, of]
                c["weight"][b, h, to] = c["weight"][b, h, of]
            c["lens"][b, h] = budget
