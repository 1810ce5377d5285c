"""What is measured of the paged key-value cache: appending to it, attention of
new tokens over it (with or without accumulating each cached token's attention
weight), and eviction by that weight.

The cache of B sequences (see include/sta.h, sta_kv_cache):
  k_pages, v_pages [num_pages, kv_heads, 64, d]   pages of 64 tokens
  page_table       [B, max_pages] int32           page of slots 64 p .. 64 p + 63
  lens, seen       [B, kv_heads] int32            filled slots; tokens ever appended
  slot_pos, weight [B, kv_heads, 64 max_pages]    position of the token in a slot;
                                                  attention weight it has gathered

With `own` false, `run` computes in elementary torch operations in 32 bits;
with `own` true it makes the calls a user makes.
"""
import math

import torch

own = False

PAGE = 64
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases
def _attend(name, B, kv, group, d, dtype, n_q, lo, hi, pages=1.0, accumulate=False):
    return {"name": name, "op": "attend", "B": B, "kv": kv, "group": group, "d": d, "dtype": dtype, "n_q": n_q,
            "lo": lo, "hi": hi, "pages": pages, "accumulate": accumulate}


def _append(name, B, kv, d, dtype, n, least, before):
    return {"name": name, "op": "append", "B": B, "kv": kv, "d": d, "dtype": dtype, "n": n, "least": least,
            "before": before}


def _evict(name, B, kv, d, dtype, lo, hi, budget, recent, sinks):
    return {"name": name, "op": "evict", "B": B, "kv": kv, "d": d, "dtype": dtype, "lo": lo, "hi": hi,
            "budget": budget, "recent": recent, "sinks": sinks}


def _step(name, B, kv, group, d, dtype, budget, recent, sinks):
    return {"name": name, "op": "step", "B": B, "kv": kv, "group": group, "d": d, "dtype": dtype, "budget": budget,
            "recent": recent, "sinks": sinks}


def listed():
    return [
        # the tiny layer's 1,024 tokens, two heads: what one call costs when there is next to nothing to read
        _attend("attend_tiny", 1, 2, 1, 64, "bf16", 1, 1024, 1024),
        # one new token over a whole 480p clip (21 x 30 x 52 tokens, 40 heads)
        _attend("attend_480p", 1, 40, 1, 128, "bf16", 1, 32760, 32760),
        # a serving batch of ragged lengths, four query heads to a key head
        _attend("attend_gqa_ragged", 32, 8, 4, 128, "bf16", 1, 65, 8192),
        # four draft tokens a sequence, checked in one call
        _attend("attend_drafts_fp16", 16, 24, 1, 128, "fp16", 4, 101, 2501),
        # block-sparse: 15% of the pages of a 720p clip (21 x 45 x 80 tokens), a list for each head
        _attend("attend_720p_pages", 1, 40, 1, 128, "bf16", 1, 75600, 75600, pages=0.15),
        # the largest: a 129-frame clip (33 x 45 x 80 tokens, 24 heads), each token's weight accumulated
        _attend("weigh_129f", 1, 24, 1, 128, "bf16", 1, 118800, 118800, accumulate=True),
        # accumulated weights of a ragged batch with eight query heads to a key head
        _attend("weigh_gqa_fp16", 8, 8, 8, 64, "fp16", 1, 500, 16384, accumulate=True),
        # one token for each of 64 sequences, as every decoding step appends
        _append("append_token", 64, 8, 128, "bf16", 1, 1, 1777),
        # a 480p prompt into an empty cache
        _append("append_480p", 1, 40, 128, "bf16", 32760, 32760, 0),
        # a 720p prompt cut to a quarter
        _evict("evict_720p", 1, 40, 128, "bf16", 75600, 75600, 18900, 3600, 64),
        # a batch of which some sequences are under the budget
        _evict("evict_batch_fp16", 64, 8, 64, "fp16", 100, 4096, 1024, 128, 4),
        # the calls together at a steady length: append a token, evict one, attend and accumulate
        _step("step_steady", 32, 8, 4, 128, "bf16", 2048, 256, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1 - 1e-9))) - 0.5 + 1e-9)) if hi > lo else lo


def _between(rng, lo, hi):
    return max(lo, min(hi, _log(rng, max(lo, 1), hi)))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "weigh", "append", "evict", "step"))
    B = _between(rng, 1, 64)
    kv = rng.choice((1, 2, 4, 8, 10, 24, 40))
    d = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "fp16"))
    most = 75600 * 40 * 128 // (B * kv * d)  # as many cached values as the 720p clip has
    if op in ("attend", "weigh"):
        group = rng.choice((1, 1, 2, 4, 5, 8))
        n_q = rng.choice((1, 1, 1, 2, 3, 5, 8))
        hi = _between(rng, 1, max(1, min(118800, most // (2 if group * n_q > 8 else 1))))
        lo = hi if rng.random() < 0.3 else rng.choice((0, 1, max(1, hi // 50)))
        pages = rng.choice((1.0, 1.0, 0.5, 0.2, 0.05)) if op == "attend" else 1.0
        c = _attend("", B, kv, group, d, dtype, n_q, lo, hi, pages, op == "weigh")
    elif op == "append":
        n = _between(rng, 1, max(1, min(32760, most // 2)))
        c = _append("", B, kv, d, dtype, n, rng.choice((0, max(1, n // 7), n)), rng.randrange(0, min(4000, most)))
    elif op == "evict":
        hi = _between(rng, 40, max(64, min(75600, most)))
        budget = max(2, int(hi * rng.uniform(0.05, 0.95)))
        sinks = min(rng.choice((0, 1, 4, 64)), budget // 4)
        c = _evict("", B, kv, d, dtype, rng.choice((1, max(1, hi // 30), hi)), hi, budget,
                   rng.randrange(0, budget - sinks), sinks)
    else:
        budget = _between(rng, 16, max(16, min(16384, most // 2)))
        sinks = min(rng.choice((0, 4)), budget // 4)
        c = _step("", B, kv, rng.choice((1, 2, 4, 8)), d, dtype, budget, budget // rng.choice((2, 4, 8)), sinks)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _ladder(lo, hi, n):
    """n lengths from lo to hi, even in their logarithm, as a mixed batch has."""
    if n == 1 or lo == hi:
        return [hi] * n
    a, b = math.log(max(lo, 0.5)), math.log(hi)
    got = [int(round(math.exp(a + (b - a) * i / (n - 1)))) for i in range(n)]
    got[0], got[-1] = lo, hi
    return got


def _pages(n):
    return -(-n // PAGE)


def _cache(case, lens, cap, g, tracked):
    """A cache whose sequence b holds lens[b] tokens and has pages for cap[b]; its pages lie in any order."""
    B, kv, d, dt = case["B"], case["kv"], case["d"], DT[case["dtype"]]
    dev = "cuda"
    need = [_pages(c) for c in cap]
    max_pages = max(1, max(need))
    num = sum(need) + 3  # and a few that nobody owns
    k = torch.empty(num, kv, PAGE, d, device=dev, dtype=dt).normal_(generator=g)
    v = torch.empty(num, kv, PAGE, d, device=dev, dtype=dt).normal_(generator=g)
    u = torch.randn(kv, d, device=dev, generator=g)  # what the queries of a head look for; some keys have more of it
    heavy = torch.rand(num, kv, PAGE, device=dev, generator=g) < 0.02
    at = heavy.nonzero(as_tuple=True)
    k[at] += u[at[1]].to(dt)
    order = torch.randperm(num, device=dev, generator=g).to(torch.int32)
    table = torch.full((B, max_pages), -1, device=dev, dtype=torch.int32)
    own_page = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table[own_page] = order[:sum(need)]
    s = {"k_pages": k, "v_pages": v, "page_table": table,
         "lens": torch.tensor(lens, device=dev, dtype=torch.int32)[:, None].expand(B, kv).contiguous(),
         "seen": None, "slot_pos": None, "weight": None, "look": u}
    if tracked:
        slots = PAGE * max_pages
        s["seen"] = s["lens"].clone()
        s["slot_pos"] = torch.arange(slots, device=dev, dtype=torch.int32).expand(B, kv, slots).contiguous()
        # gathered weights: a long tail of small ones, a few large
        e = torch.empty(B, kv, slots, device=dev).exponential_(generator=g)
        s["weight"] = e * e * e * 0.05
    return s


def _queries(case, s, n_q, g):
    B, kv, group, d = case["B"], case["kv"], case["group"], case["d"]
    q = torch.randn(B, n_q, kv, group, d, device="cuda", generator=g) * 1.2 + 0.3 * s["look"][None, None, :, None]
    return q.reshape(B, n_q, kv * group, d).to(DT[case["dtype"]])


def _permuted(v, g):
    """The lengths of the ladder, given to the sequences in an order of the seed."""
    if len(v) == 1:
        return v
    return [v[i] for i in torch.randperm(len(v), device="cuda", generator=g).tolist()]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    B, kv, d, op = case["B"], case["kv"], case["d"], case["op"]
    dt = DT[case["dtype"]]
    if op == "append":
        counts = _permuted(_ladder(case["least"], case["n"], B), g)
        s = _cache(case, [case["before"] + c for c in counts], [case["before"] + c for c in counts], g, True)
        s["counts"] = torch.tensor(counts, device="cuda", dtype=torch.int32)
        s["k_new"] = torch.empty(B, case["n"], kv, d, device="cuda", dtype=dt).normal_(generator=g)
        s["v_new"] = torch.empty(B, case["n"], kv, d, device="cuda", dtype=dt).normal_(generator=g)
    elif op == "step":
        s = _cache(case, [case["budget"]] * B, [case["budget"] + 1] * B, g, True)
        s["k_new"] = torch.empty(B, 1, kv, d, device="cuda", dtype=dt).normal_(generator=g)
        s["v_new"] = torch.empty(B, 1, kv, d, device="cuda", dtype=dt).normal_(generator=g)
        s["counts"] = None
    else:
        lens = _permuted(_ladder(case["lo"], case["hi"], B), g)
        s = _cache(case, lens, lens, g, op == "evict" or case["accumulate"])
    if op in ("attend", "step"):
        n_q = case["n_q"] if op == "attend" else 1
        s["q"] = _queries(case, s, n_q, g)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, kv * case["group"], n_q, device="cuda")
    s["page_ptr"] = s["page_idx"] = None
    if op == "attend" and case["pages"] < 1.0:
        # each head's list: a share of the sequence's pages, and always the newest one
        have = (s["lens"] + PAGE - 1) // PAGE
        p = torch.arange(s["page_table"].shape[1], device="cuda")
        mask = torch.rand(B, kv, p.numel(), device="cuda", generator=g) < case["pages"]
        mask = (mask | (p == have[..., None] - 1)) & (p < have[..., None])
        s["page_ptr"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64),
                                   mask.reshape(B * kv, -1).sum(1).cumsum(0)]).to(torch.int32)
        s["page_idx"] = mask.nonzero()[:, 2].to(torch.int32).contiguous()
    if op == "evict":
        # the lengths, positions and weights of the full cache: a pass starts from them (the rows of the tokens
        # that move are still in the slots past the budget)
        s["full"] = [s[n].clone() for n in ("lens", "slot_pos", "weight")]
    s["case"] = case
    if own:
        import block_sparse_attention_28_b200 as sta

        s["cache"] = sta.kv_cache(s["k_pages"], s["v_pages"], s["page_table"], s["lens"], s["seen"], s["slot_pos"],
                                  s["weight"])
        if op in ("attend", "step"):
            n = sta.sta_attn_fwd_cached_workspace(s["cache"], kv * case["group"], s["q"].shape[1],
                                                  op == "step" or case["accumulate"])
            s["attend_ws"] = torch.empty(n, device="cuda", dtype=torch.uint8)
        if op in ("evict", "step"):
            n = sta.sta_cache_evict_workspace(s["cache"], case["budget"])
            s["evict_ws"] = torch.empty(n, device="cuda", dtype=torch.uint8)
    return s


# -------------------------------------------------------------- plain forms
def _plain_append(s):
    """Token i of the counts[b] new ones goes to slot lens - counts + i of its sequence and head."""
    k_new, v_new, lens = s["k_new"], s["v_new"], s["lens"].long()
    B, n, kv, _ = k_new.shape
    dev = k_new.device
    counts = s["counts"].long() if s["counts"] is not None else torch.full((B,), n, device=dev)
    b, i = (torch.arange(n, device=dev)[None] < counts[:, None]).nonzero(as_tuple=True)
    slot = lens[b] - counts[b][:, None] + i[:, None]  # [tokens, kv]
    h = torch.arange(kv, device=dev)[None].expand_as(slot)
    page = s["page_table"].long()[b[:, None], slot // PAGE]
    s["k_pages"][page, h, slot % PAGE] = k_new[b, i]
    s["v_pages"][page, h, slot % PAGE] = v_new[b, i]
    s["slot_pos"][b[:, None], h, slot] = (s["seen"].long()[b] - counts[b][:, None] + i[:, None]).to(torch.int32)
    s["weight"][b[:, None], h, slot] = 0.0


def _plain_attend(s, accumulate):
    q, lens, table = s["q"], s["lens"].long(), s["page_table"].long().clamp_min(0)
    B, n_q, hq, d = q.shape
    kv = lens.shape[1]
    group, slots = hq // kv, table.shape[1] * PAGE
    slot = torch.arange(slots, device=q.device)
    held = slot < lens[..., None]  # [B, kv, slots]
    k = s["k_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, kv, slots, d).float()
    v = s["v_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, kv, slots, d).float()
    k.mul_(held[..., None])
    v.mul_(held[..., None])
    qf = q.float().reshape(B, n_q, kv, group, d).permute(0, 2, 1, 3, 4).reshape(B, kv, n_q * group, d)
    x = (qf @ k.transpose(-1, -2)) / math.sqrt(d)
    last = lens[..., None] - (n_q - 1 - torch.arange(n_q, device=q.device))  # slots that query i sees
    seen = (slot < last[..., None]).repeat_interleave(group, 2)
    if s["page_ptr"] is not None:
        ptr = s["page_ptr"].long()
        row = torch.repeat_interleave(torch.arange(B * kv, device=q.device), ptr[1:] - ptr[:-1])
        listed_page = torch.zeros(B * kv, table.shape[1], device=q.device, dtype=torch.bool)
        listed_page[row, s["page_idx"].long()] = True
        seen = seen & listed_page.reshape(B, kv, 1, -1).repeat_interleave(PAGE, 3)
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    z = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(z == 0, 1.0, z)
    lse = (top + torch.log(z))[..., 0]
    if accumulate:
        s["weight"] += (p / torch.where(z == 0, 1.0, z)).sum(2)
    s["o"].copy_(o.reshape(B, kv, n_q, group, d).permute(0, 2, 1, 3, 4).reshape(B, n_q, hq, d))
    s["lse"].copy_(lse.reshape(B, kv, n_q, group).permute(0, 1, 3, 2).reshape(B, hq, n_q))


def _plain_evict(s, budget, recent, sinks):
    """Keeps the sinks, the recent tokens and the heaviest others; a kept token past the budget moves into the
    next slot below it that was given up."""
    lens, pos, weight = s["lens"].long(), s["slot_pos"].long(), s["weight"]
    slot = torch.arange(weight.shape[2], device=weight.device)
    over = lens > budget
    safe = (pos < sinks) | (pos >= s["seen"].long()[..., None] - recent)
    key = torch.where(safe, math.inf, weight)
    key = torch.where(slot < lens[..., None], key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(safe).scatter_(2, order[..., :budget], True)
    hole = (over[..., None] & ~keep & (slot < budget)).nonzero(as_tuple=True)
    b, h, src = (over[..., None] & keep & (slot >= budget)).nonzero(as_tuple=True)
    dst = hole[2]  # as many, in the same rows, in rising order
    table = s["page_table"].long()
    for_src, for_dst = (table[b, src // PAGE], h, src % PAGE), (table[b, dst // PAGE], h, dst % PAGE)
    s["k_pages"][for_dst] = s["k_pages"][for_src]
    s["v_pages"][for_dst] = s["v_pages"][for_src]
    s["slot_pos"][b, h, dst] = s["slot_pos"][b, h, src]
    s["weight"][b, h, dst] = s["weight"][b, h, src]
    s["lens"].clamp_max_(budget)


# --------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import block_sparse_attention_28_b200 as sta
    if op == "evict":
        torch._foreach_copy_([s["lens"], s["slot_pos"], s["weight"]], s["full"])
    if op == "step":
        s["lens"].add_(1)
        s["seen"].add_(1)
    if op in ("append", "step"):
        if own:
            sta.sta_cache_append(s["cache"], s["k_new"], s["v_new"], s["counts"])
        else:
            _plain_append(s)
    if op in ("evict", "step"):
        if own:
            sta.sta_cache_evict(s["cache"], c["budget"], c["recent"], c["sinks"], s["evict_ws"])
        else:
            _plain_evict(s, c["budget"], c["recent"], c["sinks"])
    if op in ("attend", "step"):
        accumulate = op == "step" or c["accumulate"]
        if own:
            sta.sta_attn_fwd_cached(s["cache"], s["q"], s["o"], s["lse"], s["attend_ws"], page_ptr=s["page_ptr"],
                                    page_idx=s["page_idx"], accumulate=accumulate)
        else:
            _plain_attend(s, accumulate)
    return _outputs(s)


def _outputs(s):
    op = s["case"]["op"]
    if op == "attend":
        return {"o": s["o"], "lse": s["lse"], "weight": s["weight"] if s["case"]["accumulate"] else None}
    got = {n: s[n] for n in ("k_pages", "v_pages", "lens", "slot_pos", "weight")}
    if op == "step":
        got.update(o=s["o"], lse=s["lse"])
    return got


# ------------------------------------------------------------------- work
def work(case):
    B, kv, d, op = case["B"], case["kv"], case["d"], case["op"]
    row = 2 * d  # bytes of one key or value
    if op == "append":
        tokens = sum(_ladder(case["least"], case["n"], B)) * kv
        return {"bytes": tokens * (4 * row + 8), "flops": 0}
    if op == "attend":
        lens = _ladder(case["lo"], case["hi"], B)
        tokens = 0
        for n in lens:
            have = _pages(n)
            tokens += n if case["pages"] >= 1 else min(n, PAGE * (1 + (have - 1) * case["pages"])) if n else 0
        tokens *= kv
        heads = kv * case["group"]
        io = B * case["n_q"] * heads * (2 * row + 4)
        return {"bytes": tokens * (2 * row + (8 if case["accumulate"] else 0)) + io,
                "flops": 4 * d * tokens * case["group"] * case["n_q"]}
    if op == "evict":
        total = 0
        for n in _ladder(case["lo"], case["hi"], B):
            if n > case["budget"]:
                total += n * 8 + _moves(n, case) * (4 * row + 8)
        return {"bytes": max(total, 4 * B) * kv, "flops": 0}
    n = case["budget"]
    rows = B * kv
    return {"bytes": rows * ((n + 1) * 8 + n * (2 * row + 8) + 4 * row + 8 + 4 * row + case["group"] * (2 * row + 4)),
            "flops": 4 * d * rows * case["group"] * n}


def _moves(n, case):
    """Tokens that move when a sequence of n is cut to the budget, with weights in no order."""
    budget, sinks, recent = case["budget"], min(case["sinks"], n), min(case["recent"], n)
    others = max(1, n - sinks - recent)
    share = max(0, budget - sinks - recent) / others  # of the others, how many stay
    below = max(0, min(budget, n - recent) - sinks)  # of the slots under the budget, those that hold others
    return below * (1 - share)


# ------------------------------------------------------------------ exact
def _rows_of(s, b, h, n):
    """Keys and values of slots 0 .. n - 1 of one head, in 64 bits."""
    pages = s["page_table"][b, :_pages(n)].long()
    k = s["k_pages"][pages, h].reshape(-1, s["k_pages"].shape[-1])[:n].double()
    v = s["v_pages"][pages, h].reshape(-1, s["v_pages"].shape[-1])[:n].double()
    return k, v


def _exact_attend(s, lens, group, accumulate, keep=None):
    q = s["q"].double()
    B, n_q, hq, d = q.shape
    o, lse = torch.zeros_like(q), torch.full((B, hq, n_q), -math.inf, device=q.device, dtype=torch.float64)
    weight = s["weight"].double() if accumulate else None
    for b in range(B):
        for h in range(hq // group):
            n = lens[b][h]
            if not n:
                continue
            k, v = _rows_of(s, b, h, n)
            x = torch.einsum("igd,jd->igj", q[b, :, h * group:(h + 1) * group], k) / math.sqrt(d)
            hidden = torch.arange(n, device=q.device)[None] > torch.arange(n - n_q, n, device=q.device)[:, None]
            if keep is not None:
                hidden = hidden | ~keep[b][h][:n][None]
            x = x.masked_fill(hidden[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z.nan_to_num(neginf=0.0)[..., None])
            o[b, :, h * group:(h + 1) * group] = torch.einsum("igj,jd->igd", p, v)
            lse[b, h * group:(h + 1) * group] = z.transpose(0, 1)
            if accumulate:
                weight[b, h, :n] += p.sum((0, 1))
    return o, lse, weight


def _exact_evict(s, budget, recent, sinks):
    """The kept set by sorting (safe, weight, slot) tuples row by row; lens, slot_pos and weight after it."""
    lens, pos, weight, seen = (s[n].cpu().numpy().copy() for n in ("lens", "slot_pos", "weight", "seen"))
    moved = {}
    for b in range(lens.shape[0]):
        for h in range(lens.shape[1]):
            n = int(lens[b, h])
            if n <= budget:
                continue
            p, w = pos[b, h, :n], weight[b, h, :n].astype("f8")
            safe = (p < sinks) | (p >= int(seen[b, h]) - recent)
            stay = sorted(range(n), key=list(zip((~safe).tolist(), (-w * ~safe).tolist(), range(n))).__getitem__)
            stay = set(stay[:budget])
            into = [j for j in range(budget) if j not in stay]
            come = sorted(j for j in stay if j >= budget)
            moved[b, h] = (into, come)
            pos[b, h, into] = pos[b, h, come]
            weight[b, h, into] = weight[b, h, come]
            lens[b, h] = budget
    return lens, pos, weight, moved


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "attend":
        keep = None
        B, kv = s["lens"].shape
        if s["page_ptr"] is not None:
            ptr, idx = s["page_ptr"].tolist(), s["page_idx"]
            keep = [[None] * kv for _ in range(B)]
            for r in range(B * kv):
                m = torch.zeros(s["page_table"].shape[1], device="cuda", dtype=torch.bool)
                m[idx[ptr[r]:ptr[r + 1]].long()] = True
                keep[r // kv][r % kv] = m.repeat_interleave(PAGE)
        o, lse, weight = _exact_attend(s, s["lens"].tolist(), case["group"], case["accumulate"], keep)
        return {"o": o, "lse": lse, "weight": weight}
    none = {"k_pages": None, "v_pages": None}  # what moves moves bit by bit
    if op == "append":
        weight = s["weight"].double()
        for b, n in enumerate(s["counts"].tolist()):
            for h, end in enumerate(s["lens"][b].tolist()):
                weight[b, h, end - n:end] = 0
        return dict(none, lens=None, slot_pos=None, weight=weight)
    rows = case["B"] * case["kv"]
    if rows * (case["hi"] if op == "evict" else case["budget"]) > 4_000_000:
        return None
    if op == "evict":
        lens, pos, weight, _ = _exact_evict(s, case["budget"], case["recent"], case["sinks"])
        return dict(none, lens=lens, slot_pos=pos, weight=weight.astype("f8"))
    # a step: the token is appended by hand, the kept ones chosen, then attention over what is left
    n = case["budget"] + 1
    B, kv = s["lens"].shape
    s["lens"].fill_(n)
    s["seen"].fill_(n)
    for b in range(B):
        page = int(s["page_table"][b, (n - 1) // PAGE])
        s["k_pages"][page, :, (n - 1) % PAGE] = s["k_new"][b, 0]
        s["v_pages"][page, :, (n - 1) % PAGE] = s["v_new"][b, 0]
    s["slot_pos"][:, :, n - 1] = n - 1
    s["weight"][:, :, n - 1] = 0
    lens, pos, weight, moved = _exact_evict(s, case["budget"], case["recent"], case["sinks"])
    for (b, h), (into, come) in moved.items():
        table = s["page_table"][b].tolist()
        for x, y in zip(into, come):
            for pool in (s["k_pages"], s["v_pages"]):
                pool[table[x // PAGE], h, x % PAGE] = pool[table[y // PAGE], h, y % PAGE]
    s["weight"].copy_(torch.from_numpy(weight))
    o, lse, w = _exact_attend(s, lens.tolist(), case["group"], True)
    return dict(none, lens=lens, slot_pos=pos, weight=w, o=o, lse=lse)
