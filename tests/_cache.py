"""Caches of the tests: the same one as torch tensors (on any device) and as
the oracle's numpy arrays."""
import numpy as np
import torch

PAGE = 64
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# half a step of the type, relative to the value
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
# relative error of a weight split in two terms of the type
SPLIT = {"bf16": 2.0 ** -16, "fp16": 2.0 ** -22}


def make(lens, kv, d, dtype, seed, room=0, spare=2, device="cuda", tracked=True, poison=True, max_pages=None):
    """Tensors of a cache whose sequence b holds lens[b] slots (an int, or one
    for each head) and has pages for `room` more; every slot no call may look
    at holds NaN or an infinity (poison)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per_head = torch.tensor([[n] * kv if isinstance(n, int) else list(n) for n in lens], dtype=torch.int32)
    need = [max(1, -(-(int(per_head[b].max()) + room) // PAGE)) for b in range(B)]
    width = max_pages or max(need) + 1
    num = sum(need) + spare
    order = torch.randperm(num, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    t = {"k_pages": torch.randn(num, kv, PAGE, d, generator=g), "v_pages": torch.randn(num, kv, PAGE, d, generator=g)}
    if poison:
        used = torch.zeros(num, kv, PAGE, dtype=torch.bool)
        for b in range(B):
            for h in range(kv):
                for j in range(int(per_head[b, h])):
                    used[table[b, j // PAGE], h, j % PAGE] = True
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.randint(0, 3, (num, kv, PAGE, 1),
                                                                                    generator=g)]
        for n in ("k_pages", "v_pages"):
            t[n] = torch.where(used[..., None], t[n], bad)
    t = {n: x.to(DT[dtype]).to(device) for n, x in t.items()}
    t.update(page_table=table.to(device), lens=per_head.to(device), seen=None, slot_pos=None, weight=None)
    if tracked:
        slots = PAGE * width
        t["seen"] = per_head.clone().to(device)
        t["slot_pos"] = torch.arange(slots, dtype=torch.int32).expand(B, kv, slots).contiguous().to(device)
        t["weight"] = torch.rand(B, kv, slots, generator=g).to(device)
    return t


def oracle(t):
    """The oracle's copy of a cache."""
    c = {}
    for n, x in t.items():
        if x is None:
            c[n] = None
        else:
            x = x.detach().cpu()
            c[n] = x.double().numpy() if x.is_floating_point() else x.numpy().copy()
    return c


def bits(x):
    return x.detach().cpu().view(torch.int16 if x.element_size() == 2 else torch.int32)


def same_as(t, c, names=("k_pages", "v_pages", "lens", "seen", "slot_pos", "weight")):
    """Every array of the cache equal to the oracle's, value for value (NaN in
    the same places)."""
    for n in names:
        if t[n] is None:
            continue
        x = t[n].detach().cpu()
        x = x.double().numpy() if x.is_floating_point() else x.numpy()
        assert np.array_equal(x, c[n], equal_nan=x.dtype.kind == "f"), n


def queries(B, n_q, heads, d, dtype, seed, scale=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, n_q, heads, d, generator=g) * scale).to(DT[dtype]).to(device)


def check_attention(o, lse, want, d, dtype, most_slots):
    """o and lse against the oracle's (o, lse, sigma, terms). With
    u = 2^-24 (half a step of fp32):
      a score is a sum of d products in fp32, each addition off by at most one
      step (the tensor cores cut off instead of rounding) of a partial sum,
      itself at most `terms`: ds = 2 d u terms; times scale and log2 e, the
      subtraction of the maximum and the exponential (2 ulp): 16 u more,
      relative to terms + 1;
      weights are then off by a factor of 1 +- 2 (ds + 16 u (terms + 1)), the
      sums over n slots by n u (numerator and denominator: 2 n u) more, the
      split by SPLIT, and o is rounded once."""
    want_o, want_lse, sigma, terms = want
    u = 2.0 ** -24
    ds = 2 * d * u * terms + 16 * u * (terms + 1)
    rel = 2 * ds + 2 * most_slots * u + 2 * SPLIT[dtype]
    rel_o = np.moveaxis(rel, 1, 2)[..., None]
    got = o.detach().cpu().double().numpy()
    tiny = {"bf16": 0.0, "fp16": 2.0 ** -25}[dtype]  # half a step of fp16's subnormals
    limit = sigma * rel_o + (np.abs(want_o) + sigma * rel_o) * HALF[dtype] + tiny
    err = np.abs(got - want_o)
    assert np.isfinite(got).all()
    assert (err <= limit).all(), (err - limit).max()
    if lse is not None:
        got = lse.detach().cpu().double().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(want_lse))
        at = np.isfinite(want_lse)
        limit = ds + most_slots * u + 4 * u * (np.abs(np.where(at, want_lse, 0.0)) + 1)
        assert (np.abs(got - np.where(at, want_lse, 0.0))[at] <= limit[at]).all()
    return rel


def check_weight(t, c, before, rel, queries_per_slot):
    """weight against the oracle's: what was added is off by at most rel of
    itself, and each of queries_per_slot + 1 sums by half a step."""
    got, want = t["weight"].detach().cpu().double().numpy(), c["weight"]
    limit = (want - before) * float(np.max(rel)) + np.abs(want) * (queries_per_slot + 1) * 2.0 ** -24
    assert (np.abs(got - want) <= limit).all()
