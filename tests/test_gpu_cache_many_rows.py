"""Calls on many (sequence, head) rows: several rows to a thread of the
attention's prefix over the lengths, several trips of an append's CTAs."""
import numpy as np
import pytest
import torch

import _cache as C
from oracle import kv_cache as K
from test_gpu_cache import attend, cache_of, compare, ok, sta  # noqa: F401

pytestmark = pytest.mark.gpu


def lengths(B, kv, seed, most):
    """Lengths per head, most of them 0, in runs too."""
    rng = np.random.default_rng(seed)
    n = rng.integers(1, most + 1, size=(B, kv)) * (rng.random((B, kv)) < 0.3)
    n[B // 3:B // 3 + B // 4] = 0
    n[-1, -1] = most
    return [tuple(int(x) for x in row) for row in n]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("B,kv,group,n_q,d,dtype", [
    (30, 10, 1, 1, 64, "bf16"),     # 300 rows: two to a thread
    (30, 10, 4, 3, 128, "fp16"),
    (64, 40, 1, 1, 64, "bf16"),     # 2,560: twelve
    (61, 37, 2, 1, 64, "fp16"),     # 2,257: ten or eleven, the last threads with fewer or none
])
def test_attention_over_many_rows(sta, B, kv, group, n_q, d, dtype, accumulate):  # noqa: F811
    t = C.make(lengths(B, kv, B, 130), kv, d, dtype, seed=B, max_pages=5)
    compare(sta, t, C.queries(B, n_q, kv * group, d, dtype, seed=3), dtype, accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("B,kv", [(30, 10), (64, 40)])
def test_page_lists_of_many_rows(sta, B, kv, accumulate):  # noqa: F811
    lens = lengths(B, kv, B + 1, 200)
    t = C.make(lens, kv, 64, "bf16", seed=B, max_pages=5)
    rng = np.random.default_rng(B)
    lists = [[[p for p in range(-(-n // C.PAGE)) if rng.random() < 0.6] for n in heads] for heads in lens]
    compare(sta, t, C.queries(B, 1, kv, 64, "bf16", seed=4), "bf16", lists, accumulate)


@pytest.mark.parametrize("d,dtype,n", [(64, "bf16", 300), (128, "fp16", 170)])
def test_a_padded_append_of_many_sequences(sta, d, dtype, n):  # noqa: F811
    """200 sequences of 0 to n new rows (a CTA has several blocks of them), one
    count out of range and one head whose length is below the count."""
    B, kv = 200, 8
    rng = np.random.default_rng(n)
    counts = (rng.integers(0, n + 1, size=B) * (rng.random(B) < 0.1) + rng.integers(0, 3, size=B)).clip(0, n)
    counts[7], counts[90], counts[B - 1] = n, 40, n - 1
    before = rng.integers(0, 70, size=B)
    t = C.make([int(x) for x in before + counts], kv, d, dtype, seed=1)
    t["seen"] += 500
    c = C.oracle(t)
    new = [C.queries(B, n, kv, d, dtype, seed=s) for s in (1, 2)]
    given = counts.copy()
    given[33] = n + 1
    counts[33] = 0
    t["lens"][90, 5] = 39
    left = [(name, int(p), c[name][int(p), 5].copy()) for p in c["page_table"][90] if p >= 0
            for name in ("k_pages", "v_pages")]
    spared = {name: c[name][90, 5].copy() for name in ("slot_pos", "weight")}
    sta.sta_cache_append(cache_of(sta, t), *new, counts=torch.tensor(given, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert sta.sta_get_device_error() == sta.STA_ERR_BAD_CACHE
    K.append(c, *(x.double().cpu().numpy() for x in new), counts=counts)
    for name, p, was in left:
        c[name][p, 5] = was
    for name, was in spared.items():
        c[name][90, 5] = was
    c["lens"][90, 5] = 39
    C.same_as(t, c)
