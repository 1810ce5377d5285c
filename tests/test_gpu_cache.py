"""The paged key-value cache on the GPU, through the public calls, against the
fp64 oracle: append (bit for bit), attention over the cache and the weight it
accumulates (within bounds derived in _cache.check_attention), eviction (bit
for bit), and the calls together."""
import numpy as np
import pytest
import torch

import _cache as C
from oracle import kv_cache as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sta():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_sparse_attention_28_b200 as mod

    return mod


def cache_of(sta, t):
    return sta.kv_cache(**t)


def ok(sta):
    torch.cuda.synchronize()
    assert sta.sta_get_device_error() == sta.STA_OK


def garbage(n):
    """A workspace in which nothing starts at zero."""
    return torch.full((max(n, 1),), 0xA7, dtype=torch.uint8, device="cuda")


def attend(sta, t, q, lists=None, accumulate=False, sm_scale=0.0, stream=None, with_lse=True):
    cache = cache_of(sta, t)
    B, n_q, hq, _ = q.shape
    o = torch.full_like(q, 7.0)
    lse = torch.full((B, hq, n_q), 7.0, device="cuda") if with_lse else None
    ws = garbage(sta.sta_attn_fwd_cached_workspace(cache, hq, n_q, accumulate))
    ptr = idx = None
    if lists is not None:
        ptr, idx = csr(lists)
    sta.sta_attn_fwd_cached(cache, q, o, lse, ws, page_ptr=ptr, page_idx=idx, accumulate=accumulate,
                            sm_scale=sm_scale, stream=stream)
    return o, lse


def csr(lists):
    rows = [r for seq in lists for r in seq]
    ptr = torch.tensor(np.cumsum([0] + [len(r) for r in rows]), dtype=torch.int32, device="cuda")
    return ptr, torch.tensor([p for r in rows for p in r], dtype=torch.int32, device="cuda")


def compare(sta, t, q, dtype, lists=None, accumulate=False, sm_scale=0.0):
    d = q.shape[-1]
    c = C.oracle(t)
    before = None if c["weight"] is None else c["weight"].copy()
    o, lse = attend(sta, t, q, lists, accumulate, sm_scale)
    ok(sta)
    want = K.attend(c, q.double().cpu().numpy(), sm_scale or d ** -0.5, lists, accumulate)
    rel = C.check_attention(o, lse, want, d, dtype, int(c["lens"].max(initial=0)))
    if accumulate:
        C.check_weight(t, c, before, rel, q.shape[1] * (q.shape[2] // c["lens"].shape[1]))
    return o, lse


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("d,dtype,kv,lens,counts", [
    (64, "bf16", 2, [5, 64, 200], [5, 1, 70]),
    (128, "fp16", 3, [1, 63, 130], [0, 63, 129]),
    (128, "bf16", 1, [64], [64]),
    (64, "fp16", 10, [128, 65], None),
    (128, "bf16", 40, [300], None),
])
def test_append_writes_the_new_slots_and_nothing_else(sta, d, dtype, kv, lens, counts):
    n = max(counts) if counts else 65
    t = C.make(lens, kv, d, dtype, seed=d + kv)
    t["seen"] += 1000  # positions do not start at the slot's number
    c = C.oracle(t)
    new = [C.queries(len(lens), n, kv, d, dtype, seed=s) for s in (1, 2)]
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    sta.sta_cache_append(cache_of(sta, t), *new, counts=cnt)
    ok(sta)
    K.append(c, *(x.double().cpu().numpy() for x in new), counts=counts)
    C.same_as(t, c)
    sta.sta_cache_append(cache_of(sta, t), *new, counts=cnt)  # changes no length: the same again
    ok(sta)
    C.same_as(t, c)


def test_append_without_positions_and_weights(sta):
    t = C.make([70, 3], 2, 64, "bf16", seed=1, tracked=False)
    c = C.oracle(t)
    new = [C.queries(2, 3, 2, 64, "bf16", seed=s) for s in (1, 2)]
    sta.sta_cache_append(cache_of(sta, t), *new)
    ok(sta)
    K.append(c, *(x.double().cpu().numpy() for x in new))
    C.same_as(t, c)


def test_append_leaves_out_what_does_not_fit(sta):
    """A count past the rows given or past the length, a length past the page
    table and a page outside the pool: recorded, the rest written."""
    t = C.make([10, 10, 10, 10], 2, 64, "bf16", seed=2)
    t["lens"][1, 1] = 2  # fewer than it is said to have got
    t["lens"][2, 0] = C.PAGE * t["page_table"].shape[1] + 1
    t["page_table"][3, 0] = t["k_pages"].shape[0]
    before = {n: x.clone() for n, x in t.items()}
    c = C.oracle(t)
    counts = torch.tensor([5, 3, 3, 3], dtype=torch.int32, device="cuda")
    new = [C.queries(4, 4, 2, 64, "bf16", seed=s) for s in (1, 2)]
    sta.sta_cache_append(cache_of(sta, t), *new, counts=counts)
    torch.cuda.synchronize()
    assert sta.sta_get_device_error() == sta.STA_ERR_BAD_CACHE
    for n in ("lens", "seen"):
        assert torch.equal(t[n], before[n])
    for b, h in ((0, 0), (0, 1), (1, 1), (2, 0)):
        page = int(t["page_table"][b, 0])
        for n in ("k_pages", "v_pages"):
            assert torch.equal(C.bits(t[n][page, h]), C.bits(before[n][page, h]))
    c["lens"][1, 1] = c["lens"][2, 0] = 10  # the oracle writes those too; only the other heads are looked at
    for b, h in ((1, 0), (2, 1)):
        one = {n: (x if x is None or n.endswith("pages") else x[b:b + 1]) for n, x in c.items()}
        K.append(one, *(x[b:b + 1].double().cpu().numpy() for x in new), counts=[3])
        page = int(t["page_table"][b, 0])
        assert np.array_equal(t["k_pages"][page, h].double().cpu().numpy(), c["k_pages"][page, h], equal_nan=True)
    owned = t["page_table"].cpu().unique().tolist()
    for p in range(t["k_pages"].shape[0]):
        if p not in owned:
            assert torch.equal(C.bits(t["k_pages"][p]), C.bits(before["k_pages"][p]))
    assert sta.sta_get_device_error() == sta.STA_OK


# ---------------------------------------------------------------- attention
LENGTHS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 700]


# columns of the page table: as many as the lengths need (few and short rows: a
# cluster of CTAs each), or so many that the rows are shared out in chunks
@pytest.mark.parametrize("max_pages", [None, 700])
@pytest.mark.parametrize("d,dtype,kv,group,n_q", [
    (64, "bf16", 2, 1, 1), (128, "bf16", 1, 4, 1), (128, "fp16", 2, 8, 1), (64, "fp16", 1, 5, 3),
    (128, "bf16", 3, 1, 7), (64, "bf16", 1, 16, 4), (128, "fp16", 1, 1, 64), (128, "bf16", 2, 3, 9),
    (128, "bf16", 1, 64, 1), (64, "fp16", 2, 17, 1), (64, "bf16", 8, 1, 1), (128, "fp16", 12, 2, 1), (64, "fp16", 5, 2, 1),
    (64, "bf16", 2, 8, 4), (64, "fp16", 1, 11, 3), (64, "bf16", 1, 3, 16),
])
def test_attention_of_every_length(sta, d, dtype, kv, group, n_q, max_pages):
    t = C.make(LENGTHS, kv, d, dtype, seed=d + group + n_q, max_pages=max_pages)
    q = C.queries(len(LENGTHS), n_q, kv * group, d, dtype, seed=3, scale=1.5)
    compare(sta, t, q, dtype)


@pytest.mark.parametrize("d,dtype,kv,group,n_q", [
    (64, "bf16", 2, 1, 1), (128, "bf16", 1, 4, 1), (128, "fp16", 2, 8, 1), (64, "fp16", 1, 5, 3),
    (128, "bf16", 1, 1, 40), (64, "bf16", 2, 4, 5), (64, "fp16", 1, 8, 4), (64, "bf16", 1, 16, 3),
])
def test_accumulated_weight(sta, d, dtype, kv, group, n_q):
    t = C.make(LENGTHS, kv, d, dtype, seed=d + group + n_q)
    q = C.queries(len(LENGTHS), n_q, kv * group, d, dtype, seed=4, scale=1.5)
    compare(sta, t, q, dtype, accumulate=True)


def test_accumulation_does_not_change_the_output(sta):
    """Of rows shared out in chunks (short ones take other sums without it)."""
    t = C.make(LENGTHS, 2, 128, "fp16", seed=138, max_pages=700)
    q = C.queries(len(LENGTHS), 1, 16, 128, "fp16", seed=4, scale=1.5)
    o1, lse1 = attend(sta, t, q, accumulate=True)
    o2, lse2 = attend(sta, t, q)
    ok(sta)
    assert torch.equal(C.bits(o1), C.bits(o2)) and torch.equal(lse1, lse2)


def test_heads_of_different_lengths(sta):
    t = C.make([(3, 0, 130), (64, 65, 1)], 3, 128, "bf16", seed=5)
    compare(sta, t, C.queries(2, 2, 6, 128, "bf16", seed=5), "bf16", accumulate=True)


@pytest.mark.parametrize("accumulate,max_pages", [(False, None), (False, 700), (True, None)])
def test_page_lists(sta, accumulate, max_pages):
    """Lists of some pages, of all, of none; the last page listed or not."""
    lens = [700, 700, 64, 0, 1000]
    t = C.make(lens, 2, 128, "bf16", seed=6, max_pages=max_pages)
    lists = [[[0, 3, 10], []], [list(range(11)), [5]], [[0], []], [[], []], [[14, 15], [0, 1, 2, 7, 9, 13]]]
    q = C.queries(5, 3, 4, 128, "bf16", seed=6)
    compare(sta, t, q, "bf16", lists, accumulate)


def test_empty_lists_of_every_head(sta):
    t = C.make([100, 5], 2, 64, "bf16", seed=7)
    q = C.queries(2, 1, 2, 64, "bf16", seed=7)
    o, lse = compare(sta, t, q, "bf16", [[[], []], [[], []]], True)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("accumulate", [False, True])
def test_bad_list_entries_are_left_out(sta, accumulate):
    """The same index twice, one out of order, one past the last page, a
    negative one: recorded, the others attended to."""
    t = C.make([300, 300], 2, 64, "bf16", seed=8)
    c = C.oracle(t)
    before = c["weight"].copy()
    q = C.queries(2, 1, 2, 64, "bf16", seed=8)
    given = [[[1, 1, 3], [2, 1, 4]], [[0, 5], [-1, 0]]]
    o, lse = attend(sta, t, q, given, accumulate)
    torch.cuda.synchronize()
    assert sta.sta_get_device_error() == sta.STA_ERR_BAD_MASK
    want = K.attend(c, q.double().cpu().numpy(), 64 ** -0.5, [[[1, 3], [2, 4]], [[0], [0]]], accumulate)
    rel = C.check_attention(o, lse, want, 64, "bf16", 300)
    C.check_weight(t, c, before, rel, 1)


@pytest.mark.parametrize("ptr", [[0, 2, 1, 3, 4], [0, 1, 2, 3, 99], [-3, 1, 2, 3, 4], [3, 2, 1, 0, -1]])
@pytest.mark.parametrize("accumulate", [False, True])
def test_bad_list_offsets(sta, ptr, accumulate):
    """Offsets that decrease, pass the entries or are negative: recorded, and
    nothing past the given entries is looked at; the outputs are finite."""
    t = C.make([300, 300], 2, 64, "bf16", seed=8)
    q = C.queries(2, 1, 2, 64, "bf16", seed=8)
    cache = cache_of(sta, t)
    o, lse = torch.zeros_like(q), torch.zeros(2, 2, 1, device="cuda")
    ws = garbage(sta.sta_attn_fwd_cached_workspace(cache, 2, 1, accumulate))
    sta.sta_attn_fwd_cached(cache, q, o, lse, ws, page_ptr=torch.tensor(ptr, dtype=torch.int32, device="cuda"),
                            page_idx=torch.arange(4, dtype=torch.int32, device="cuda"), accumulate=accumulate)
    torch.cuda.synchronize()
    assert sta.sta_get_device_error() == sta.STA_ERR_BAD_MASK
    assert torch.isfinite(o.float()).all() and torch.isfinite(t["weight"]).all()


@pytest.mark.parametrize("accumulate", [False, True])
def test_bad_pages_and_lengths_are_left_out(sta, accumulate):
    t = C.make([200, 200, 200, 10], 1, 64, "bf16", seed=9)
    c = C.oracle(t)
    q = C.queries(4, 1, 1, 64, "bf16", seed=9)
    t["page_table"][0, 1] = t["k_pages"].shape[0] + 5
    t["page_table"][1, 3] = -1
    t["lens"][3, 0] = -7
    t["lens"][2, 0] = 1 << 29
    c["lens"][2, 0] = c["lens"][3, 0] = 0
    before = c["weight"].copy()
    o, lse = attend(sta, t, q, accumulate=accumulate)
    torch.cuda.synchronize()
    assert sta.sta_get_device_error() == sta.STA_ERR_BAD_CACHE
    want = K.attend(c, q.double().cpu().numpy(), 64 ** -0.5, [[[0, 2, 3]], [[0, 1, 2]], [[]], [[]]], accumulate)
    rel = C.check_attention(o, lse, want, 64, "bf16", 200)
    C.check_weight(t, c, before, rel, 1)


def test_non_finite_values_of_a_newer_token(sta):
    """Draft token 2's value and key are infinite / NaN: queries 0 and 1, who
    do not see it, are not touched; query 3, who does, gets what the formula
    gives."""
    for bad in (float("inf"), float("nan")):
        t = C.make([66, 130], 2, 64, "bf16", seed=10)
        q = C.queries(2, 4, 4, 64, "bf16", seed=10)
        for b, n in ((0, 66), (1, 130)):
            j = n - 2  # of the newest four, number 2
            page = int(t["page_table"][b, j // C.PAGE])
            t["v_pages"][page, :, j % C.PAGE, 5] = bad
        c = C.oracle(t)
        o, lse = attend(sta, t, q)
        ok(sta)
        assert torch.isfinite(o[:, :2].float()).all() and torch.isfinite(lse).all()
        with np.errstate(invalid="ignore"):
            want = K.attend(c, q.double().cpu().numpy(), 64 ** -0.5)
        got = o.double().cpu().numpy()
        assert np.array_equal(np.isfinite(got), np.isfinite(want[0]))
        early = tuple(x[:, :2] if x.ndim == 4 else x[:, :, :2] for x in want)
        C.check_attention(o[:, :2], lse[:, :, :2], early, 64, "bf16", 130)


@pytest.mark.parametrize("d,group,n_q,kv", [(64, 1, 4, 2), (128, 5, 3, 1), (128, 4, 6, 1), (64, 8, 8, 1),
                                            (128, 1, 64, 1), (64, 4, 6, 1)])
@pytest.mark.parametrize("max_pages", [None, 700])
@pytest.mark.parametrize("what", ["k_pages", "v_pages"])
def test_non_finite_draft_tokens(sta, d, group, n_q, kv, what, max_pages):
    """Every second one of the newest tokens has a key or a value that is not
    finite: a query is touched by those it sees and by no others, whatever
    page and piece of a page they lie in."""
    lens = [n_q, 33, 64, 65, 70, 96, 127, 200]
    t = C.make(lens, kv, d, "bf16", seed=50 + n_q, max_pages=max_pages)
    q = C.queries(len(lens), n_q, kv * group, d, "bf16", seed=51)
    for b, n in enumerate(lens):
        for i in range(1, n_q, 2):
            j = n - n_q + i
            if j >= 0:
                page = int(t["page_table"][b, j // C.PAGE])
                t[what][page, :, j % C.PAGE, (7 * i) % d] = float("nan")
    c = C.oracle(t)
    o, lse = attend(sta, t, q)
    ok(sta)
    got = o.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, want_lse, sigma, terms = K.attend(c, q.double().cpu().numpy(), d ** -0.5)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = torch.from_numpy(~np.isnan(want))
    zero = lambda x: np.where(np.isnan(x), 0.0, x)  # noqa: E731
    rows = ~np.isnan(want).any(-1)  # [B, n_q, heads]: nothing but finite outputs
    C.check_attention(torch.where(fine & torch.from_numpy(rows)[..., None], o.cpu().float(), torch.tensor(0.0)), None,
                      (zero(want) * rows[..., None], zero(want_lse), zero(sigma) * rows[..., None], zero(terms)), d,
                      "bf16", 200)
    if what == "k_pages":
        assert np.array_equal(np.isnan(lse.cpu().numpy()), np.isnan(want_lse))


def test_a_wait_that_runs_out_is_reported(sta):
    """With a limit far below a load's latency (every SM fetching from a cache
    four times the size of L2) waits give up: the call says so, ends, and the
    next one is as ever."""
    for d, group, n_q in ((128, 1, 1), (64, 8, 1), (128, 4, 5), (64, 8, 8)):
        kv, B = 2, 8
        pages = (256 << 20) // (kv * C.PAGE * d * 2)  # 256 MB of keys, as much of values
        k, v = (torch.randn(pages, kv, C.PAGE, d, device="cuda").bfloat16() for _ in range(2))
        width = pages // B
        table = torch.randperm(pages, device="cuda")[:B * width].int().reshape(B, width).contiguous()
        lens = torch.full((B, kv), C.PAGE * width - 5, dtype=torch.int32, device="cuda")
        lens[3] = 0
        t = {"k_pages": k, "v_pages": v, "page_table": table, "lens": lens, "seen": None, "slot_pos": None,
             "weight": torch.zeros(B, kv, C.PAGE * width, device="cuda")}
        q = C.queries(B, n_q, kv * group, d, "bf16", seed=61)
        first = attend(sta, t, q, accumulate=True)
        ok(sta)
        weight = t["weight"].clone()
        try:
            sta.sta_set_wait_limit(1000)
            attend(sta, t, q, accumulate=True)
            torch.cuda.synchronize()
            assert sta.sta_get_device_error() == sta.STA_ERR_TIMEOUT
        finally:
            sta.sta_set_wait_limit(0)
        t["weight"].zero_()
        again = attend(sta, t, q, accumulate=True)
        ok(sta)
        assert torch.equal(C.bits(first[0]), C.bits(again[0])) and torch.equal(first[1], again[1])
        assert torch.equal(t["weight"], weight)


def test_a_wait_that_runs_out_in_a_cluster(sta):
    """The same for short rows, whose CTAs wait for one another as well: every
    SM fetches its 14 pages at once from a cache that has been driven out of
    L2 (58 MB: some 9 us, 16 times the limit)."""
    B, kv, d, n = 16, 8, 128, 850
    k, v = (torch.randn(B * 14, kv, C.PAGE, d, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(B * 14, device="cuda").int().reshape(B, 14)
    t = {"k_pages": k, "v_pages": v, "page_table": table, "seen": None, "slot_pos": None, "weight": None,
         "lens": torch.full((B, kv), n, dtype=torch.int32, device="cuda")}
    q = C.queries(B, 1, kv * 4, d, "bf16", seed=63)
    first = attend(sta, t, q)
    ok(sta)
    try:
        sta.sta_set_wait_limit(1000)
        torch.empty(512 << 20, dtype=torch.uint8, device="cuda").fill_(1)
        attend(sta, t, q)
        torch.cuda.synchronize()
        assert sta.sta_get_device_error() == sta.STA_ERR_TIMEOUT
    finally:
        sta.sta_set_wait_limit(0)
    again = attend(sta, t, q)
    ok(sta)
    assert torch.equal(C.bits(first[0]), C.bits(again[0])) and torch.equal(first[1], again[1])


def test_large_scores_and_a_given_scale(sta):
    """Scores of some hundreds: the maximum is taken off before the
    exponential; and one key far above the others."""
    t = C.make([500, 65], 2, 128, "bf16", seed=11)
    q = C.queries(2, 1, 4, 128, "bf16", seed=11, scale=30.0)
    compare(sta, t, q, "bf16")
    compare(sta, t, q, "bf16", sm_scale=0.003)
    t = C.make([3000], 1, 128, "fp16", seed=12)
    q = C.queries(1, 1, 2, 128, "fp16", seed=12, scale=4.0)
    compare(sta, t, q, "fp16", accumulate=True)


def test_a_long_row_and_many_short_ones(sta):
    t = C.make([9000] + [i % 70 for i in range(40)], 2, 64, "bf16", seed=13)
    compare(sta, t, C.queries(41, 1, 4, 64, "bf16", seed=13), "bf16", accumulate=True)


@pytest.mark.parametrize("d,dtype,group,n_q", [(128, "bf16", 1, 1), (64, "fp16", 4, 1), (128, "fp16", 9, 2),
                                               (64, "bf16", 8, 3), (128, "bf16", 7, 9), (64, "fp16", 64, 1)])
def test_many_pages_to_a_cta(sta, d, dtype, group, n_q):
    """Rows of thousands of pages (read again and again from a few): the ring
    of pages goes round many times, for every number of query rows."""
    n = [300_017, 200_000]
    t = C.make([640, 640], 1, d, dtype, seed=40)
    few = t["page_table"][:, :10]
    g = torch.Generator().manual_seed(41)
    cols = [few[b].cpu()[torch.randint(0, 10, (5000,), generator=g)] for b in range(2)]
    t["page_table"] = torch.stack(cols).cuda().contiguous()
    t["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    t["seen"], t["slot_pos"] = None, None
    t["weight"] = torch.rand(2, 1, 5000 * C.PAGE, device="cuda")
    before = t["weight"].double()
    q = C.queries(2, n_q, group, d, dtype, seed=42)
    o, lse = attend(sta, t, q, accumulate=True)
    ok(sta)
    want = [torch.zeros(2, n_q, group, d, dtype=torch.float64, device="cuda") for _ in range(2)]
    want += [torch.zeros(2, group, n_q, dtype=torch.float64, device="cuda") for _ in range(2)]
    added = torch.zeros_like(before)
    for b in range(2):
        pages = t["page_table"][b].long()
        k = t["k_pages"][pages, 0].reshape(-1, d)[:n[b]].double()
        v = t["v_pages"][pages, 0].reshape(-1, d)[:n[b]].double()
        for i in range(n_q):
            m = n[b] - (n_q - 1 - i)
            x = q[b, i].double() @ k[:m].T * d ** -0.5
            p = x.softmax(-1)
            want[0][b, i], want[1][b, i] = p @ v[:m], p @ v[:m].abs()
            want[2][b, :, i] = x.logsumexp(-1)
            want[3][b, :, i] = (q[b, i].double().abs() @ k[:m].T.abs()).amax(-1) * d ** -0.5
            added[b, 0, :m] += p.sum(0)
    order = (0, 2, 1, 3)  # o, lse, sigma, terms
    # additions one after another: at most 5000 / 148 pages of a CTA, 32 slots each, and the 148 parts
    rel = C.check_attention(o, lse, [want[x].cpu().numpy() for x in order], d, dtype, 34 * 32 + 148)
    limit = added * float(rel.max()) + (before + added) * (group * n_q + 1) * 2.0 ** -24
    assert ((t["weight"].double() - before - added).abs() <= limit).all()


def test_every_sequence_empty(sta):
    t = C.make([0, 0, 0], 2, 128, "fp16", seed=14)
    o, lse = compare(sta, t, C.queries(3, 2, 2, 128, "fp16", seed=14), "fp16", accumulate=True)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_attention_without_lse_and_without_tracking(sta):
    t = C.make([100, 200], 2, 64, "bf16", seed=15, tracked=False)
    q = C.queries(2, 1, 2, 64, "bf16", seed=15)
    o1, _ = attend(sta, t, q)
    o2, _ = attend(sta, t, q, with_lse=False)
    ok(sta)
    assert torch.equal(C.bits(o1), C.bits(o2))


def test_offsets_past_32_bits(sta):
    """Pools of over 2^31 values (4.3 GB each), the sequence in their last
    pages."""
    kv, d = 8, 128
    num = (1 << 31) // (kv * C.PAGE * d) + 40
    k = torch.empty(num, kv, C.PAGE, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[-40:].normal_()
    v[-40:].normal_()
    t = {"k_pages": k, "v_pages": v, "page_table": torch.arange(num - 1, num - 11, -1, dtype=torch.int32, device="cuda")[None],
         "lens": torch.full((1, kv), 600, dtype=torch.int32, device="cuda"), "seen": None, "slot_pos": None,
         "weight": None}
    small = dict(t, k_pages=k[-40:].contiguous(), v_pages=v[-40:].contiguous(),
                 page_table=(t["page_table"] - (num - 40)).contiguous())
    q = C.queries(1, 1, kv, d, "bf16", seed=16)
    new = [C.queries(1, 3, kv, d, "bf16", seed=s) for s in (1, 2)]
    outs = []
    for one in (t, small):
        sta.sta_cache_append(cache_of(sta, one), *new)
        outs.append(attend(sta, one, q))
    ok(sta)
    assert torch.equal(C.bits(outs[0][0]), C.bits(outs[1][0])) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(C.bits(t["k_pages"][-40:]), C.bits(small["k_pages"]))


def test_attention_is_deterministic_and_splits_do_not_show(sta):
    """The same call again is bit-identical; the same tokens in other pages too."""
    t = C.make([5000, 77], 2, 128, "bf16", seed=17)
    q = C.queries(2, 1, 8, 128, "bf16", seed=17)
    first = attend(sta, t, q)
    again = attend(sta, t, q)
    perm = torch.randperm(t["k_pages"].shape[0], generator=torch.Generator().manual_seed(1)).cuda()
    moved = dict(t)
    for n in ("k_pages", "v_pages"):
        moved[n] = torch.empty_like(t[n])
        moved[n][perm] = t[n]
    moved["page_table"] = torch.where(t["page_table"] >= 0, perm[t["page_table"].long().clamp_min(0)].int(),
                                      t["page_table"])
    other = attend(sta, moved, q)
    ok(sta)
    for x in (again, other):
        assert torch.equal(C.bits(first[0]), C.bits(x[0])) and torch.equal(first[1], x[1])


# -------------------------------------------------------------------- evict
def evict(sta, t, budget, recent, sinks):
    cache = cache_of(sta, t)
    sta.sta_cache_evict(cache, budget, recent, sinks, garbage(sta.sta_cache_evict_workspace(cache, budget)))


def shuffled(t, seed):
    """Positions in any order, as an earlier eviction leaves them."""
    g = torch.Generator().manual_seed(seed)
    for b in range(t["lens"].shape[0]):
        for h in range(t["lens"].shape[1]):
            n = int(t["lens"][b, h])
            t["slot_pos"][b, h, :n] = torch.randperm(n, generator=g).int().cuda()
    return t


@pytest.mark.parametrize("d,dtype,lens,budget,recent,sinks", [
    (64, "bf16", [0, 1, 5, 64, 65, 300], 5, 2, 1),
    (128, "fp16", [300, 299, 301], 300, 10, 4),
    (128, "bf16", [200, 500], 64, 64, 0),
    (64, "fp16", [130], 1, 0, 0),
    (64, "bf16", [130], 1, 1, 0),
    (128, "bf16", [5000, 1024, 1025], 1024, 100, 16),
    (64, "bf16", [40, 50], 1000, 10, 10),
    (64, "bf16", [5000, 50], 6000, 10, 10),
    (128, "bf16", [5000, 5060, 4990], 5000, 10, 10),
])
def test_evict(sta, d, dtype, lens, budget, recent, sinks):
    for order in (False, True):
        t = C.make(lens, 3, d, dtype, seed=budget)
        if order:
            shuffled(t, budget)
        c = C.oracle(t)
        evict(sta, t, budget, recent, sinks)
        ok(sta)
        K.evict(c, budget, recent, sinks)
        C.same_as(t, c)
        evict(sta, t, budget, recent, sinks)  # nothing is over the budget now
        ok(sta)
        C.same_as(t, c)


def test_evict_equal_weights_go_by_slot(sta):
    t = C.make([700, 700, 2100], 2, 64, "bf16", seed=20)
    t["weight"][0] = 0.0
    t["weight"][1] = (torch.arange(t["weight"].shape[2], device="cuda") % 3).float()
    t["weight"][2] = torch.where(t["weight"][2] < 0.5, -0.0, 0.0)
    c = C.oracle(t)
    evict(sta, t, 200, 20, 3)
    ok(sta)
    K.evict(c, 200, 20, 3)
    C.same_as(t, c)


@pytest.mark.parametrize("lens,kv,budget,recent,sinks,ties", [
    ([20_000, 17_000, 300], 2, 5000, 700, 9, False),   # clusters of 2 CTAs, of 4 and of 8
    ([40_001], 1, 39_999, 5, 0, True),
    ([100_003, 64], 1, 20_000, 9000, 64, False),
    ([90_000], 3, 30_000, 0, 0, True),
    ([70_000], 200, 100, 10, 2, True),                # many rows: two CTAs, for the keys' sake
    ([400_000], 1, 150_000, 1000, 64, True),          # more keys than a cluster's memory holds
])
def test_evict_long_rows(sta, lens, kv, budget, recent, sinks, ties):
    """Rows shared out over a cluster of CTAs, with few equal weights and with
    hardly any others."""
    d, B = 64, len(lens)
    need = [-(-n // C.PAGE) for n in lens]
    num, width = sum(need), max(need)
    g = torch.Generator(device="cuda").manual_seed(budget)
    t = {n: torch.randint(-30000, 30000, (num, kv, C.PAGE, d), generator=g, device="cuda",
                          dtype=torch.int16).view(torch.bfloat16) for n in ("k_pages", "v_pages")}
    order = torch.randperm(num, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")[:, None].expand(B, kv).contiguous()
    w = torch.rand(B, kv, C.PAGE * width, generator=g, device="cuda")
    t.update(page_table=table, lens=length, seen=length.clone(), weight=(w * 3).floor() if ties else w,
             slot_pos=torch.rand(w.shape, generator=g, device="cuda").argsort(-1).int())
    want = {n: x.clone() for n, x in t.items()}
    evict(sta, t, budget, recent, sinks)
    ok(sta)
    for b in range(B):
        n = lens[b]
        if n <= budget:
            continue
        for h in range(kv):
            p, x = want["slot_pos"][b, h, :n], want["weight"][b, h, :n].double()
            safe = (p < sinks) | (p >= n - recent)
            key = torch.where(safe, 1e9, x)
            stay = torch.zeros(n, dtype=torch.bool, device="cuda")
            stay[torch.sort(key, descending=True, stable=True).indices[:budget]] = True
            to = (~stay[:budget]).nonzero()[:, 0]
            of = budget + stay[budget:].nonzero()[:, 0]
            for name in ("k_pages", "v_pages"):
                pool = want[name].view(torch.int16)
                pool[table[b, to // C.PAGE].long(), h, to % C.PAGE] = \
                    pool[table[b, of // C.PAGE].long(), h, of % C.PAGE]
            for name in ("slot_pos", "weight"):
                want[name][b, h, to] = want[name][b, h, of]
            want["lens"][b, h] = budget
    for name in ("k_pages", "v_pages"):
        assert torch.equal(t[name].view(torch.int16), want[name].view(torch.int16)), name
    for name in ("slot_pos", "weight", "lens", "seen"):
        assert torch.equal(t[name], want[name]), name


def test_evict_special_weights(sta):
    """Infinite, NaN, negative, subnormal weights; what is protected stays
    whatever its weight."""
    t = C.make([400], 4, 64, "bf16", seed=21)
    w = t["weight"]
    w[0, 0, ::7] = float("inf")
    w[0, 1, ::3] = float("nan")
    w[0, 2] = w[0, 2] - 0.5
    w[0, 2, 390:] = -float("inf")
    w[0, 3] = w[0, 3] * 1e-42
    c = C.oracle(t)
    evict(sta, t, 150, 30, 5)
    ok(sta)
    K.evict(c, 150, 30, 5)
    C.same_as(t, c)


def test_evict_with_more_protected_than_the_budget(sta):
    """Positions a caller's own rule made equal: the first slots of the
    protected stay."""
    t = C.make([300], 1, 64, "bf16", seed=22)
    t["slot_pos"].fill_(299)
    c = C.oracle(t)
    evict(sta, t, 100, 10, 0)
    ok(sta)
    K.evict(c, 100, 10, 0)
    C.same_as(t, c)


def test_evict_leaves_out_a_bad_page(sta):
    t = C.make([300], 1, 64, "bf16", seed=23)
    c = C.oracle(t)
    t["page_table"][0, 4] = -1
    K.evict(c, 100, 10, 0)
    evict(sta, t, 100, 10, 0)
    torch.cuda.synchronize()
    assert sta.sta_get_device_error() == sta.STA_ERR_BAD_CACHE
    C.same_as(t, c, ("lens", "slot_pos", "weight"))


# ----------------------------------------------------------------- together
@pytest.mark.parametrize("d,dtype,kv,group,budget", [(64, "bf16", 2, 4, 100), (128, "fp16", 3, 1, 64)])
def test_a_prompt_then_steps_with_eviction(sta, d, dtype, kv, group, budget):
    """A padded batch of prompts, then tokens one by one: append, evict,
    attend and accumulate, as a decoding loop runs them; the oracle goes on
    from the GPU's weights (sums in another order) after each step."""
    prompts = [130, 40, 5]
    t = C.make([0, 0, 0], kv, d, dtype, seed=30, room=200)
    t["weight"].zero_()
    c = C.oracle(t)
    steps = [prompts] + [[1, 1, 1]] * 8
    for k, counts in enumerate(steps):
        n = max(counts)
        new = [C.queries(3, n, kv, d, dtype, seed=100 * k + s) for s in (1, 2)]
        cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
        for x in ("lens", "seen"):
            t[x] += cnt[:, None]
            c[x] += np.array(counts, dtype=np.int32)[:, None]
        sta.sta_cache_append(cache_of(sta, t), *new, counts=cnt)
        K.append(c, *(x.double().cpu().numpy() for x in new), counts=counts)
        evict(sta, t, budget, 10, 2)
        ok(sta)
        K.evict(c, budget, 10, 2)
        C.same_as(t, c)
        compare(sta, t, C.queries(3, 1, kv * group, d, dtype, seed=k), dtype, accumulate=True)
        c["weight"] = t["weight"].double().cpu().numpy()


def test_captured_steps_follow_the_lengths(sta):
    """A step captured once and replayed: the lengths live on the device, so
    each replay appends one further and attends over one more; an eager call
    on the same cache in between does not disturb it."""
    kv, group, d = 2, 2, 64
    t = C.make([60, 10], kv, d, "bf16", seed=31, room=20)
    ref = {n: x.clone() for n, x in t.items()}
    k_new, v_new = (C.queries(2, 1, kv, d, "bf16", seed=s) for s in (1, 2))
    q = C.queries(2, 1, kv * group, d, "bf16", seed=3)

    def step(t, o, lse, ws, ews):
        cache = cache_of(sta, t)
        t["lens"].add_(1)
        t["seen"].add_(1)
        sta.sta_cache_append(cache, k_new, v_new)
        sta.sta_cache_evict(cache, 64, 5, 1, ews)
        sta.sta_attn_fwd_cached(cache, q, o, lse, ws, accumulate=True)

    def buffers(t):
        cache = cache_of(sta, t)
        return (torch.empty_like(q), torch.empty(2, kv * group, 1, device="cuda"),
                garbage(sta.sta_attn_fwd_cached_workspace(cache, kv * group, 1, True)),
                garbage(sta.sta_cache_evict_workspace(cache, 64)))

    mine, theirs = buffers(t), buffers(ref)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(t, *mine)
    for i in range(9):
        k_new.normal_()
        q.normal_()
        graph.replay()
        step(ref, *theirs)
        torch.cuda.synchronize()
        assert torch.equal(C.bits(mine[0]), C.bits(theirs[0])) and torch.equal(mine[1], theirs[1])
    ok(sta)
    assert t["lens"].tolist() == [[64, 64], [19, 19]]
    for n in ("lens", "seen", "slot_pos", "weight"):
        assert torch.equal(t[n], ref[n])
    assert torch.equal(C.bits(t["k_pages"]), C.bits(ref["k_pages"]))


def test_two_streams_at_once(sta):
    """Two attention calls on two streams, a workspace each, over one cache
    that neither writes; and a stream that is not the current one."""
    t = C.make([4000, 300], 2, 128, "bf16", seed=32)
    qs = [C.queries(2, 1, 8, 128, "bf16", seed=s) for s in (1, 2)]
    want = [attend(sta, t, q) for q in qs]
    torch.cuda.synchronize()
    cache = cache_of(sta, t)
    streams = [torch.cuda.Stream() for _ in qs]
    bufs = [(torch.empty_like(q), torch.empty(2, 8, 1, device="cuda"),
             garbage(sta.sta_attn_fwd_cached_workspace(cache, 8, 1))) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, (o, lse, ws) in zip(streams, qs, bufs):
            sta.sta_attn_fwd_cached(cache, q, o, lse, ws, stream=s)
    ok_all = [s.synchronize() for s in streams]
    assert len(ok_all) == 2
    ok(sta)
    for (o, lse, _), (wo, wl) in zip(bufs, want):
        assert torch.equal(C.bits(o), C.bits(wo)) and torch.equal(lse, wl)
