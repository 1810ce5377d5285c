"""Several new tokens at once over a cache whose slots are not in order of
position, as evictions leave it: each token sees those up to its own position,
wherever they lie. Against the fp64 oracle, which goes by position too."""
import numpy as np
import pytest
import torch

import _cache as C
from oracle import kv_cache as K
from test_gpu_cache import attend, cache_of, evict, garbage, ok, shuffled, sta  # noqa: F401

pytestmark = pytest.mark.gpu


def compare(sta, t, q, dtype, lists=None, accumulate=False):  # noqa: F811
    d = q.shape[-1]
    c = C.oracle(t)
    before = c["weight"].copy()
    o, lse = attend(sta, t, q, lists, accumulate)
    ok(sta)
    want = K.attend(c, q.double().cpu().numpy(), d ** -0.5, lists, accumulate, by_position=True)
    rel = C.check_attention(o, lse, want, d, dtype, int(c["lens"].max(initial=0)))
    if accumulate:
        C.check_weight(t, c, before, rel, q.shape[1] * (q.shape[2] // c["lens"].shape[1]))
    return o, lse, c


LENGTHS = [0, 1, 2, 5, 31, 32, 33, 64, 65, 130, 700]


# columns of the page table: few and short rows (a cluster of CTAs each, where
# nothing is accumulated) or rows shared out in chunks
@pytest.mark.parametrize("max_pages", [None, 700])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("d,dtype,kv,group,n_q", [
    (64, "bf16", 1, 1, 2), (128, "fp16", 2, 2, 4), (64, "fp16", 1, 2, 8), (128, "bf16", 1, 3, 5),
    (64, "bf16", 2, 8, 4), (128, "bf16", 1, 8, 4), (64, "fp16", 1, 1, 64), (128, "fp16", 1, 4, 16),
])
def test_slots_in_any_order(sta, d, dtype, kv, group, n_q, accumulate, max_pages):  # noqa: F811
    t = shuffled(C.make(LENGTHS, kv, d, dtype, seed=d + group + n_q, max_pages=max_pages), 7 + n_q)
    q = C.queries(len(LENGTHS), n_q, kv * group, d, dtype, seed=3, scale=1.5)
    compare(sta, t, q, dtype, accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
def test_page_lists_over_slots_in_any_order(sta, accumulate):  # noqa: F811
    lens = [700, 700, 64, 0, 1000]
    t = shuffled(C.make(lens, 2, 128, "bf16", seed=6), 6)
    lists = [[[0, 3, 10], []], [list(range(11)), [5]], [[0], []], [[], []], [[14, 15], [0, 1, 2, 7, 9, 13]]]
    q = C.queries(5, 5, 4, 128, "bf16", seed=6)
    compare(sta, t, q, "bf16", lists, accumulate)


def test_a_token_that_sees_nothing(sta):  # noqa: F811
    """Every slot holds a token newer than the first query."""
    t = C.make([3, 70], 1, 64, "bf16", seed=9)
    t["seen"] += 10
    t["slot_pos"][0, 0, :3] = torch.tensor([12, 10, 11], device="cuda")
    t["slot_pos"][1, 0, :70] = torch.arange(80 - 70, 80, device="cuda").int()
    q = C.queries(2, 4, 2, 64, "bf16", seed=9)
    o, lse, _ = compare(sta, t, q, "bf16", accumulate=True)
    assert torch.isneginf(lse[0, :, 0]).all() and (o[0, 0] == 0).all() and torch.isfinite(lse[0, :, 1:]).all()


def test_positions_of_a_cache_of_another_alignment(sta):  # noqa: F811
    """slot_pos begins four bytes past a boundary of 16."""
    t = shuffled(C.make([300, 65], 2, 128, "bf16", seed=12), 12)
    room = torch.empty(t["slot_pos"].numel() + 1, dtype=torch.int32, device="cuda")
    room[1:].copy_(t["slot_pos"].flatten())
    t["slot_pos"] = room[1:].view(t["slot_pos"].shape)
    assert t["slot_pos"].data_ptr() % 16 == 4
    compare(sta, t, C.queries(2, 4, 4, 128, "bf16", seed=12), "bf16")


@pytest.mark.parametrize("what", ["k_pages", "v_pages"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d,group,n_q", [(64, 1, 4), (128, 2, 3), (64, 8, 8), (128, 4, 6)])
def test_a_newer_token_that_is_not_finite(sta, d, group, n_q, bad, what):  # noqa: F811
    """The newest token's key or value is not finite, in a slot among older
    ones: the queries before it are not touched."""
    lens = [40, 64, 200]
    t = shuffled(C.make(lens, 1, d, "bf16", seed=d + n_q), n_q)
    at = [int((t["slot_pos"][b, 0, :n] == n - 1).nonzero()) for b, n in enumerate(lens)]
    assert all(j < n - n_q for j, n in zip(at, lens))  # among the older ones
    for b, j in enumerate(at):
        t[what][int(t["page_table"][b, j // C.PAGE]), 0, j % C.PAGE, 5] = bad
    q = C.queries(len(lens), n_q, group, d, "bf16", seed=10)
    c = C.oracle(t)
    o, lse = attend(sta, t, q)
    ok(sta)
    with np.errstate(invalid="ignore", over="ignore"):
        want = K.attend(c, q.double().cpu().numpy(), d ** -0.5, by_position=True)
    early = tuple(x[:, :-1] if x.ndim == 4 else x[:, :, :-1] for x in want)
    C.check_attention(o[:, :-1], lse[:, :, :-1], early, d, "bf16", 200)
    if what == "v_pages":
        got = o[:, -1].double().cpu().numpy()
        assert np.array_equal(np.isfinite(got), np.isfinite(want[0][:, -1]))


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("d,dtype,kv,group,n_q,budget", [
    (64, "bf16", 2, 4, 4, 100), (128, "fp16", 3, 1, 2, 64), (128, "bf16", 1, 8, 7, 150), (64, "fp16", 1, 2, 32, 100)])
def test_drafts_after_evictions(sta, d, dtype, kv, group, n_q, budget, accumulate):  # noqa: F811
    """A padded batch of prompts, then n_q tokens at a time: append, evict,
    attend. The evictions put the newest tokens into the slots of given-up
    ones; the oracle goes on from the GPU's weights after each step."""
    prompts = [130, 40, 5]
    t = C.make([0, 0, 0], kv, d, dtype, seed=30, room=200)
    t["weight"].zero_()
    c = C.oracle(t)
    moved = False
    for k, counts in enumerate([prompts] + [[n_q] * 3] * 5):
        n = max(counts)
        new = [C.queries(3, n, kv, d, dtype, seed=100 * k + s) for s in (1, 2)]
        cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
        for x in ("lens", "seen"):
            t[x] += cnt[:, None]
            c[x] += np.array(counts, dtype=np.int32)[:, None]
        sta.sta_cache_append(cache_of(sta, t), *new, counts=cnt)
        K.append(c, *(x.double().cpu().numpy() for x in new), counts=counts)
        evict(sta, t, budget, n_q, 2)
        ok(sta)
        K.evict(c, budget, n_q, 2)
        C.same_as(t, c)
        length, seen = int(c["lens"][0, 0]), int(c["seen"][0, 0])
        moved |= bool((c["slot_pos"][0, 0, length - n_q:length] != np.arange(seen - n_q, seen)).any())
        compare(sta, t, C.queries(3, n_q, kv * group, d, dtype, seed=k), dtype, accumulate=accumulate)
        if accumulate:
            c["weight"] = t["weight"].double().cpu().numpy()
    # at some step the newest tokens were not the last slots in order (with equal weights they are: the first slots
    # stay, and the newest tokens fill the last ones)
    assert moved or not accumulate


def test_drafts_that_the_eviction_gave_up(sta):  # noqa: F811
    """Nothing recent is protected and the drafts have no weight: some are gone
    when they are attended for, the others are seen by position as ever."""
    n_q, kv, d = 5, 2, 64
    t = C.make([120, 75], kv, d, "bf16", seed=41, room=n_q)
    new = [C.queries(2, n_q, kv, d, "bf16", seed=s) for s in (1, 2)]
    t["lens"] += n_q
    t["seen"] += n_q
    sta.sta_cache_append(cache_of(sta, t), *new)
    t["weight"][0, :, 121] = 1e9  # one draft that is heavy all the same
    t["weight"][0, :, 123] = 1e9
    evict(sta, t, 78, 0, 0)
    ok(sta)
    newest = (t["slot_pos"][0, :, :78] >= 120).sum(-1)
    assert (newest == 2).all() and t["lens"].tolist() == [[78, 78], [78, 78]]
    compare(sta, t, C.queries(2, n_q, kv * 2, d, "bf16", seed=4), "bf16", accumulate=True)


def test_drafts_taken_back_before_the_eviction(sta):  # noqa: F811
    """Append four drafts, attend, take two back, evict, and go on: what was
    taken back is overwritten, the rest goes by position."""
    n_q, kv, d, budget = 4, 2, 128, 90
    t = C.make([88, 200], kv, d, "fp16", seed=42, room=80)
    c = C.oracle(t)
    for k in range(6):
        new = [C.queries(2, n_q, kv, d, "fp16", seed=10 * k + s) for s in (1, 2)]
        for x in ("lens", "seen"):
            t[x] += n_q
            c[x] += n_q
        sta.sta_cache_append(cache_of(sta, t), *new)
        K.append(c, *(x.double().cpu().numpy() for x in new))
        compare(sta, t, C.queries(2, n_q, kv * 4, d, "fp16", seed=k), "fp16", accumulate=True)
        for x in ("lens", "seen"):
            t[x] -= 2
            c[x] -= 2
        c["weight"] = t["weight"].double().cpu().numpy()
        evict(sta, t, budget, 8, 2)
        ok(sta)
        K.evict(c, budget, 8, 2)
        C.same_as(t, c)


def test_captured_steps_with_drafts(sta):  # noqa: F811
    """Append three tokens, evict, attend and accumulate, captured once and
    replayed, against the same calls made one by one on another stream."""
    n_q, kv, group, d, budget = 3, 2, 4, 64, 70
    t = C.make([60, 100], kv, d, "bf16", seed=43, room=40)
    ref = {n: x.clone() for n, x in t.items()}
    k_new, v_new = (C.queries(2, n_q, kv, d, "bf16", seed=s) for s in (1, 2))
    q = C.queries(2, n_q, kv * group, d, "bf16", seed=3)

    def buffers(t):
        cache = cache_of(sta, t)
        return (cache, torch.empty_like(q), torch.empty(2, kv * group, n_q, device="cuda"),
                garbage(sta.sta_attn_fwd_cached_workspace(cache, kv * group, n_q, True)),
                garbage(sta.sta_cache_evict_workspace(cache, budget)))

    def step(t, cache, o, lse, ws, ews):
        t["lens"].add_(n_q)
        t["seen"].add_(n_q)
        sta.sta_cache_append(cache, k_new, v_new)
        sta.sta_cache_evict(cache, budget, n_q, 1, ews)
        sta.sta_attn_fwd_cached(cache, q, o, lse, ws, accumulate=True)

    mine, theirs, side = buffers(t), buffers(ref), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(t, *mine)
    for _ in range(8):
        k_new.normal_()
        q.normal_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            step(ref, *theirs)
        torch.cuda.synchronize()
        assert torch.equal(C.bits(mine[1]), C.bits(theirs[1])) and torch.equal(mine[2], theirs[2])
    ok(sta)
    for n in ("lens", "seen", "slot_pos", "weight"):
        assert torch.equal(t[n], ref[n])
