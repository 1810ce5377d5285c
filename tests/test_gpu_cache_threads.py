"""Cache calls from several host threads at once, each on a stream, a cache and
workspaces of its own: sizes that need different amounts of shared memory do
not get into one another's way."""
import threading

import pytest
import torch

import _cache as C
from test_gpu_cache import attend, cache_of, garbage, ok, sta  # noqa: F401

pytestmark = pytest.mark.gpu


def together(works, times):
    """Runs every function `times` times, a thread each; the errors."""
    errors, start = [], threading.Barrier(len(works))

    def run(work):
        start.wait()
        try:
            for _ in range(times):
                work()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def test_the_first_call_of_a_thread(sta):  # noqa: F811
    """A thread that has made no other call to the GPU has no context of its
    own yet; the calls that describe their inputs to the driver bind it."""
    t = C.make([300, 70], 2, 64, "bf16", seed=2)
    cache, q = cache_of(sta, t), C.queries(2, 1, 4, 64, "bf16", seed=2)
    want = attend(sta, t, q)
    o, lse = torch.empty_like(q), torch.empty(2, 4, 1, device="cuda")
    ws = garbage(sta.sta_attn_fwd_cached_workspace(cache, 4, 1))
    g = sta.grid(2, 16, 16)
    tiled = [C.queries(1, 1, sta.sta_tiled_len(g), 64, "bf16", seed=s).contiguous() for s in range(3)]
    nt = sta.sta_num_tiles(g)
    ptr = torch.arange(0, (nt + 1) * nt, nt, dtype=torch.int32, device="cuda")
    idx = torch.arange(nt, dtype=torch.int32, device="cuda").repeat(nt)
    outs = [torch.empty_like(tiled[0]) for _ in range(2)]
    sta.sta_attn_fwd(*tiled, outs[0], None, ptr, idx, 1, 1, 64, g)
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()
    for work in (lambda: sta.sta_attn_fwd_cached(cache, q, o, lse, ws, stream=stream),
                 lambda: sta.sta_attn_fwd(*tiled, outs[1], None, ptr, idx, 1, 1, 64, g, stream=stream)):
        assert together([work], 1) == []
    ok(sta)
    assert torch.equal(C.bits(o), C.bits(want[0])) and torch.equal(lse, want[1])
    assert torch.equal(C.bits(outs[0]), C.bits(outs[1]))


def test_attention_with_other_numbers_of_query_rows(sta):  # noqa: F811
    t = C.make([300, 70], 1, 128, "bf16", seed=1, tracked=False, max_pages=700)
    cache, works, outs = cache_of(sta, t), [], []
    for n_q in (16, 40, 9, 64):
        q = C.queries(2, n_q, 1, 128, "bf16", seed=n_q)
        o, lse = torch.empty_like(q), torch.empty(2, 1, n_q, device="cuda")
        ws, s = garbage(sta.sta_attn_fwd_cached_workspace(cache, 1, n_q)), torch.cuda.Stream()
        outs.append((o, lse, attend(sta, t, q)))
        works.append(lambda q=q, o=o, lse=lse, ws=ws, s=s: sta.sta_attn_fwd_cached(cache, q, o, lse, ws, stream=s))
    torch.cuda.synchronize()
    assert together(works, 2000) == []
    ok(sta)
    for o, lse, (want_o, want_lse) in outs:
        assert torch.equal(C.bits(o), C.bits(want_o)) and torch.equal(lse, want_lse)


def test_evictions_under_tables_of_other_widths(sta):  # noqa: F811
    works, ends = [], []
    for width, n in ((70, 4300), (300, 200), (640, 40_000), (66, 100)):
        t = C.make([n], 1, 64, "bf16", seed=width, max_pages=max(width, -(-n // 64)), poison=False)
        cache, s = cache_of(sta, t), torch.cuda.Stream()
        ws = garbage(sta.sta_cache_evict_workspace(cache, n // 2))
        ends.append((t, n // 2))
        works.append(lambda c=cache, b=n // 2, ws=ws, s=s: sta.sta_cache_evict(c, b, 5, 1, ws, stream=s))
    torch.cuda.synchronize()
    assert together(works, 2000) == []
    ok(sta)
    assert all((t["lens"] == n).all() for t, n in ends)
