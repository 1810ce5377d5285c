"""The paged key-value cache without a GPU: what the calls refuse before
anything runs, workspace sizes, the binding's checks, and the oracle pinned
to dense attention and to cases worked by hand."""
import ctypes
import os
import runpy
import subprocess

import numpy as np
import pytest
import torch

import _cache as C
from oracle import kv_cache as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sta():
    runpy.run_path(os.path.join(ROOT, "block_sparse_attention_28_b200", "build.py"), run_name="sta_build")["build"]()
    import block_sparse_attention_28_b200 as mod

    return mod


def desc(sta, **over):
    d = sta.KvCacheDesc(2, 4, 128, sta.STA_BF16, 10, 5, 256, 512, 16, 16, 16, 16, 16)
    for n, x in over.items():
        setattr(d, n, x)
    return d


BAD_SIZES = [("B", 0, 1), ("kv_heads", 0, 1), ("num_pages", 0, 1), ("max_pages", 0, 1), ("B", -1, 1), ("d", 96, 2),
             ("d", 0, 2), ("dtype", 2, 2), ("B", 65536, 2), ("num_pages", 1 << 23, 2), ("max_pages", (1 << 24) + 1, 2),
             ("max_pages", 1 << 29, 2)]
BAD_POINTERS = [("k_pages", None), ("v_pages", None), ("page_table", None), ("lens", None), ("k_pages", 24),
                ("v_pages", 8), ("page_table", 18), ("lens", 17), ("seen", 2), ("slot_pos", 2), ("weight", 2),
                ("seen", None)]


def calls(sta, d, ws=256, ws_bytes=1 << 30):
    p = None if d is None else ctypes.byref(d)
    lib = sta._lib
    return {
        "append": lib.sta_cache_append(p, 16, 16, 3, None, None),
        "attend": lib.sta_attn_fwd_cached(p, 16, 32, None, 8, 1, None, None, 0, 0, ws, ws_bytes, 0.0, None),
        "evict": lib.sta_cache_evict(p, 16, 4, 2, ws, ws_bytes, None),
    }


def test_bad_caches_are_refused(sta):
    assert set(calls(sta, None).values()) == {sta.STA_ERR_INVALID_ARG}
    for name, value, status in BAD_SIZES:
        assert set(calls(sta, desc(sta, **{name: value})).values()) == {status}, (name, value)
        assert sta._lib.sta_attn_fwd_cached_workspace(ctypes.byref(desc(sta, **{name: value})), 8, 1, 1) == 0
        assert sta._lib.sta_cache_evict_workspace(ctypes.byref(desc(sta, **{name: value})), 16) == 0
    for name, value in BAD_POINTERS:
        assert set(calls(sta, desc(sta, **{name: value})).values()) == {sta.STA_ERR_INVALID_ARG}, (name, value)


def test_bad_arguments_are_refused(sta):
    lib, good = sta._lib, desc(sta)
    p = ctypes.byref(good)
    INV, UNS, WS = sta.STA_ERR_INVALID_ARG, sta.STA_ERR_UNSUPPORTED, sta.STA_ERR_WORKSPACE
    for k, v, n, counts, want in ((None, 16, 1, None, INV), (16, None, 1, None, INV), (8, 16, 1, None, INV),
                                  (16, 16, 0, None, INV), (16, 16, -1, None, INV), (16, 16, 1, 3, INV),
                                  (16, 16, 1 << 22, None, UNS)):
        assert lib.sta_cache_append(p, k, v, n, counts, None) == want

    def attend(q=16, o=32, lse=None, heads=8, n_q=1, ptr=None, idx=None, cap=0, acc=0, ws=256, n=1 << 30, scale=0.0,
               c=good):
        return lib.sta_attn_fwd_cached(ctypes.byref(c), q, o, lse, heads, n_q, ptr, idx, cap, acc, ws, n, scale, None)

    for kw, want in ((dict(q=None), INV), (dict(o=None), INV), (dict(o=16), INV), (dict(q=8), INV), (dict(o=24), INV), (dict(lse=2), INV),
                     (dict(heads=0), INV), (dict(heads=6), INV), (dict(n_q=0), INV), (dict(heads=8, n_q=33), UNS),
                     (dict(heads=4 * 65), UNS), (dict(ptr=16), INV), (dict(idx=16), INV), (dict(cap=4), INV),
                     (dict(ptr=16, idx=16, cap=-1), INV), (dict(ptr=17, idx=16, cap=4), INV), (dict(acc=2), INV),
                     (dict(acc=-1), INV), (dict(acc=1, c=desc(sta, weight=None)), INV), (dict(scale=-1.0), INV),
                     (dict(scale=float("nan")), INV), (dict(ws=None), WS), (dict(ws=128), WS), (dict(n=0), WS)):
        assert attend(**kw) == want, kw
    need = lib.sta_attn_fwd_cached_workspace(p, 8, 1, 1)
    assert need > 0 and need % 256 == 0 and need >= lib.sta_attn_fwd_cached_workspace(p, 8, 1, 0)
    assert attend(acc=1, n=need - 1) == WS
    assert lib.sta_attn_fwd_cached_workspace(p, 6, 1, 0) == 0 and lib.sta_attn_fwd_cached_workspace(p, 8, 99, 0) == 0

    def evict(budget=16, recent=4, sinks=2, ws=256, n=1 << 30, c=good):
        return lib.sta_cache_evict(ctypes.byref(c), budget, recent, sinks, ws, n, None)

    for kw, want in ((dict(budget=0), INV), (dict(budget=-5), INV), (dict(recent=-1), INV), (dict(sinks=-1), INV),
                     (dict(recent=15), INV), (dict(recent=2**31 - 1, sinks=2**31 - 1), INV),
                     (dict(c=desc(sta, weight=None)), INV), (dict(c=desc(sta, slot_pos=None)), INV),
                     (dict(ws=None), WS), (dict(ws=255), WS), (dict(n=8), WS)):
        assert evict(**kw) == want, kw
    assert lib.sta_cache_evict_workspace(p, 0) == 0 and lib.sta_cache_evict_workspace(p, 16) % 256 == 0


def test_the_binding_checks_its_tensors(sta):
    t = C.make([70, 3], 2, 64, "bf16", seed=1, device="cpu")
    cache = sta.kv_cache(**t)
    for name, bad in (("k_pages", t["k_pages"].float()), ("k_pages", t["k_pages"][0]),
                      ("v_pages", t["v_pages"].half()), ("v_pages", t["v_pages"][:-1]),
                      ("v_pages", t["v_pages"].transpose(0, 1).contiguous().transpose(0, 1)),
                      ("page_table", t["page_table"].long()), ("page_table", t["page_table"][0]),
                      ("page_table", t["page_table"].t().contiguous().t()), ("lens", t["lens"].long()),
                      ("lens", t["lens"][:, :1]), ("seen", t["seen"].float()), ("slot_pos", t["slot_pos"][..., :-1]),
                      ("weight", t["weight"].double()), ("weight", t["weight"][:, :, ::2]), ("lens", None)):
        with pytest.raises((ValueError, AttributeError)):
            sta.kv_cache(**dict(t, **{name: bad}))
    new = torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    q, lse = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 1)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: sta.sta_cache_append(cache, new.half(), new), lambda: sta.sta_cache_append(cache, new, new[:1]),
                 lambda: sta.sta_cache_append(cache, new[:, ::2], new[:, ::2]),
                 lambda: sta.sta_cache_append(cache, new[0], new[0]),
                 lambda: sta.sta_cache_append(cache, new, new, counts=torch.zeros(2)),
                 lambda: sta.sta_cache_append(cache, new, new, counts=torch.zeros(3, dtype=torch.int32)),
                 lambda: sta.sta_attn_fwd_cached(cache, q.float(), q, lse, ws),
                 lambda: sta.sta_attn_fwd_cached(cache, q, q[:1], lse, ws),
                 lambda: sta.sta_attn_fwd_cached(cache, q, q, lse[:, :2], ws),
                 lambda: sta.sta_attn_fwd_cached(cache, q, q, lse, ws.float()),
                 lambda: sta.sta_attn_fwd_cached(cache, q, q, lse, None),
                 lambda: sta.sta_attn_fwd_cached(cache, q, q, lse, ws, page_ptr=torch.zeros(4, dtype=torch.int32),
                                                 page_idx=torch.zeros(4, dtype=torch.int32)),
                 lambda: sta.sta_cache_evict(cache, 4, 1, 1, None),
                 # all as it should be, but not on a GPU
                 lambda: sta.sta_cache_append(cache, new, new),
                 lambda: sta.sta_attn_fwd_cached(cache, q, q, lse, ws),
                 lambda: sta.sta_cache_evict(cache, 4, 1, 1, ws)):
        with pytest.raises(ValueError):
            call()
    assert sta.sta_attn_fwd_cached_workspace(cache, 4, 1, True) > 0
    assert sta.sta_cache_evict_workspace(cache, 4) > 0


def test_the_description_of_a_cache_is_laid_out_as_in_the_header(sta):
    text = open(os.path.join(ROOT, "include", "sta.h")).read()
    body = text[text.index("#define STA_BF16"):text.index("} sta_kv_cache;")]
    at = [body.index(n) for n in ("int32_t B, kv_heads, d;", "int32_t dtype;", "int32_t num_pages;",
                                  "int32_t max_pages;", "*k_pages, *v_pages;", "*page_table;", "*lens;", "*seen;",
                                  "*slot_pos;", "*weight;")]
    assert at == sorted(at)
    assert [n for n, _ in sta.KvCacheDesc._fields_] == ["B", "kv_heads", "d", "dtype", "num_pages", "max_pages",
                                                        "k_pages", "v_pages", "page_table", "lens", "seen",
                                                        "slot_pos", "weight"]
    assert ctypes.sizeof(sta.KvCacheDesc) == 6 * 4 + 7 * 8


# -------------------------------------------------------- index arithmetic
@pytest.fixture(scope="module")
def index(tmp_path_factory):
    """The kernels' index header, compiled for the host."""
    d = tmp_path_factory.mktemp("index")
    header = os.path.join(ROOT, "block_sparse_attention_28_b200", "csrc", "sta_cache_index.h")
    (d / "index.cpp").write_text(f'''#include "{header}"
using namespace sta::cache;
extern "C" {{
int length(int len, int max_pages) {{ return length_ok(len, max_pages); }}
int page(int page, int num_pages) {{ return page_ok(page, num_pages); }}
int filled(int len) {{ return filled_pages(len); }}
int list(int first, int next, long long capacity, int max_pages) {{ return list_ok(first, next, capacity, max_pages); }}
int column(int column, int before, int filled) {{ return column_ok(column, before, filled); }}
int units(int pages) {{ return row_units(pages); }}
// 0 if the chunks of `units` cover them one after another, none twice, in at
// most `workers` chunks, and of() finds each unit in its chunk (of every unit,
// or of the first and last of each chunk)
int chunks(int units, int workers, int every) {{
  const Chunks c = make_chunks(units, workers);
  if (c.begin(0) != 0 || c.size < 1 || c.begin(workers) != units || c.begin(workers + 5) != units) return 1;
  for (int i = 0; i < workers && c.begin(i) < units; ++i) {{
    const int u0 = c.begin(i), u1 = c.begin(i + 1);
    if (u0 >= u1 || c.of(u0) != i || c.of(u1 - 1) != i) return 2;
    for (int u = u0; every && u < u1; ++u)
      if (c.of(u) != i) return 3;
  }}
  return 0;
}}
int part(int chunk, int begins) {{ return part_of(chunk, begins != 0); }}
}}''')
    so = d / "index.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", str(so), str(d / "index.cpp")], check=True)
    lib = ctypes.CDLL(str(so))
    lib.list.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int]
    return lib


def test_what_is_out_of_bounds(index):
    """Lengths, page numbers, list offsets and entries that a kernel leaves out."""
    top = 2**31 - 1
    assert [index.length(n, 3) for n in (-2**31, -1, 0, 1, 192, 193, top)] == [0, 0, 1, 1, 1, 0, 0]
    assert index.length(1 << 30, 1 << 24) and not index.length((1 << 30) + 1, 1 << 24)
    assert [index.page(n, 7) for n in (-2**31, -1, 0, 6, 7, top)] == [0, 0, 1, 1, 0, 0]
    assert [index.filled(n) for n in (-5, 0, 1, 64, 65, 1 << 30)] == [0, 0, 1, 1, 2, 1 << 24]
    assert index.list(0, 0, 0, 1) and index.list(2, 6, 6, 4)
    for bad in ((-1, 2, 9, 9), (3, 2, 9, 9), (2, 10, 9, 9), (0, 5, 9, 4), (-2**31, top, 9, 9), (top, -2**31, 9, 9)):
        assert not index.list(*bad), bad
    assert index.column(0, -1, 1) and index.column(5, 3, 6)
    for bad in ((-1, -1, 4), (4, 3, 4), (2, 2, 4), (1, 2, 4), (0, -1, 0)):
        assert not index.column(*bad), bad


def test_chunks_cover_the_units_once(index):
    for workers in (1, 2, 7, 32, 296, 592, 1036):
        for units in list(range(0, 60)) + [workers * k + r for k in (1, 3, 4, 5, 13, 20, 100) for r in (-1, 0, 1)]:
            assert index.chunks(units, workers, 1) == 0, (units, workers)
        for units in (2**31 - 1, 2**31 - 2, 10**9 + 7):
            assert index.chunks(units, workers, 0) == 0, (units, workers)
    assert len({index.part(c, b) for c in range(9) for b in (0, 1)}) == 18
    assert [index.units(n) for n in (0, 1, 5)] == [0, 2, 6]


# ------------------------------------------------------------------- oracle
def test_oracle_attention_is_dense_attention():
    t = C.make([70, 130], 2, 64, "bf16", seed=3, device="cpu")
    c = C.oracle(t)
    q = C.queries(2, 3, 4, 64, "bf16", seed=4, device="cpu").double()
    o, lse, _, _ = K.attend(c, q.numpy(), 0.2, accumulate=True)
    for b, n in enumerate((70, 130)):
        pages = t["page_table"][b, :-(-n // 64)].long()
        k = t["k_pages"][pages].double().transpose(0, 1).reshape(2, -1, 64)[:, :n]
        v = t["v_pages"][pages].double().transpose(0, 1).reshape(2, -1, 64)[:, :n]
        s = 0.2 * torch.einsum("ihd,hjd->hij", q[b], k.repeat_interleave(2, 0))
        s = s.masked_fill(torch.arange(n)[None] > torch.arange(n - 3, n)[:, None], -float("inf"))
        p = s.softmax(-1)
        assert np.allclose(o[b], torch.einsum("hij,hjd->ihd", p, v.repeat_interleave(2, 0)).numpy(), atol=1e-12)
        assert np.allclose(lse[b], s.logsumexp(-1).numpy(), atol=1e-12)
        added = c["weight"][b, :, :n] - t["weight"][b, :, :n].double().numpy()
        assert np.allclose(added, p.reshape(2, 2, 3, n).sum((1, 2)).numpy(), atol=1e-12)


def test_oracle_lists_and_hidden_slots():
    """A list of every page is no list; a query that sees nothing gives zero."""
    t = C.make([70], 1, 64, "bf16", seed=3, device="cpu")
    c = C.oracle(t)
    q = C.queries(1, 1, 1, 64, "bf16", seed=4, device="cpu").double().numpy()
    assert np.array_equal(K.attend(c, q, 0.1)[0], K.attend(c, q, 0.1, [[[0, 1]]])[0])
    o, lse, _, _ = K.attend(c, q, 0.1, [[[]]])
    assert not o.any() and np.isneginf(lse).all()
    c["lens"][:] = 1
    q3 = np.repeat(q, 3, axis=1)
    o, lse, _, _ = K.attend(c, q3, 0.1)
    assert np.isneginf(lse[0, 0, :2]).all() and np.isfinite(lse[0, 0, 2]) and not o[0, :2].any()
    page, row = K.where(c, 0, 0)
    assert np.allclose(o[0, 2, 0], c["v_pages"][page, 0, row])


def test_oracle_append_and_evict_by_hand():
    """Six tokens, budget four, one sink and one recent: of the others (weights
    3, 1, 2, 2 in slots 1 to 4) the 3 and, of the equal 2s, the lower slot stay;
    slot 2 is given up below the budget, and slot 5 (the recent one) moves in."""
    t = C.make([6], 1, 64, "bf16", seed=5, device="cpu")
    c = C.oracle(t)
    c["weight"][0, 0, :6] = [0, 3, 1, 2, 2, 0]
    page, _ = K.where(c, 0, 0)
    k = c["k_pages"][page, 0].copy()
    K.evict(c, 4, 1, 1)
    assert c["lens"][0, 0] == 4
    assert c["slot_pos"][0, 0, :6].tolist() == [0, 1, 5, 3, 4, 5]
    assert c["weight"][0, 0, :6].tolist() == [0, 3, 0, 2, 2, 0]
    assert np.array_equal(c["k_pages"][page, 0, :6], k[[0, 1, 5, 3, 4, 5]])
    # the next token goes behind them, at position 6
    c["lens"] += 1
    c["seen"] += 1
    new = np.full((1, 1, 1, 64), 9.0)
    K.append(c, new, -new)
    assert c["slot_pos"][0, 0, 4] == 6 and c["weight"][0, 0, 4] == 0
    assert (c["k_pages"][page, 0, 4] == 9).all() and (c["v_pages"][page, 0, 4] == -9).all()
    assert np.array_equal(c["k_pages"][page, 0, 5], k[5])


def test_oracle_goes_by_position():
    """Slots in order: as by slot. After an eviction, whose moves put new
    tokens into earlier slots: dense causal attention over the kept tokens put
    back in order of position."""
    t = C.make([70, 130], 2, 64, "bf16", seed=3, device="cpu")
    q = C.queries(2, 4, 4, 64, "bf16", seed=4, device="cpu").double().numpy()
    c = C.oracle(t)
    for x, y in zip(K.attend(c, q, 0.2), K.attend(c, q, 0.2, by_position=True)):
        assert np.array_equal(x, y)
    K.evict(c, 50, 4, 2)
    pos = c["slot_pos"][:, :, :50]
    assert (c["lens"] == 50).all() and any((pos[b, :, :46] >= n - 4).any() for b, n in ((0, 70), (1, 130)))
    o, lse, _, _ = K.attend(c, q, 0.2, by_position=True)
    for b in range(2):
        for h in range(2):
            order = np.argsort(pos[b, h])
            at = [K.where(c, b, j) for j in order]
            k = np.stack([c["k_pages"][p, h, r] for p, r in at])
            v = np.stack([c["v_pages"][p, h, r] for p, r in at])
            for g in (2 * h, 2 * h + 1):
                s = 0.2 * q[b, :, g] @ k.T
                s[np.arange(50)[None] > np.arange(46, 50)[:, None]] = -np.inf  # the last four are the newest
                e = np.exp(s)
                assert np.allclose(o[b, :, g], e / e.sum(1, keepdims=True) @ v, atol=1e-12)
                assert np.allclose(lse[b, g], np.log(e.sum(1)), atol=1e-12)
