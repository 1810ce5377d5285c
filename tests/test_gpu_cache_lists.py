"""Page lists that are not in order: an entry counts only if it is above every
entry before it, so that no page is attended to twice, however a list is cut
into chunks and batches."""
import numpy as np
import pytest
import torch

import _cache as C
from oracle import kv_cache as K
from test_gpu_cache import attend, sta  # noqa: F401

pytestmark = pytest.mark.gpu


def kept(entries, filled):
    """The entries that count: those above all before them, of filled pages."""
    out, top = [], -1
    for e in entries:
        if top < e < filled:
            out.append(e)
        top = max(top, e)
    return out


def check(sta, t, lists, accumulate, d, dtype="bf16", group=1, n_q=1):  # noqa: F811
    B, kv = t["lens"].shape
    c = C.oracle(t)
    before = c["weight"].copy()
    start = t["weight"].clone()
    q = C.queries(B, n_q, kv * group, d, dtype, seed=8)
    first = None
    for _ in range(5):
        t["weight"].copy_(start)
        o, lse = attend(sta, t, q, lists, accumulate)
        torch.cuda.synchronize()
        assert sta.sta_get_device_error() == sta.STA_ERR_BAD_MASK
        got = (C.bits(o), C.bits(lse), C.bits(t["weight"]))
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))
    valid = [[kept(x, -(-int(c["lens"][b, h]) // C.PAGE)) for h, x in enumerate(heads)]
             for b, heads in enumerate(lists)]
    want = K.attend(c, q.double().cpu().numpy(), d ** -0.5, valid, accumulate)
    rel = C.check_attention(o, lse, want, d, dtype, int(c["lens"].max()))
    C.check_weight(t, c, before, rel, n_q * group)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("d,group,n_q", [(64, 1, 1), (128, 4, 2), (64, 8, 4)])
def test_a_page_after_a_bad_entry_is_not_attended_to_again(sta, accumulate, d, group, n_q):  # noqa: F811
    t = C.make([300, 300], 2, d, "bf16", seed=8)
    check(sta, t, [[[1, 3, 2, 3], [1, 2, 1, 2]], [[4, 0, 1, 4], [0, 9, 3, 4]]], accumulate, d, group=group, n_q=n_q)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows", [1, 30])
def test_long_lists_out_of_order(sta, accumulate, rows):  # noqa: F811
    """Lists of hundreds of entries, cut into chunks of a few (one row) or read
    in several batches (many rows): an entry far back is what rules one out."""
    pages = 310
    t = C.make([pages * C.PAGE - 7], rows, 64, "bf16", seed=rows)
    rng = np.random.default_rng(rows)
    lists = []
    for r in range(rows):
        x = sorted(rng.choice(pages, size=290, replace=False).tolist())
        kind = r % 5
        if kind == 0:
            x = x[:150] + x[100:240]  # goes back by 50, then over them again
        elif kind == 1:
            x = [x[40]] + x[:289]  # one at the front rules out 41
        elif kind == 2:
            x = x[:7] + [pages + 2] + x[7:289]  # past the last page: nothing after it counts
        elif kind == 3:
            x = [v for p in zip(x[0::2], x[1::2]) for v in (p[1], p[0])]  # every pair swapped
        else:
            x = x[:32] + x[:32] + x[:64] + x[32:190]
        lists.append(x)
    check(sta, t, [lists], accumulate, 64)
