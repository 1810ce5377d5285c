"""Runs the cache calls on small seeded cases and saves outputs and device
statuses to an .npz file (argv[1]); test_cache_checked.py runs it under the
checked build and the product build and compares. Needs a GPU."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import _cache as C  # noqa: E402
import block_sparse_attention_28_b200 as sta  # noqa: E402

out = {}


def keep(name, x):
    x = x.detach().cpu()
    out[name] = (x.view(torch.int16) if x.element_size() == 2 else x).numpy()


for d, dtype, kv, group, n_q, budget in ((64, "bf16", 2, 1, 1, 100), (128, "fp16", 3, 4, 1, 64),
                                         (128, "bf16", 1, 3, 6, 700), (64, "fp16", 2, 8, 8, 1000)):
    tag = f"{d}_{dtype}_{group}_{n_q}"
    lens = [0, 1, 65, 700, 3000, 20_000 if n_q == 1 else 130]
    t = C.make(lens, kv, d, dtype, seed=d + n_q, room=80)
    cache = sta.kv_cache(**t)
    new = [C.queries(len(lens), 70, kv, d, dtype, seed=s) for s in (1, 2)]
    counts = torch.tensor([70, 0, 1, 64, 3, 70], dtype=torch.int32, device="cuda")
    t["lens"] += counts[:, None]
    t["seen"] += counts[:, None]
    sta.sta_cache_append(cache, *new, counts=counts)
    q = C.queries(len(lens), n_q, kv * group, d, dtype, seed=3)
    o, lse = torch.zeros_like(q), torch.zeros(len(lens), kv * group, n_q, device="cuda")
    ws = torch.full((sta.sta_attn_fwd_cached_workspace(cache, kv * group, n_q, True),), 0xA7, dtype=torch.uint8,
                    device="cuda")
    sta.sta_attn_fwd_cached(cache, q, o, lse, ws, accumulate=True)
    keep(tag + "_o", o)
    keep(tag + "_lse", lse)
    keep(tag + "_weight", t["weight"])
    ews = torch.full((sta.sta_cache_evict_workspace(cache, budget),), 0xA7, dtype=torch.uint8, device="cuda")
    sta.sta_cache_evict(cache, budget, 20, 3, ews)
    for n in ("k_pages", "v_pages", "lens", "slot_pos", "weight"):
        keep(f"{tag}_{n}", t[n])
    rows = len(lens) * kv
    ptr = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    idx = torch.zeros(rows, dtype=torch.int32, device="cuda")
    t["lens"].clamp_min_(1)
    sta.sta_attn_fwd_cached(cache, q, o, lse, ws, page_ptr=ptr, page_idx=idx)
    keep(tag + "_listed", lse)
    torch.cuda.synchronize()
    out["status_" + tag] = np.int64(sta.sta_get_device_error())
out["debug_build"] = np.int64(sta.sta_debug_build())
np.savez(sys.argv[1], **out)
