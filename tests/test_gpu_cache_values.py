"""What the two-term weights of the products with V leave of small weights, and
what values that are not finite do."""
import numpy as np
import pytest
import torch

import _cache as C
from oracle import kv_cache as K
from test_gpu_cache import attend, ok, sta  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_small_weights_beside_a_token_of_value_zero(sta, d, dtype):  # noqa: F811
    """One key takes nearly all of the weight and its value is zero; the others
    have weights of 2^-16.25 to 2^-35.25 of it and large values, each of a column of
    its own: the outputs are those weights, one by one. With u = 2^-24 and w
    the weight (of a largest weight 1, the sum being 1 + 2^-11 at most):
      the score is an exact product of one column (q one, k a number of 8 bits)
      times scale and log2 e (1.5 u of at most 37 each), minus the maximum (u of
      37): the exponent is off by less than 37 * 4 u, the weight by 37 * 4 u ln 2
      and two ulp of the exponential more: 110 u of itself;
      the sum of the weights by 200 u; the split by what the header states;
      the output is rounded once (half a step, fp16's smallest being 2^-24)."""
    n = 21
    t = C.make([n], 1, d, dtype, seed=1, tracked=False, poison=False)
    page = int(t["page_table"][0, 0])
    k, v = t["k_pages"][page, 0], t["v_pages"][page, 0]
    k.zero_()
    v.zero_()
    below = torch.arange(16, 16 + n - 1, device="cuda") + 0.25  # of the first key's score, in powers of two
    k[1:n, 0] = -below.to(k.dtype)
    v[torch.arange(1, n), torch.arange(1, n)] = 32768.0
    q = torch.zeros(1, 1, 1, d, dtype=k.dtype, device="cuda")
    q[0, 0, 0, 0] = 1.0
    o, _ = attend(sta, t, q, sm_scale=float(np.log(2.0)))
    ok(sta)
    want = K.attend(C.oracle(t), q.double().cpu().numpy(), float(np.float32(np.log(2.0))))[0][0, 0, 0, 1:n]
    w = want / 32768.0
    u = 2.0 ** -24
    split = w * 2.0 ** -16 if dtype == "bf16" else np.maximum(w * 2.0 ** -22, 2.0 ** -39)
    limit = 32768.0 * (split + 310 * u * w)
    tiny = {"bf16": 0.0, "fp16": 2.0 ** -25}[dtype]
    limit += np.maximum((want + limit) * C.HALF[dtype], tiny)
    got = o[0, 0, 0, 1:n].double().cpu().numpy()
    assert (np.abs(got - want) <= limit).all(), (got - want) / limit


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d,group,n_q", [(64, 1, 1), (128, 4, 1), (64, 8, 4), (128, 2, 3)])
def test_a_value_in_view_that_is_not_finite(sta, d, group, n_q, bad):  # noqa: F811
    """A token that is the newest at first and then ages: the column of its value
    that is not finite is not finite for every query that sees it, at any age;
    all other columns are untouched."""
    for age in (0, 1, 3, 70, 200):
        lens = [age + 5, age + 90]
        t = C.make(lens, 1, d, "bf16", seed=age)
        for b, n in enumerate(lens):
            j = n - 1 - age
            t["v_pages"][int(t["page_table"][b, j // C.PAGE]), 0, j % C.PAGE, 7] = bad
        q = C.queries(2, n_q, group, d, "bf16", seed=3)
        o, lse = attend(sta, t, q)
        ok(sta)
        c = C.oracle(t)
        sees = [i for i in range(n_q) if n_q - 1 - i <= age]
        with np.errstate(invalid="ignore"):
            want = K.attend(c, q.double().cpu().numpy(), d ** -0.5)
        assert torch.isfinite(lse).all() and not torch.isfinite(o[:, sees][..., 7].float()).any()
        keep = np.arange(d) != 7
        part = tuple(x[..., keep] if x.ndim == 4 else x for x in want)
        C.check_attention(o[..., keep], lse, part, d, "bf16", max(lens))
        early = [i for i in range(n_q) if i not in sees]
        if early:
            assert torch.isfinite(o[:, early].float()).all()
