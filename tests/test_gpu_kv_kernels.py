"""Attention over the 8-bit cache, kernel by kernel: every kernel and work mapping that a call can take,
against the plain 64-bit form (kv_reference.py), and calls that once went wrong in one of them."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
from bit_gemm_fwht_amd import kv
from test_gpu_kv import DEV, DT, Setup, host

pytestmark = pytest.mark.gpu


def bounds(dtype, absv, mag, cnt, out):
    """How far out and lse may be from the exact ones.
    Scores: products with K are exact; D <= 256 additions and the scale err by 2^-23 of sum |q k| each at
    most (the matrix core's additions taken as no better than truncating): es = 258 * 2^-23 * mag. A
    score's difference to the maximum in log2 units is rounded once (2^-23 * 2 mag) and the exponential is
    good to 2 ulp: a weight is off by a factor 1 +- (2 es + 2^-21 mag + 2^-21). A sum of n weights errs by
    n * 2^-23 of the sum of their sizes, numerator and denominator alike, rescales included. bf16 queries:
    weights are sums of two bf16, the first cut after 8 significant bits (the rest is below 2^-7 of the
    weight's power of two), the second rounded to 8 (2^-16 of it): 2^-16, numerator only; and the output
    is rounded (2^-9). fp32 queries: three bf16, exact; one rounding of the output."""
    es = 258 * 2.0 ** -23 * mag
    w = 2 * es + 2.0 ** -21 * mag + 2.0 ** -21 + cnt * 2.0 ** -23
    rel = 2 * w[..., None] + (2.0 ** -16 if dtype == "bf16" else 0.0)
    tol = rel * absv * 1.01 + np.abs(out) * (2.0 ** -9 * 1.01 if dtype == "bf16" else 2.0 ** -22) + 1e-37
    return tol, w + 2.0 ** -22 * (1 + mag + np.log(np.maximum(cnt, 1)))


def check(s, q_heads, dtype, causal=True, window=0, scale=None, q=None, kv_heads=None):
    """One call against the reference; what it does not write would show as NaN. kv_heads: the reference
    looks at these only (and at their query heads)."""
    q = s.draw(q_heads, dtype) if q is None else q
    lse = torch.full((s.tokens, q_heads), math.nan, device=DEV)
    out = torch.full_like(q, math.nan)
    kv.attention(q, s.cache, s.batch, scale=scale, causal=causal, window=window, lse=lse, out=out)
    torch.cuda.synchronize()
    r, group = s.ref, q_heads // s.heads
    hs = list(range(s.heads)) if kv_heads is None else kv_heads
    hq = [h * group + g for h in hs for g in range(group)]
    part = r if kv_heads is None else ref.Cache(r.k[:, hs], r.v[:, hs], r.ks[:, hs], r.vs[:, hs])
    eo, el, absv, mag, cnt = ref.attention(host(q)[:, hq], part, s.cu, s.context, s.table,
                                           1 / math.sqrt(s.dim) if scale is None else scale, causal, window)
    bad = (~torch.isfinite(out)).any(2) | torch.isnan(lse)
    assert not bad.any().item(), f"{int(bad.sum())} of {bad.numel()} rows, (token, head) {bad.nonzero()[0].tolist()} first"
    o, got = host(out)[:, hq], host(lse)[:, hq]
    tol, ltol = bounds(dtype, absv, mag, cnt, eo)
    err, none = np.abs(o - eo), cnt == 0
    assert (err <= tol).all(), f"worst excess {(err / tol).max():.3g}"
    assert np.array_equal(np.isneginf(got), none) and not o[none].any()
    assert (np.abs(got[~none] - el[~none]) <= ltol[~none]).all()
    return out


# ------------------------------------------------------------------------------------------ hints
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,group,hint", [
    ([(1, 5000), (4, 2500), (1, 1)], 2, 4, (1, 5000)),  # 16 rows of a tile, the hint says 4
    ([(5, 8000)] * 8, 8, 1, (1, 8000)),                 # 5 rows, the hint says 1
    ([(9, 6000), (1, 4000)], 1, 3, (2, 3000)),          # two tiles, the second short; the context too small as well
])
def test_hints_that_are_too_small_leave_no_row_unwritten(lens, heads, group, hint, dtype):
    """Contexts that are split over the chip, with fewer rows of a sequence promised than there are."""
    s = Setup(lens, heads, 64, 32, seed=30)
    s.batch = kv.Batch(s.batch.cu_tokens, s.batch.context, s.batch.table, max_tokens=hint[0], max_context=hint[1])
    check(s, heads * group, dtype)
