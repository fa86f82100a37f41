"""Attention over the 8-bit cache, kernel by kernel: every kernel and work mapping that a call can take,
against the plain 64-bit form (kv_reference.py), and calls that once went wrong in one of them."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
from bit_gemm_fwht_amd import kv
from bit_gemm_fwht_amd.fp4 import Fp4Error
from test_gpu_kv import DEV, DT, Setup, host

pytestmark = pytest.mark.gpu


def bounds(dtype, absv, mag, cnt):
    """How far out may be from the exact one before it is rounded to its type, and lse.
    Scores: products with K are exact; D <= 256 additions and the scale err by 2^-23 of sum |q k| each at
    most (the matrix core's additions taken as no better than truncating): es = 258 * 2^-23 * mag. A
    score's difference to the maximum in log2 units is rounded once (2^-23 * 2 mag) and the exponential is
    good to 2 ulp: a weight is off by a factor 1 +- (2 es + 2^-21 mag + 2^-21). A sum of n weights errs by
    n * 2^-23 of the sum of their sizes, numerator and denominator alike, rescales included. bf16 queries:
    weights are sums of two bf16, the first cut after 8 significant bits (the rest is below 2^-7 of the
    weight's power of two), the second rounded to 8 (2^-16 of it): 2^-16, numerator only. fp32 queries:
    three bf16, exact."""
    es = 258 * 2.0 ** -23 * mag
    w = 2 * es + 2.0 ** -21 * mag + 2.0 ** -21 + cnt * 2.0 ** -23
    rel = 2 * w[..., None] + (2.0 ** -16 if dtype == "bf16" else 0.0)
    return rel * absv * 1.01 + 1e-37, w + 2.0 ** -22 * (1 + mag + np.log(np.maximum(cnt, 1)))


def rounded(x, dtype):
    return torch.from_numpy(x).to(torch.float32).to(DT[dtype]).to(torch.float64).numpy()


def check(s, q_heads, dtype, causal=True, window=0, scale=None, q=None, kv_heads=None, chain=None):
    """One call against the reference; what it does not write would show as NaN. kv_heads: the reference
    looks at these only (and at their query heads). chain: additions that a sum goes through at most, where
    these are fewer than its keys."""
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
    tol, ltol = bounds(dtype, absv, mag, cnt if chain is None else np.minimum(cnt, chain))
    # rounding keeps the order: out lies between the rounded ends of what it may have been before
    lo, hi = rounded(eo - tol, dtype), rounded(eo + tol, dtype)
    wrong = (o < lo) | (o > hi)
    assert not wrong.any(), f"{wrong.sum()} of {wrong.size} off, up to {(np.abs(o - eo) / tol)[wrong].max():.3g} bounds"
    none = cnt == 0
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


# --------------------------------------------------------------------- places that hold nothing
def poison_scales(s, code=255):
    """Every scale of a page that holds no token of the batch, page 0's among them (the page that stands in
    for one that is missing), set to `code`."""
    used = {int(p) for i, n in enumerate(s.need) for p in s.table[i, :n] if 0 <= p < s.ref.pages}
    free = [p for p in range(s.ref.pages) if p not in used]
    if 0 in used:  # page 0 changes places with a free one
        f = free[0]
        s.table[s.table == 0] = f
        for a in (s.ref.k, s.ref.v, s.ref.ks, s.ref.vs):
            a[f] = a[0]
        free[0] = 0
        s.batch.table.copy_(torch.from_numpy(s.table))
    s.ref.ks[free], s.ref.vs[free] = code, code
    s.ref.k[free], s.ref.v[free] = 0x7F, 0xFF
    for t, a in ((s.cache.k_codes, s.ref.k), (s.cache.v_codes, s.ref.v), (s.cache.k_scales, s.ref.ks),
                 (s.cache.v_scales, s.ref.vs)):
        t.copy_(torch.from_numpy(a))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,group,dim,page", [
    ([(1, 37), (3, 100), (2, 1000)], 2, 3, 64, 16),       # few rows
    ([(1, 5000), (2, 4000)], 2, 4, 128, 32),              # split over the chip
    ([(700, 700), (300, 900)], 8, 8, 64, 16),             # many rows
    ([(300, 800)], 32, 8, 64, 64),                        # many rows, enough tiles for eight waves
])
def test_scales_of_places_without_a_token_are_not_used(lens, heads, group, dim, page, dtype):
    """Pages that are missing in the middle of a context, and pages wholly before a window, under scale
    codes of 255 (not a number)."""
    s = Setup(lens, heads, dim, page, seed=31, fill=0x7F)
    poison_scales(s)
    hs = [0, heads - 1]
    check(s, heads * group, dtype, kv_heads=hs)
    at = [min(n - 1, 2 + 3 * i) for i, n in enumerate(s.need)]
    gone = [int(s.table[i, j]) for i, j in enumerate(at)]
    for i, j in enumerate(at):
        s.table[i, j] = [-1, s.ref.pages, 1 << 30][i % 3]
    s.batch.table.copy_(torch.from_numpy(s.table))
    s.ref.ks[gone], s.ref.vs[gone] = 255, 255  # nobody's now
    s.cache.k_scales.copy_(torch.from_numpy(s.ref.ks))
    s.cache.v_scales.copy_(torch.from_numpy(s.ref.vs))
    for scale in (None, 0.0):
        check(s, heads * group, dtype, scale=scale, kv_heads=hs)
    # pages before every window belong to nobody either, but stay in the table
    window = 70
    before = [int(p) for i, (n, ctx) in enumerate(lens) for p in s.table[i, :max(0, ctx - n - window + 1) // page]
              if 0 <= p < s.ref.pages]
    s.ref.ks[before], s.ref.vs[before] = 255, 255
    s.ref.k[before], s.ref.v[before] = 0x7F, 0x7F
    for t, a in ((s.cache.k_codes, s.ref.k), (s.cache.v_codes, s.ref.v), (s.cache.k_scales, s.ref.ks),
                 (s.cache.v_scales, s.ref.vs)):
        t.copy_(torch.from_numpy(a))
    check(s, heads * group, dtype, window=window, kv_heads=hs)


# ------------------------------------------------------------------------------------- wide windows
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 7, 2 ** 33])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,group", [
    ([(3, 0), (0, 10), (4, 2), (2, 50), (10, 2)], 2, 3),  # rows before the first token
    ([(10, 2), (5, 4000), (6, 3)], 2, 4),                 # beside a context that is split
    ([(200, 150), (90, 90), (500, 400)], 8, 8),           # many rows
])
def test_windows_wider_than_any_context_mask_nothing(lens, heads, group, dtype, causal, window):
    """The widest windows there are, with rows whose tokens lie before the first one: position - window
    does not fit 32 bits."""
    s = Setup(lens, heads, 64, 32, seed=32, fill=0x7F)
    q = s.draw(heads * group, dtype)
    hs = [0, heads - 1]
    out = check(s, heads * group, dtype, causal=causal, window=window, q=q, kv_heads=hs)
    plain = check(s, heads * group, dtype, causal=causal, q=q, kv_heads=hs)
    assert torch.equal(out, plain)


# ------------------------------------------------------------------------------------ long contexts
@pytest.mark.parametrize("hint", [None, 100])
def test_contexts_past_2_30(hint):
    """A context of 2^30 + 3005 tokens: nearly all of its pages are one page whose keys get no weight, the
    others lie at its start, at 2^29, on both sides of 2^30 and at its end. Split over the chip, and (as
    the hint speaks of a short context) in one workgroup."""
    page, dim = 128, 16
    ctx = 2 ** 30 + 3005
    width = -(-ctx // page)
    at = [0, 2 ** 29 // page, 2 ** 30 // page - 1, 2 ** 30 // page, width - 1]
    s = Setup([(1, 5 * page)], 1, dim, page, seed=33)
    s.context[:] = 4 * page + ctx - (width - 1) * page  # the pages at `at`, for the reference
    q = s.draw(4, "bf16")
    q[:, :, 0] = 8.0
    s.ref.k[..., 0] = 0
    dull = [p for p in range(s.ref.pages) if p not in s.table[0]][0]
    s.ref.k[dull] = 0
    s.ref.k[dull, :, :, 0] = 0xFE  # -448
    s.ref.ks[dull] = 127
    for t, a in ((s.cache.k_codes, s.ref.k), (s.cache.k_scales, s.ref.ks)):
        t.copy_(torch.from_numpy(a))
    table = torch.full((1, width), dull, dtype=torch.int32, device=DEV)
    table[0, at] = s.batch.table[0]
    s.batch = kv.Batch(s.batch.cu_tokens, torch.tensor([ctx], dtype=torch.int32, device=DEV), table,
                       max_context=hint)
    check(s, 4, "bf16", scale=0.25, q=q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 1, 50, 10000])
@pytest.mark.parametrize("n,heads,group", [(3, 2, 4), (500, 8, 8)])
def test_contexts_past_their_table(n, heads, group, window, dtype):
    """A context far past what its table holds: the table's keys are all there is, positions lie behind
    them (and windows with them)."""
    s = Setup([(n, 1000), (2, 3000)], heads, 64, 32, seed=34, fill=0x7F)
    for ctx in (2 ** 31 - 1, 1100):
        s.context[0] = ctx
        s.table[0, 31] = -1  # tokens 992 on
        s.batch.context.copy_(torch.from_numpy(s.context))
        s.batch.table.copy_(torch.from_numpy(s.table))
        check(s, heads * group, dtype, window=window, kv_heads=[0])


# --------------------------------------------------------------------------------- kernel by kernel
def ragged(n, rows, longest):
    """n sequences of 1 to `rows` rows and uneven contexts up to `longest`."""
    return [(1 + i % rows, max(rows, round(longest * ((i + 1) * 0.6180339887 % 1.0)))) for i in range(n)]


# name: lens, kv heads, query heads to each, dim, page, dtype, kernel, rows of a tile. Contexts of several
# steps, tiles that end inside a sequence, dims below and at multiples of 64.
ROWS, SPLIT, NEAR, TILES = kv.PLAN_ROWS, kv.PLAN_ROWS_SPLIT, kv.PLAN_ROWS_NEAR, kv.PLAN_TILES
UNEVEN = [(300, 300), (500, 900), (0, 7), (129, 1640)]
KERNELS = {
    "rows, 70 sequences": (ragged(70, 1, 1000), 2, 4, 128, 32, "bf16", ROWS, 16),
    "rows, 150 sequences": (ragged(150, 3, 700), 1, 5, 80, 16, "bf16", ROWS, 16),
    "rows, 129 sequences, fp32": (ragged(129, 2, 500), 1, 3, 256, 64, "f32", ROWS, 16),
    "rows, 5000 sequences": (ragged(5000, 2, 60), 1, 2, 32, 16, "bf16", ROWS, 16),
    "split, 300 sequences": (ragged(300, 2, 3000), 1, 2, 32, 16, "f32", SPLIT, 16),
    "split, 100 sequences": (ragged(100, 1, 5000), 2, 4, 64, 32, "bf16", SPLIT, 16),
    "split, 80": (ragged(5, 2, 7000), 2, 3, 80, 16, "bf16", SPLIT, 16),
    "split, 256": (ragged(3, 1, 6000), 2, 8, 256, 128, "bf16", SPLIT, 16),
    "split, 256, fp32": (ragged(4, 1, 4000), 1, 5, 256, 16, "f32", SPLIT, 16),
    "near, 128": ([(24, 3000), (40, 5000), (0, 3), (17, 2500)], 2, 4, 128, 32, "bf16", NEAR, 16),
    "near, 70 sequences": (ragged(70, 9, 3000), 1, 4, 64, 64, "bf16", NEAR, 16),
    "near, 80, fp32": ([(20, 2500), (9, 4100)], 2, 5, 80, 16, "f32", NEAR, 16),
    "near, 256": ([(33, 3300), (5, 2600)], 1, 8, 256, 32, "bf16", NEAR, 16),
    "eight waves, 128": ([(600, 600)], 32, 4, 128, 32, "bf16", TILES, 256),
    "eight waves, uneven": (UNEVEN, 16, 4, 128, 16, "bf16", TILES, 256),
    "eight waves, 64": (UNEVEN, 16, 4, 64, 64, "bf16", TILES, 256),
    "eight waves, 48": (UNEVEN, 16, 4, 48, 128, "bf16", TILES, 256),
    "eight waves, 112": ([(600, 600)], 32, 4, 112, 16, "bf16", TILES, 256),
    "eight waves, 64, fp32": (UNEVEN, 16, 4, 64, 32, "f32", TILES, 256),
    "eight waves, 32, fp32": ([(600, 700)], 32, 4, 32, 32, "f32", TILES, 256),
    "eight waves, 300 sequences": ([(20 + i % 41, 70 + i % 97) for i in range(300)], 2, 8, 32, 16, "bf16", TILES, 256),
    "four waves, 128": ([(700, 1500), (33, 40)], 8, 4, 128, 32, "bf16", TILES, 128),
    "four waves, 80": ([(400, 900)], 4, 8, 80, 16, "bf16", TILES, 128),
    "four waves, 192": ([(232, 440)], 16, 8, 192, 64, "bf16", TILES, 128),
    "four waves, 256": ([(600, 600)], 32, 4, 256, 32, "bf16", TILES, 128),
    "four waves, 64, fp32": ([(400, 900)], 4, 8, 64, 16, "f32", TILES, 128),
    "four waves, 128, fp32": ([(232, 440)], 16, 8, 128, 128, "f32", TILES, 128),
    "four waves, 176, fp32": ([(232, 380)], 16, 8, 176, 32, "f32", TILES, 128),
    "four waves, 192, fp32": ([(232, 380)], 16, 8, 192, 16, "f32", TILES, 128),
    "four waves, 240, fp32": ([(232, 380)], 16, 8, 240, 64, "f32", TILES, 128),
    "four waves, 256, fp32": ([(232, 380)], 16, 8, 256, 32, "f32", TILES, 128),
}


def setup(name, **kw):
    lens, heads, group, dim, page, dtype, kernel, rows = KERNELS[name]
    s = Setup(lens, heads, dim, page, **kw)
    return s, heads * group, dtype, [0] if heads == 1 else [0, heads - 1]


def runs_in(s, q_heads, dtype, name, window=0):
    """Whether the call takes the kernel that the case is meant for (as on 256 CUs)."""
    p = kv.attention_plan(s.cache, s.batch, s.tokens, q_heads, DT[dtype], window)
    return (p.kernel, p.tile_rows) == KERNELS[name][6:8]


@pytest.mark.parametrize("name", KERNELS)
def test_every_kernel(name):
    s, q_heads, dtype, hs = setup(name, seed=40, fill=0x7F)
    assert runs_in(s, q_heads, dtype, name)
    check(s, q_heads, dtype, kv_heads=hs)


@pytest.mark.parametrize("causal,scale", [(False, None), (True, 0.0), (True, -0.2), (False, -0.3), (True, 2.0)])
@pytest.mark.parametrize("name", ["rows, 150 sequences", "split, 80", "near, 128", "eight waves, uneven",
                                  "eight waves, 64, fp32", "four waves, 80", "four waves, 192, fp32"])
def test_every_kernel_scales_and_no_mask(name, causal, scale):
    s, q_heads, dtype, hs = setup(name, seed=41, fill=0xFF)
    assert runs_in(s, q_heads, dtype, name)
    check(s, q_heads, dtype, causal=causal, scale=scale, kv_heads=hs)


# (a window changes what a kernel costs and so the choice: here the shapes that keep theirs)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name,window", [
    ("rows, 70 sequences", 90), ("rows, 150 sequences", 1), ("rows, 129 sequences, fp32", 33),
    ("split, 100 sequences", 2100), ("split, 80", 3000), ("split, 256, fp32", 2500),
    ("near, 128", 2300), ("near, 80, fp32", 2222), ("near, 256", 2049),
    ("eight waves, 128", 200), ("eight waves, uneven", 130), ("eight waves, 48", 1), ("eight waves, 64, fp32", 77),
    ("four waves, 128", 300), ("four waves, 80", 65), ("four waves, 256", 100), ("four waves, 128, fp32", 150),
])
def test_every_kernel_windows(name, window, causal):
    s, q_heads, dtype, hs = setup(name, seed=42, fill=0x7F)
    assert runs_in(s, q_heads, dtype, name, window)
    check(s, q_heads, dtype, causal=causal, window=window, kv_heads=hs)


@pytest.mark.parametrize("name", ["rows, 70 sequences", "split, 80", "split, 256, fp32", "near, 128", "eight waves, 128",
                                  "eight waves, uneven", "eight waves, 64, fp32", "four waves, 128", "four waves, 80",
                                  "four waves, 256, fp32"])
def test_every_kernel_with_pages_missing(name):
    """Every fifth page of a table names none: past the cache, negative, in turn."""
    s, q_heads, dtype, hs = setup(name, seed=43, fill=0x7F)
    assert runs_in(s, q_heads, dtype, name)
    for i, n in enumerate(s.need):
        at = np.arange(2 + i % 3, n, 5)
        s.table[i, at] = np.resize([-1, s.ref.pages, 1 << 30, -7], len(at))
    s.batch.table.copy_(torch.from_numpy(s.table))
    check(s, q_heads, dtype, kv_heads=hs)


@pytest.mark.parametrize("low,high", [(-60, 60), (-20, 20), (-90, -90), (40, 40)])
@pytest.mark.parametrize("name", ["rows, 70 sequences", "split, 80", "near, 128", "eight waves, uneven", "eight waves, 64, fp32",
                                  "four waves, 80", "four waves, 240, fp32"])
def test_every_kernel_with_blocks_of_uneven_size(name, low, high):
    """V's block exponents far apart, and all of them far from one; blocks of zeros among them."""
    s, q_heads, dtype, hs = setup(name, seed=44)
    assert runs_in(s, q_heads, dtype, name)
    r = s.ref
    r.vs[:] = np.where(np.arange(r.pages)[:, None] % 2, 127 + high, 127 + low)
    r.v[s.table[0, 0]] = 0
    r.vs[s.table[0, 0]] = 0
    s.cache.v_codes.copy_(torch.from_numpy(r.v))
    s.cache.v_scales.copy_(torch.from_numpy(r.vs))
    check(s, q_heads, dtype, kv_heads=hs)


@pytest.mark.parametrize("name", ["rows, 150 sequences", "split, 80", "split, 256, fp32", "near, 128", "eight waves, uneven",
                                  "eight waves, 64, fp32", "four waves, 80", "four waves, 192, fp32"])
def test_weights_are_held_to_2_16(name):
    """A quarter of the keys have weight 1 and values -1, the others weight w near 1/3 and values 1: the
    numerator all but cancels, and weights of fewer bits would show (one bf16: 2^-9 of the sum). Shares
    here are of 512 keys, of at most 30 to a tile."""
    s, q_heads, dtype, hs = setup(name, seed=45)
    assert runs_in(s, q_heads, dtype, name)
    r = s.ref
    r.k[:], r.v[:], r.ks[:], r.vs[:] = 0, 0x38, 127, 127
    r.k[..., 0] = 0x38
    r.k[:, :, ::4] = 0
    r.v[..., ::4] = 0xB8
    for t, a in ((s.cache.k_codes, r.k), (s.cache.v_codes, r.v), (s.cache.k_scales, r.ks), (s.cache.v_scales, r.vs)):
        t.copy_(torch.from_numpy(a))
    q = s.draw(q_heads, dtype)
    q[:, :, 0] = -torch.linspace(1.0, 1.2, s.tokens * q_heads, device=DEV).view(s.tokens, q_heads).to(DT[dtype])
    split = KERNELS[name][6] in (SPLIT, NEAR)
    check(s, q_heads, dtype, causal=False, scale=1.0, q=q, kv_heads=hs, chain=512 + 2 + 30 if split else None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_shares_of_a_tile_than_a_join_has_threads(dtype):
    """293 shares of two units of 256 keys: sums go through at most 512 keys, two joins of waves and the
    shares."""
    s = Setup([(2, 150000)], 1, 16, 128, seed=46)
    assert kv.attention_plan(s.cache, s.batch, 2, 4, DT[dtype]).kernel == SPLIT
    check(s, 4, dtype, chain=512 + 2 + 293)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wide_tables_are_dealt_in_larger_units(dtype):
    """A table with room for 2^31 - 4096 tokens, 130 heads: units of 256 keys would be too many to count."""
    s = Setup([(1, 9000)], 130, 16, 128, seed=48)
    table = torch.full((1, 2 ** 24 - 32), -1, dtype=torch.int32, device=DEV)
    table[:, :s.table.shape[1]] = s.batch.table
    s.batch = kv.Batch(s.batch.cu_tokens, s.batch.context, table)
    assert kv.attention_plan(s.cache, s.batch, 1, 260, DT[dtype]).kernel == SPLIT
    check(s, 260, dtype, kv_heads=[0, 77, 129])


def test_a_tile_gives_the_same_bits_whatever_else_is_in_the_batch():
    """A prompt alone, and behind another one, both in tiles of 256 rows."""
    s = Setup([(576, 576), (576, 1000)], 16, 128, 32, seed=47)
    q = s.draw(128, "bf16")
    one = kv.Batch(torch.tensor([0, 576], dtype=torch.int32, device=DEV), s.batch.context[1:], s.batch.table[1:],
                   max_tokens=576, max_context=1000)
    for b, n in ((s.batch, 1152), (one, 576)):
        p = kv.attention_plan(s.cache, b, n, 128)
        assert (p.kernel, p.tile_rows) == (TILES, 256)
    assert torch.equal(kv.attention(q[576:], s.cache, one), kv.attention(q, s.cache, s.batch)[576:])


# ------------------------------------------------------------------------------------- long batches
def test_batches_of_more_pages_than_one_axis_of_a_launch_takes():
    """2^28 + 37 tokens of one head in pages of 16, more than 2^24 of them: written and read back, whole
    numbers that E4M3 holds exactly under any scale of theirs."""
    page, dim = 16, 16
    tokens = 2 ** 28 + 37
    pages = -(-tokens // page)
    g = torch.Generator(device=DEV).manual_seed(49)
    rows = torch.randint(-8, 9, (2, tokens, 1, dim), generator=g, device=DEV, dtype=torch.int8)
    k, v = rows[0].to(torch.bfloat16), rows[1].to(torch.bfloat16)
    cache = kv.empty_cache(pages, 1, page, dim, DEV)
    table = torch.arange(pages - 1, -1, -1, device=DEV, dtype=torch.int32)[None]
    batch = kv.Batch(torch.tensor([0, tokens], dtype=torch.int32, device=DEV),
                     torch.tensor([tokens], dtype=torch.int32, device=DEV), table)
    kv.append(cache, k, v, batch)
    for got, want in zip(kv.read(cache, batch, tokens), (k, v)):
        assert torch.equal(got, want)
    del rows, k, v, cache, got, want
    torch.cuda.empty_cache()


# --------------------------------------------------------------------------- one batch, many threads
def test_calls_of_different_row_counts_share_a_batch(monkeypatch):
    """A call with other rows that comes between the size query and the call of a first one (as another
    thread's may: the library's calls run without the interpreter's lock) takes nothing from it."""
    s = Setup([(4, 5000), (3, 4000)], 2, 64, 32, seed=50)
    q = s.draw(8, "bf16")
    want = kv.attention(q, s.cache, s.batch).clone()
    first = kv.attention(q[:4], s.cache, s.batch).clone()
    real, between = kv.lib().fp4_kv_attention_workspace_bytes, []

    def query(*args):
        n = real(*args)
        if not between:
            between.append(None)
            between.append(kv.attention(q[:4], s.cache, s.batch))
        return n

    monkeypatch.setattr(kv.lib(), "fp4_kv_attention_workspace_bytes", query)
    out = torch.full_like(q, math.nan)
    kv.attention(q, s.cache, s.batch, out=out)
    assert torch.equal(out, want) and torch.equal(between[1], first)


# -------------------------------------------------------------------------- batches that descend
@pytest.mark.parametrize("name", ["rows, 70 sequences", "split, 80", "near, 128", "eight waves, uneven", "four waves, 80"])
def test_batches_that_descend_touch_their_rows_only(name):
    """cu_tokens out of order and out of range: every call returns and stays inside the rows it was given,
    and the next call with a sound batch is right."""
    s, q_heads, dtype, hs = setup(name, seed=51)
    good = s.batch.cu_tokens.clone()
    g = torch.Generator(device=DEV).manual_seed(51)
    cu = good[torch.randperm(len(good), generator=g, device=DEV)]
    cu[0], cu[-1] = 2 ** 31 - 1, -5
    s.batch.cu_tokens.copy_(cu)
    room = torch.full((s.tokens + 20, q_heads, s.dim), 9.0, device=DEV, dtype=DT[dtype])
    kv.attention(s.draw(q_heads, dtype), s.cache, s.batch, out=room[10:-10])
    spaces = [torch.full((s.tokens + 20, s.heads, s.dim), 9.0, device=DEV, dtype=DT[dtype]) for _ in range(2)]
    kv.read(s.cache, s.batch, s.tokens, out=tuple(x[10:-10] for x in spaces))
    for x in (room, *spaces):
        assert (x[:10] == 9.0).all() and (x[-10:] == 9.0).all()
    s.batch.cu_tokens.copy_(good)
    check(s, q_heads, dtype, kv_heads=hs)


def test_queries_refuse_types_as_the_calls_do():
    s = Setup([(2, 20)], 2, 64, 16)
    for ask in (kv.attention_workspace_bytes, kv.attention_plan):
        with pytest.raises(TypeError):
            ask(s.cache, s.batch, 2, 4, torch.float16)
        with pytest.raises(Fp4Error):
            ask(s.cache, s.batch, 2, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_thousands_of_sequences_are_written_and_read(dtype):
    """More sequences than two steps of a search by 64 tell apart, every seventh without a row."""
    lens = [(i * 5 % 7, i * 5 % 7 + i % 40) for i in range(5000)]
    s = Setup(lens, 2, 16, 16, seed=52)
    k, v = s.draw(2, dtype), s.draw(2, dtype)
    ref.append(s.ref, host(k), host(v), s.cu, s.context, s.table, True)
    kv.append(s.cache, k, v, s.batch)
    for got, want in ((s.cache.k_scales, s.ref.ks), (s.cache.v_scales, s.ref.vs), (s.cache.k_codes, s.ref.k),
                      (s.cache.v_codes, s.ref.v)):
        assert np.array_equal(got.cpu().numpy(), want)
    for got, want in zip(kv.read(s.cache, s.batch, s.tokens), ref.read(s.ref, s.cu, s.context, s.table)):
        assert np.array_equal(host(got), rounded(want, "bf16"))
