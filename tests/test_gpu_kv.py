"""The 8-bit key / value cache on the GPU against its plain 64-bit form (kv_reference.py): writing is
compared code for code, reading value for value, attention within bounds that follow from its
arithmetic (test `bounds`)."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
from bit_gemm_fwht_amd import fp4, kv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Setup:
    """A cache full of finite random codes, uneven scales, shuffled pages, and a batch. lens: (new
    tokens, context) of each sequence."""

    def __init__(self, lens, kv_heads, dim, page, seed=0, spare=2, width=None, scale_spread=6, fill=None, hints=True):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.page, self.dim, self.heads = rng, lens, page, dim, kv_heads
        need = [-(-max(c, 0) // page) for _, c in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        width = width or max(max(need), 1)
        table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :min(n, width)] = order[at:at + min(n, width)]
            at += n
        codes = [rng.integers(0, 256, s, dtype=np.uint8) for s in
                 ((pages, kv_heads, page, dim), (pages, kv_heads, dim, page))]
        if fill is None:  # codes that a cache of normal values holds: mostly large ones of either sign
            codes = [np.where((c & 0x7F) == 0x7F, c ^ 1, c) for c in codes]
        scales = [(127 - 9 + rng.integers(-scale_spread, 1, (pages, kv_heads))).astype(np.uint8) for _ in range(2)]
        self.table, self.need = table, need
        self.ref = ref.Cache(codes[0], codes[1], scales[0], scales[1])
        if fill is not None:
            self.poison(fill)
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.context = np.array([c for _, c in lens], np.int32)
        self.tokens = int(self.cu[-1])
        dev = [torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in
               (self.ref.k, self.ref.v, self.ref.ks, self.ref.vs, self.cu, self.context, table)]
        self.cache = kv.KVCache(*dev[:4])
        self.hint = dict(max_tokens=max(n for n, _ in lens), max_context=max(max(c for _, c in lens), 1)) if hints else {}
        self.batch = kv.Batch(*dev[4:], **self.hint)

    def poison(self, code):
        """Set every place that holds no token to `code`."""
        r = self.ref
        used = np.zeros((r.pages, r.page), bool)
        for s, (_, ctx) in enumerate(self.lens):
            for j in range(self.need[s]):
                if j < self.table.shape[1]:
                    used[self.table[s, j], :max(0, min(self.page, ctx - j * self.page))] = True
        r.k[:] = np.where((r.k & 0x7F) == 0x7F, r.k ^ 1, r.k)
        r.v[:] = np.where((r.v & 0x7F) == 0x7F, r.v ^ 1, r.v)
        r.k[:] = np.where(used[:, None, :, None], r.k, code)
        r.v[:] = np.where(used[:, None, None, :], r.v, code)

    def draw(self, heads, dtype, size=1.0):
        x = (self.rng.standard_normal((self.tokens, heads, self.dim)) * size).astype(np.float32)
        return torch.from_numpy(x).to(DEV).to(DT[dtype])


def bounds(dtype, absv, mag, cnt, out):
    """How far the kernel's out may be from the exact one, and lse.
    Scores: the products with K are exact, D <= 256 additions and the scale multiply err by at most
    2^-23 of sum |q k| each (the matrix core's additions are taken as no better than truncating), so
    each score is off by es <= 258 * 2^-23 * mag; its difference to the maximum in log2 units is
    rounded once (2^-23 * 2 mag) and the exponential is good to 2 ulp: each weight is off by a factor
    1 +- (2 es + 2^-21 mag + 2^-21). Sums of n weights err by n 2^-23 of the sum of their sizes at most.
    That holds for the numerator (sizes w |v|) and the denominator. bf16 queries: weights rounded to
    bf16 (2^-9 each, numerator only) and the output rounded (2^-9). Rescales of the running sums: one
    rounding for each 64 keys, within n 2^-23."""
    es = 258 * 2.0 ** -23 * mag
    w = 2 * es + 2.0 ** -21 * mag + 2.0 ** -21 + cnt * 2.0 ** -23
    rel = 2 * w[..., None] + (2.0 ** -9 if dtype == "bf16" else 0.0)
    tol = rel * absv * 1.01 + np.abs(out) * (2.0 ** -9 * 1.01 if dtype == "bf16" else 2.0 ** -23) + 1e-37
    return tol, w + 2.0 ** -22 * (1 + mag + np.log(np.maximum(cnt, 1)))


def check_attention(s, q_heads, dtype, causal=True, window=0, scale=None, q=None, size=1.0, rel=None, **kw):
    q = s.draw(q_heads, dtype, size) if q is None else q
    lse = torch.full((s.tokens, q_heads), 7.0, device=DEV)
    o = kv.attention(q, s.cache, s.batch, scale=scale, causal=causal, window=window, lse=lse, **kw)
    torch.cuda.synchronize()
    eo, el, absv, mag, cnt = ref.attention(host(q), s.ref, s.cu, s.context, s.table,
                                           1 / math.sqrt(s.dim) if scale is None else scale, causal, window)
    tol, ltol = bounds(dtype, absv, mag, cnt, eo)
    assert o.shape == q.shape and o.dtype == q.dtype
    err = np.abs(host(o) - eo)
    assert np.isfinite(host(o)).all()
    assert (err <= tol).all(), f"worst excess {(err / tol).max():.3g}"
    none = cnt == 0
    got = host(lse)
    assert np.array_equal(np.isneginf(got), none)
    assert (np.abs(got[~none] - el[~none]) <= ltol[~none]).all()
    assert not host(o)[none].any()
    return o, lse


# ------------------------------------------------------------------------------------------- writing
APPEND = [
    # lens, kv heads, dim, page
    ([(1, 1)], 1, 16, 16),
    ([(1, 517)], 8, 128, 32),
    ([(1, 1), (1, 32), (1, 33), (1, 64), (1, 500)], 2, 64, 32),
    ([(33, 33), (0, 5), (7, 40), (16, 16), (64, 129)], 3, 80, 16),
    ([(300, 300), (129, 400)], 2, 256, 128),
    ([(5, 3), (4, 0), (3, 3)], 1, 48, 64),           # rows before the first token, an empty context
    ([(1, 100 + i) for i in range(70)], 1, 32, 16),  # more sequences than a wave has lanes
]


@pytest.mark.parametrize("rule", ["ceil", "floor"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,dim,page", APPEND)
def test_append_writes_the_reference_codes(lens, heads, dim, page, dtype, rule):
    s = Setup(lens, heads, dim, page, seed=1)
    k, v = s.draw(heads, dtype, 0.7), s.draw(heads, dtype, 30.0)
    mode = kv.SCALE_E8M0_CEIL if rule == "ceil" else kv.SCALE_E8M0_FLOOR
    ref.append(s.ref, host(k), host(v), s.cu, s.context, s.table, rule == "ceil")
    for again in range(2):  # the same tokens written again give the same cache
        kv.append(s.cache, k, v, s.batch, scale_mode=mode)
        for got, want in ((s.cache.k_scales, s.ref.ks), (s.cache.v_scales, s.ref.vs),
                          (s.cache.k_codes, s.ref.k), (s.cache.v_codes, s.ref.v)):
            assert np.array_equal(got.cpu().numpy(), want), again


def test_append_token_by_token_grows_the_scale():
    """A block written one token at a time, each larger than the one before, then smaller ones: the
    block's scale follows the largest, and older codes are carried over."""
    s = Setup([(1, 1), (1, 1)], 2, 64, 16, seed=2, width=3, spare=6)
    s.table[:] = [[0, 1, 2], [3, 4, 5]]
    s.batch.table.copy_(torch.from_numpy(s.table))
    for t in range(1, 41):
        s.context[:] = [t, t]
        s.batch.context.fill_(t)
        size = 2.0 ** (t % 13)
        k, v = s.draw(2, "f32", size), s.draw(2, "f32", 1 / size)
        kv.append(s.cache, k, v, s.batch)
        ref.append(s.ref, host(k), host(v), s.cu, s.context, s.table, True)
        assert np.array_equal(s.cache.k_scales.cpu().numpy(), s.ref.ks)
        assert np.array_equal(s.cache.v_scales.cpu().numpy(), s.ref.vs)
        assert np.array_equal(s.cache.k_codes.cpu().numpy(), s.ref.k)
        assert np.array_equal(s.cache.v_codes.cpu().numpy(), s.ref.v)


@pytest.mark.parametrize("rule", ["ceil", "floor"])
def test_append_extreme_values(rule):
    """Zeros, subnormals, the largest fp32, values at and around rounding and saturation boundaries."""
    s = Setup([(64, 64)], 1, 64, 16, seed=3)
    x = np.zeros((64, 1, 64), np.float32)
    x[0:16] = 0.0
    x[16:32] = s.rng.standard_normal((16, 1, 64)) * 1e-41
    x[32:48] = s.rng.uniform(-1, 1, (16, 1, 64)) * 3.4e38
    grid = ref.E4M3[:0x7F]
    mid = (grid[1:] + grid[:-1]) / 2
    vals = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), 0), np.nextafter(mid.astype(np.float32), 500),
                           [449.0, 460.0, 464.0, 479.9, 511.9]]).astype(np.float32)
    x[48:] = np.resize(np.concatenate([vals, -vals]), (16, 1, 64))
    x[48:, 0, 0] = 440.0
    k = torch.from_numpy(x).to(DEV)
    v = torch.from_numpy(np.ascontiguousarray(x[::-1])).to(DEV)
    kv.append(s.cache, k, v, s.batch, scale_mode=kv.SCALE_E8M0_CEIL if rule == "ceil" else kv.SCALE_E8M0_FLOOR)
    ref.append(s.ref, host(k), host(v), s.cu, s.context, s.table, rule == "ceil")
    assert np.array_equal(s.cache.k_scales.cpu().numpy(), s.ref.ks)
    assert np.array_equal(s.cache.k_codes.cpu().numpy(), s.ref.k)
    assert np.array_equal(s.cache.v_codes.cpu().numpy(), s.ref.v)


def test_append_takes_strided_rows_and_leaves_other_pages():
    """k and v as slices of one fused projection, heads broadcast, a table with pages that do not exist."""
    s = Setup([(40, 50), (20, 20)], 4, 64, 16, seed=4)
    s.table[0, 3] = s.ref.pages + 5  # tokens 48, 49 have no page
    s.table[1, 1] = -3               # tokens 16 .. 19
    s.batch.table.copy_(torch.from_numpy(s.table))
    qkv = torch.randn(s.tokens, 3, 4, 64, device=DEV, dtype=torch.bfloat16)
    k, v = qkv[:, 1], qkv[:, 2, :1].expand(-1, 4, -1)
    kv.append(s.cache, k, v, s.batch)
    ref.append(s.ref, host(k), host(v), s.cu, s.context, s.table, True)
    assert np.array_equal(s.cache.k_codes.cpu().numpy(), s.ref.k)
    assert np.array_equal(s.cache.v_codes.cpu().numpy(), s.ref.v)
    assert np.array_equal(s.cache.v_scales.cpu().numpy(), s.ref.vs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,dim,page", APPEND)
def test_read_gives_the_values_back(lens, heads, dim, page, dtype):
    s = Setup(lens, heads, dim, page, seed=5, scale_spread=40)
    out = [torch.full((s.tokens, 2, heads, dim), 7.0, device=DEV, dtype=DT[dtype])[:, i] for i in range(2)]
    got = kv.read(s.cache, s.batch, s.tokens, out=tuple(out))
    for g, want in zip(got, ref.read(s.ref, s.cu, s.context, s.table)):
        assert np.array_equal(host(g), np.where(np.isnan(want), 7.0, want))
    if not np.isnan(want).any():
        k, v = kv.read(s.cache, s.batch, s.tokens, dtype=DT[dtype])
        assert torch.equal(k, got[0]) and torch.equal(v, got[1])


# ----------------------------------------------------------------------------------------- attention
LENS = {
    "one": [(1, 1)],
    "short": [(1, 37)],
    "ragged": [(1, 1), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 700)],
    "drafts": [(5, 5), (3, 100), (1, 64), (7, 333)],
    "prompt": [(130, 130), (65, 65)],
    "chunks": [(64, 200), (17, 18), (100, 1000)],
    "empty": [(3, 0), (0, 10), (4, 2), (2, 50)],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("heads,group,dim,page", [(2, 1, 64, 16), (1, 4, 128, 32), (2, 5, 80, 64), (1, 8, 256, 128),
                                                  (1, 3, 16, 32), (1, 7, 112, 16), (1, 2, 192, 64)])
def test_attention(lens, heads, group, dim, page, dtype):
    s = Setup(LENS[lens], heads, dim, page, seed=6, fill=0x7F)  # NaN in every place without a token
    check_attention(s, heads * group, dtype)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 33), (False, 40), (True, 64), (True, 5000)])
@pytest.mark.parametrize("lens", ["ragged", "drafts", "chunks", "empty"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_masks(lens, causal, window, dtype):
    s = Setup(LENS[lens], 2, 64, 32, seed=7, fill=0xFF)
    check_attention(s, 6, dtype, causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hint", [None, (1, 100), (4, 5000), (100, 1 << 20)])
def test_attention_long_context_split_over_the_chip(hint, dtype):
    """Keys split over workgroups; hints, too small and too large ones among them, change no result
    beyond the order of sums."""
    s = Setup([(1, 5000), (4, 2500), (1, 1)], 2, 128, 32, seed=8)
    if hint:
        s.batch = kv.Batch(s.batch.cu_tokens, s.batch.context, s.batch.table, max_tokens=hint[0], max_context=hint[1])
    check_attention(s, 8, dtype)


def test_attention_window_does_not_look_at_pages_before_it():
    """Pages wholly before every window may be gone: their table entries name no page."""
    s = Setup([(1, 1000), (6, 800)], 2, 64, 16, seed=9)
    for i, (n, ctx) in enumerate(s.lens):
        gone = (ctx - n - 100 + 1) // 16
        r = s.table[i, :gone].copy()
        s.ref.k[r] = 0x7F
        s.ref.v[r] = 0x7F
        s.table[i, :gone] = [-1, 1 << 30] * (gone // 2) + [-1] * (gone % 2)
    s.cache.k_codes.copy_(torch.from_numpy(s.ref.k))
    s.cache.v_codes.copy_(torch.from_numpy(s.ref.v))
    s.batch.table.copy_(torch.from_numpy(s.table))
    check_attention(s, 4, "bf16", window=100)
    # pages missing in the middle of what is attended: their tokens are masked
    s.table[0, 60] = -7
    s.batch.table.copy_(torch.from_numpy(s.table))
    check_attention(s, 4, "bf16", window=100)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_extreme_scores_and_scales(dtype):
    """Scores of hundreds (weights underflow), a zero and a negative scale, block exponents far apart:
    a block of tiny V beside blocks of huge V."""
    s = Setup([(2, 300), (1, 90)], 1, 64, 16, seed=10, scale_spread=60)
    check_attention(s, 4, dtype, scale=1.0)
    check_attention(s, 4, dtype, scale=0.0)
    check_attention(s, 4, dtype, scale=-0.3)
    s.ref.vs[:] = np.where(np.arange(s.ref.pages)[:, None] % 2, 127 + 60, 127 - 60)
    s.ref.ks[:] = 127 - 8
    s.cache.v_scales.copy_(torch.from_numpy(s.ref.vs))
    s.cache.k_scales.copy_(torch.from_numpy(s.ref.ks))
    check_attention(s, 4, dtype)


@pytest.mark.parametrize("lens", ["short", "drafts", "chunks"])
def test_attention_takes_strided_queries_and_outputs(lens):
    s = Setup(LENS[lens], 2, 64, 32, seed=11)
    fused = torch.randn(s.tokens, 10, 64, device=DEV, dtype=torch.bfloat16)
    q = fused[:, 1:7]
    room = torch.full((6, s.tokens, 64), 9.0, device=DEV, dtype=torch.bfloat16)
    out = room.transpose(0, 1)
    o, _ = check_attention(s, 6, "bf16", q=q, out=out)
    assert o.data_ptr() == room.data_ptr()
    plain = kv.attention(q.contiguous(), s.cache, s.batch)
    assert torch.equal(plain, o)
    one = q[:, :1].expand(-1, 6, -1)  # one query head for all
    check_attention(s, 6, "bf16", q=one)


def test_rows_of_one_query_agree_whatever_they_are_batched_with():
    """The last row of a prompt, alone and within it, is the same query over the same keys."""
    s = Setup([(150, 400)], 2, 128, 32, seed=12)
    q = s.draw(8, "bf16")
    whole, _ = check_attention(s, 8, "bf16", q=q)
    for at in (0, 77, 149):
        cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        ctx = torch.tensor([250 + at + 1], dtype=torch.int32, device=DEV)
        one = kv.attention(q[at:at + 1], s.cache, kv.Batch(cu, ctx, s.batch.table))
        assert (one.float() - whole[at:at + 1].float()).abs().max() <= 2.0 ** -6 * whole[at].float().abs().max()


def test_same_call_gives_the_same_bits():
    s = Setup([(1, 4000), (1, 3000), (90, 500)], 2, 128, 32, seed=13)
    q = s.draw(8, "bf16")
    first = kv.attention(q, s.cache, s.batch)
    for _ in range(5):
        assert torch.equal(kv.attention(q, s.cache, s.batch), first)


def test_cache_beyond_32_bits():
    """Pages past 2^32 bytes: written, read back and attended."""
    heads, page, dim = 8, 128, 128
    pages = (1 << 32) // (heads * page * dim) + 40
    s = Setup([(1, 1)], heads, dim, page)
    cache = kv.KVCache(*(torch.zeros(sh, dtype=torch.uint8, device=DEV) for sh in
                         ((pages, heads, page, dim), (pages, heads, dim, page), (pages, heads), (pages, heads))))
    table = np.array([[pages - 1, 3, pages - 17]], np.int32)
    s.ref = ref.Cache(np.zeros((3, heads, page, dim), np.uint8), np.zeros((3, heads, dim, page), np.uint8),
                      np.zeros((3, heads), np.uint8), np.zeros((3, heads), np.uint8))
    s.lens, s.cu, s.context, s.tokens = [(300, 300)], np.array([0, 300], np.int32), np.array([300], np.int32), 300
    s.table = np.array([[0, 1, 2]], np.int32)
    s.cache = cache
    s.batch = kv.Batch(*(torch.from_numpy(a).to(DEV) for a in (s.cu, s.context, table)))
    k, v = s.draw(heads, "bf16"), s.draw(heads, "bf16")
    kv.append(cache, k, v, s.batch)
    ref.append(s.ref, host(k), host(v), s.cu, s.context, s.table, True)
    at = torch.from_numpy(table[0]).long().to(DEV)
    assert np.array_equal(cache.k_codes[at].cpu().numpy(), s.ref.k)
    assert np.array_equal(cache.v_codes[at].cpu().numpy(), s.ref.v)
    for g, want in zip(kv.read(cache, s.batch, 300), ref.read(s.ref, s.cu, s.context, s.table)):
        assert np.array_equal(host(g), want)
    check_attention(s, heads, "bf16")
    s.lens, s.cu = [(1, 300)], np.array([0, 1], np.int32)
    s.tokens = 1
    s.batch = kv.Batch(torch.from_numpy(s.cu).to(DEV), s.batch.context, s.batch.table)
    check_attention(s, heads, "bf16")


def test_a_step_on_another_stream_and_in_a_graph():
    """append + attention + read of a decode step: on a side stream, and captured and replayed with
    eager work between replays, against the eager results."""
    s = Setup([(1, 900), (1, 33), (1, 64)], 2, 128, 32, seed=14)
    k, v, q = s.draw(2, "bf16"), s.draw(2, "bf16"), s.draw(8, "bf16")
    state = [t.clone() for t in (s.cache.k_codes, s.cache.v_codes, s.cache.k_scales, s.cache.v_scales)]
    parts = (s.cache.k_codes, s.cache.v_codes, s.cache.k_scales, s.cache.v_scales)
    out = torch.zeros(3, 8, 128, device=DEV, dtype=torch.bfloat16)
    back = tuple(torch.zeros(3, 2, 128, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    ws = torch.empty(max(1, kv.attention_workspace_bytes(s.cache, s.batch, 3, 8)), dtype=torch.uint8, device=DEV)

    def step():
        kv.append(s.cache, k, v, s.batch)
        kv.attention(q, s.cache, s.batch, out=out, workspace=ws)
        kv.read(s.cache, s.batch, 3, out=back)

    def snapshot():
        torch.cuda.synchronize()
        return [t.clone() for t in (*parts, out, *back)]

    def reset():
        for t, o in zip(parts, state):
            t.copy_(o)
        out.fill_(3.0)
        for b in back:
            b.fill_(3.0)
        torch.cuda.synchronize()

    step()
    want = snapshot()
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    for a, b in zip(want, snapshot()):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(4):
        reset()
        kv.attention(q, s.cache, s.batch)  # eager work between replays
        torch.cuda.synchronize()
        g.replay()
        for i, (a, b) in enumerate(zip(want, snapshot())):
            assert torch.equal(a, b), (rep, i)


def test_no_rows():
    s = Setup([(0, 5), (0, 0)], 2, 64, 16)
    empty = torch.empty(0, 2, 64, device=DEV)
    kv.append(s.cache, empty, empty, s.batch)
    assert kv.attention(torch.empty(0, 4, 64, device=DEV), s.cache, s.batch).shape == (0, 4, 64)
    assert kv.read(s.cache, s.batch, 0)[0].shape == (0, 2, 64)


def test_binding_refuses_wrong_tensors():
    s = Setup([(2, 20)], 2, 64, 16)
    c = s.cache
    x = torch.randn(2, 2, 64, device=DEV)
    with pytest.raises(ValueError):
        kv.KVCache(c.k_codes, c.k_codes, c.k_scales, c.v_scales)  # V is [pages, heads, dim, page]
    with pytest.raises(ValueError):
        kv.KVCache(c.k_codes, c.v_codes, c.k_scales[:1], c.v_scales)
    with pytest.raises(ValueError):
        kv.KVCache(c.k_codes.cpu(), c.v_codes, c.k_scales, c.v_scales)
    with pytest.raises(ValueError):
        kv.Batch(s.batch.cu_tokens.long(), s.batch.context, s.batch.table)
    with pytest.raises(ValueError):
        kv.Batch(s.batch.cu_tokens, s.batch.context, s.batch.table.t())
    with pytest.raises(ValueError):
        kv.append(c, x, x[:1], s.batch)
    with pytest.raises(ValueError):
        kv.append(c, x, x.bfloat16(), s.batch)
    with pytest.raises(TypeError):
        kv.append(c, x.half(), x.half(), s.batch)
    with pytest.raises(ValueError):
        kv.append(c, x.cpu(), x.cpu(), s.batch)
    with pytest.raises(ValueError):
        kv.append(c, x[..., :32], x[..., :32], s.batch)
    with pytest.raises(ValueError):
        kv.attention(x.transpose(1, 2).contiguous().transpose(1, 2), c, s.batch)
    with pytest.raises(fp4.Fp4Error) as e:
        kv.attention(torch.randn(2, 3, 64, device=DEV), c, s.batch)  # 3 query heads on 2
    assert e.value.status == fp4.ERR_INVALID_ARG
    with pytest.raises(fp4.Fp4Error) as e:
        kv.attention(torch.randn(2, 4, 66, device=DEV)[..., 2:], c, s.batch)  # rows not 16-byte aligned
    assert e.value.status == fp4.ERR_ALIGNMENT
    with pytest.raises(ValueError):
        kv.attention(torch.randn(2, 4, 64, device=DEV), c, s.batch, lse=torch.zeros(2, 4))
    with pytest.raises(ValueError):
        kv.attention(torch.randn(2, 4, 64, device=DEV), c, s.batch, out=torch.zeros(2, 4, 64, device=DEV).bfloat16())


# -------------------------------------------------------- prompts: the kernel for many rows, both tile sizes
PROMPTS = {
    "whole": ([(700, 700)], 2, 3),
    "uneven": ([(300, 300), (1, 900), (0, 7), (129, 640), (64, 64)], 2, 4),
    "behind a context": ([(256, 1500), (33, 2000)], 4, 2),
    "many sequences": ([(40, 40 + i) for i in range(66)], 8, 2),  # tiles of 256 rows are too many for 128
    "no tokens before": ([(200, 150), (90, 90)], 2, 4),            # rows before the first token
}


@pytest.mark.parametrize("prompt", PROMPTS)
@pytest.mark.parametrize("dim,page,dtype", [(128, 32, "bf16"), (64, 16, "bf16"), (48, 128, "bf16"), (112, 64, "bf16"),
                                            (256, 32, "bf16"), (64, 64, "f32"), (128, 16, "f32")])
def test_attention_of_prompts(prompt, dim, page, dtype):
    lens, heads, group = PROMPTS[prompt]
    s = Setup(lens, heads, dim, page, seed=20, fill=0x7F)
    check_attention(s, heads * group, dtype)


@pytest.mark.parametrize("causal,window,scale", [(False, 0, None), (True, 100, None), (False, 77, None), (True, 1, None),
                                                 (True, 0, -0.2), (True, 0, 0.0), (True, 300, 3.0)])
def test_attention_of_prompts_masks_and_scales(causal, window, scale):
    lens, heads, group = PROMPTS["uneven"]
    s = Setup(lens, heads, 128, 32, seed=21, fill=0xFF)
    check_attention(s, heads * group, "bf16", causal=causal, window=window, scale=scale)


@pytest.mark.parametrize("low,high", [(-60, 60), (-20, 20), (-90, -90), (40, 40)])
def test_attention_of_prompts_with_blocks_of_uneven_size(low, high):
    """V's block exponents far apart, and all of them far from one; blocks of zeros among them (exponent
    -127, whose keys have their weights all the same)."""
    s = Setup([(500, 500)], 2, 64, 32, seed=22)
    r = s.ref
    r.vs[:] = np.where(np.arange(r.pages)[:, None] % 2, 127 + high, 127 + low)
    r.v[s.table[0, 5]] = 0
    r.vs[s.table[0, 5]] = 0
    s.cache.v_codes.copy_(torch.from_numpy(r.v))
    s.cache.v_scales.copy_(torch.from_numpy(r.vs))
    if low == -90:  # fp16 keeps what is above 2^-84 here: the absolute bound of the layout's description
        o = kv.attention(s.draw(4, "f32"), s.cache, s.batch)
        assert torch.isfinite(o).all() and o.abs().max() <= 448 * 2.0 ** -90
    else:
        check_attention(s, 4, "bf16")


def test_attention_of_prompts_with_pages_missing():
    s = Setup([(300, 600)], 2, 64, 16, seed=23)
    s.table[0, [7, 20, 30]] = [-1, s.ref.pages, 1 << 30]
    s.batch.table.copy_(torch.from_numpy(s.table))
    check_attention(s, 4, "bf16")


def test_attention_does_not_depend_on_what_else_is_in_the_batch():
    """A prompt alone, and behind another one, in one kernel: the same tiles, the same bits."""
    s = Setup([(400, 400), (400, 1000)], 2, 128, 32, seed=24)
    q = s.draw(8, "bf16")
    both = kv.attention(q, s.cache, s.batch)
    one = kv.attention(q[400:], s.cache, kv.Batch(torch.tensor([0, 400], dtype=torch.int32, device=DEV),
                                                  s.batch.context[1:], s.batch.table[1:], max_tokens=400, max_context=1000))
    assert (one.float() - both[400:].float()).abs().max() <= 2.0 ** -6 * both.float().abs().max()
