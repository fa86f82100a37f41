// Attention over the 8-bit key / value cache.
//
// With s_j = scale q.k_j, one pass over the keys keeps per query row the running maximum m, the sum
// l = sum exp(s_j - m) and o = sum exp(s_j - m) v_j, all fp32, rescaled when m grows; disjoint key
// ranges are joined by the same rule, so keys can be split over waves and workgroups.
//
// Both products run on the bf16 matrix cores: every E4M3 code times a power of two is exactly a bf16,
// so K and V enter exactly (the scaled convert applies V's block scale; K's multiplies the scores).
// The transposed products S^T = K Q^T and O^T = V^T P^T put a query row in a lane of every result, so
// m, l and the rescale need no broadcast, and the accumulator of S^T is, lane for lane, the second
// operand of O^T's instruction: contraction order is free, so the keys of a 64-key step are dealt
// such that the 16 scores that a lane holds belong to 16 consecutive keys. Those are 16 consecutive
// bytes of a channel of V as the cache stores it, and (page sizes being multiples of 16) lie in one
// page, under one scale. Nothing is transposed and nothing moves between lanes but the statistics.
#include <algorithm>
#include <type_traits>

#include "fp4_internal.h"
#include "kv_device.h"

namespace bgf {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kNegInf = -__builtin_huge_valf();

// 8 E4M3 codes times the power of two `scale` -> 8 bf16, exact
__device__ __forceinline__ bf16x8 cvt8(uint32_t a, uint32_t b, float scale) {
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
    return __builtin_bit_cast(bf16x8, r);
}

// 8 floats as sums of NS bf16. NS = 1: rounded. NS = 2: cut after 8 significant bits, the rest (below 2^-7 of
// the value's power of two) rounded to 8: 2^-16 off at most, which keeps softmax weights (rounded to one
// bf16 they would add as much error as the bf16 output's own rounding) out of the result for one more
// product; with a third the error against 64 bits stays the same to five digits (prompt of 4096 tokens
// 1.6112e-3, windowed chunks 1.6417e-3, the output's rounding). NS = 3: exact (the 24
// significant bits in three runs of 8), so that products with bf16 lose nothing of an fp32 operand.
// INF: the values may be infinite (queries); an infinity has no rest (inf - inf would be NaN).
template <int NS, bool INF>
__device__ __forceinline__ void split8(const float* x, bf16x8 (&out)[NS]) {
    u32x4 r[NS];
    if constexpr (NS == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[0][i] = pack_bf16x2_rne(x[2 * i], x[2 * i + 1]);
    } else {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (NS == 2 && n == 1) {
                    r[n][i] = pack_bf16x2_rne(y[2 * i], y[2 * i + 1]);
                    continue;
                }
                // the two high halves, the first value's in the low half of the word
                r[n][i] = __builtin_amdgcn_perm(__float_as_uint(y[2 * i + 1]), __float_as_uint(y[2 * i]), 0x07060302u);
                if (n + 1 < NS) {
#pragma unroll
                    for (int j = 2 * i; j < 2 * i + 2; ++j) {
                        const uint32_t cut = __float_as_uint(y[j]) & 0xFFFF0000u;
                        y[j] = INF && (cut & 0x7F800000u) == 0x7F800000u ? 0.0f : y[j] - __uint_as_float(cut);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) out[n] = __builtin_bit_cast(bf16x8, r[n]);
}

// One tile of TR query rows (a row = a token and one of the G query heads of a kv head, token major)
// and the keys that any of them may attend.
struct AttnTile {
    int s;            // sequence
    int tok0;         // first row of the sequence in the batch
    int r0, r1;       // its rows [r0, r1) of n * G
    int p0;           // position of the sequence's first row
    int keys;         // keys that exist: min(context, table)
    int lo, hi;       // keys that some row may attend (lo: past the keys where windows are)
    int flo, fhi;     // keys that every row may attend
};

// First key in the window of the query at position pos; below 0: every key is. (A query before the first
// token sees what the one at -1 sees: pos - window itself need not fit 32 bits.)
__device__ __forceinline__ int window_from(int pos, int window) { return max(pos, -1) - window + 1; }

template <int TR>
__device__ __forceinline__ AttnTile attn_tile(const KvAttnArgs& a, int s, int tile) {
    const KvView& c = a.c;
    AttnTile t;
    t.s = s;
    t.tok0 = cu_at(c, s);
    const int n = cu_at(c, s + 1) - t.tok0;
    t.r0 = tile * TR;
    t.r1 = min(t.r0 + TR, n * a.G);
    const int ctx = max(c.ctx[s], 0);
    t.keys = (int)min((int64_t)ctx, (int64_t)c.W << c.pshift);
    t.p0 = ctx - n;
    const int pa = t.p0 + t.r0 / a.G, pb = t.p0 + (t.r1 - 1) / a.G;  // positions of the first and last row
    t.hi = a.causal ? max(min(t.keys, pb + 1), 0) : t.keys;
    t.fhi = a.causal ? min(t.keys, pa + 1) : t.keys;
    t.lo = a.window ? max(window_from(pa, a.window), 0) : 0;
    t.flo = a.window ? window_from(pb, a.window) : 0;
    return t;
}

// One query row's softmax state at the end of a split: written as the output, or as a partial result.
__device__ __forceinline__ float safe_rcp(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? kNegInf : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

template <int DT>
__device__ __forceinline__ void store_out4(void* out, int64_t at, f32x4 y) {
    if constexpr (DT == DT_BF16) {
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + at) =
            make_uint2(pack_bf16x2_rne(y[0], y[1]), pack_bf16x2_rne(y[2], y[3]));
    } else {
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + at) = y;
    }
}

// ---------------------------------------------------------------------------------------------
// Few rows: tiles of 16, the keys dealt to the waves in steps of 64 each, straight from memory to
// registers (no two waves read the same key).
//
// What there is to do is counted in units of a.unit keys of a tile of a kv head (2^31: of whole tiles),
// sequence by sequence; every workgroup takes the same number of consecutive units (a.share_min at least), wherever in a tile
// they begin and end. However uneven the contexts, all CUs read as much: a step of 64 sequences of 4127
// tokens on average (32 heads on 8 kv heads, 554 MB) takes 113 + 9 us, 4.9 TB/s, two of 131071 tokens 98 + 9
// us, 5.4 TB/s of the 5.96 that plain reading reaches; bound by the reads and, where tiles change within a
// share, by the latency of the next one's first keys. A tile that lies
// within one workgroup's share is written as output. Of the others each workgroup leaves at most two
// partial results, of the tile that its share begins in (place 0) and of the one that it ends in
// (place 1), which k_kv_attn_join puts together.
// ---------------------------------------------------------------------------------------------
constexpr int kRows = 16;
constexpr uint32_t kWholeTiles = 1u << 31;  // a unit that no tile has two of

// the key that a sequence's units begin at; p0: position of its first row
__device__ __forceinline__ int units_from(const KvAttnArgs& a, int p0, int keys) {
    return a.window ? min(max(window_from(p0, a.window), 0), keys) & ~63 : 0;
}

// tiles of a sequence, units of each of them, and its units in all (-1: cu_tokens descends)
__device__ __forceinline__ int seq_units(const KvAttnArgs& a, int s, int* tiles, int* units) {
    const KvView& c = a.c;
    const int n = cu_at(c, s + 1) - cu_at(c, s), ctx = max(c.ctx[s], 0);
    const int keys = (int)min((int64_t)ctx, (int64_t)c.W << c.pshift);
    const int lo = units_from(a, ctx - n, keys);
    *tiles = max(n * a.G + kRows - 1, 0) / kRows;
    *units = keys > lo ? (int)(((uint32_t)(keys - lo) + a.unit - 1) / a.unit) : 1;
    return n < 0 ? -1 : c.H * *tiles * *units;
}

// The batch's units, and the place of one of them. All lanes of a wave take part; lane i counts
// sequence i of 64 at a time (what it counted is kept where there are no more).
struct Units {
    int total, share;
    int tiles, units, count, upto;  // lane i: sequence i's, and the units up to its end
};
__device__ __forceinline__ void count_64(const KvAttnArgs& a, int s0, Units* q) {
    const int lane = __lane_id(), s = s0 + lane;
    q->tiles = q->units = q->count = 0;
    if (s < a.c.S) q->count = seq_units(a, s, &q->tiles, &q->units);
    q->upto = q->count;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(q->upto, o);
        if (lane >= o) q->upto += v;
    }
}
__device__ __forceinline__ Units count_units(const KvAttnArgs& a) {
    Units q;
    q.total = 0;
    uint64_t down = 0;
    for (int s0 = 0; s0 < a.c.S; s0 += 64) {
        count_64(a, s0, &q);
        q.total += __builtin_amdgcn_readlane(q.upto, 63);
        down |= __ballot(q.count < 0);
    }
    // (the host holds the sum to kMaxUnits for rows that are counted once: a batch that descends has more)
    if (down) q.total = 0;
    q.share = max((int)(((unsigned)q.total + a.grid - 1) / (unsigned)a.grid), a.share_min);
    return q;
}
struct UnitPlace {
    int s, h, tile, u, units;  // unit u of `units` of a tile
};
__device__ __forceinline__ UnitPlace find_unit(const KvAttnArgs& a, Units& q, int at) {
    int before = 0, s0 = 0;
    if (a.c.S > 64) {
        for (;; s0 += 64) {
            count_64(a, s0, &q);
            const int n = __builtin_amdgcn_readlane(q.upto, 63);
            if (at < before + n || s0 + 64 >= a.c.S) break;
            before += n;
        }
    }
    const int i = __popcll(__ballot(before + q.upto <= at));  // sequences that end before
    UnitPlace p;
    p.s = s0 + min(i, 63);
    const int units = max(__builtin_amdgcn_readlane(q.units, min(i, 63)), 1);
    const int tiles = max(__builtin_amdgcn_readlane(q.tiles, min(i, 63)), 1);
    const int rel = at - before - __builtin_amdgcn_readlane(q.upto - q.count, min(i, 63));
    const int j = rel / units;
    p.u = rel - j * units;
    p.units = units;
    p.h = j / tiles;
    p.tile = j - p.h * tiles;
    return p;
}

constexpr float kSlack = 8.0f;

// Waves that a SIMD holds at once, by registers (a lane holds 16 U of K and V each on their way, 16 U of
// o, 8 U (fp32: 24 U) of q): two, or one.
constexpr int rows_waves(int dt, int u) { return (dt == DT_BF16 ? u <= 3 : u <= 2) ? 2 : 1; }

// Keys [begin, end) of a tile (begin a multiple of 64); part: place of the partial result, -1: output.
// U: 64-channel pieces of a head; FULL: the head fills them; NW: waves
template <int DT, int U, bool FULL, int NW>
__device__ __forceinline__ void attn_rows(const KvAttnArgs& a, const AttnTile& t, int h, int begin, int end, int part) {
    constexpr int NS = DT == DT_BF16 ? 1 : 3, NP = DT == DT_BF16 ? 2 : 3;  // bf16 a query and a weight take
    const KvView& c = a.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int D = FULL ? 64 * U : c.D, P = c.P;

    // this lane's query row
    const int r = t.r0 + li;
    const bool row_ok = r < t.r1;
    const int tok = row_ok ? r / a.G : 0;
    const int head = h * a.G + (row_ok ? r - tok * a.G : 0);
    const int pos = t.p0 + tok;
    const int row_hi = !row_ok ? 0 : a.causal ? min(t.keys, pos + 1) : t.keys;
    const int row_lo = a.window ? window_from(pos, a.window) : 0;
    f32x4 o[4 * U];
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) o[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    float m = kNegInf, l = 0.0f;

    const int gk = li >> 2;  // S^T row li of piece e is key 16 gk + 4 e + (li & 3) of the step
    // Order of a step: V on its way, the next step's pages looked up, scores from the K that the step
    // before has sent for, the next step's K (into the same registers) on its way, softmax, V's product.
    // Nothing is loaded under a condition (after a branch the compiler no longer knows what is still on
    // its way and waits for all of it): a lane with nothing to load reads page 0 and is masked below, a
    // piece past the head's channels is read from its start and not used, the last step's table entry
    // and next K are read from wherever the index was held to.
    const int32_t* const row = c.table + (int64_t)t.s * c.table_ld;
    const auto entry_of = [&](int key) { return row[min(key >> c.pshift, c.W - 1)]; };
    const auto page_of = [&](int entry, int key) {
        return key < t.hi && entry >= 0 && (int64_t)entry < c.pages ? entry : -1;
    };
    u32x4 kraw[4][U], vraw[4 * U];
    // K of the 16 keys at tk (this lane: its row of each of the four pieces) in page pk
    const auto load_k = [&](int tk, int pk) {
        const uint8_t* kp = c.kc + ((((int64_t)max(pk, 0) * c.H + h) << c.pshift) + (tk & (P - 1)) + (li & 3)) * D + 16 * g;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = FULL || 64 * u + 16 * g < D;
                kraw[e][u] = *reinterpret_cast<const u32x4*>(kp + 4 * e * D + (in ? 64 * u : -16 * g));
            }
    };
    int kb = begin + 64 * wave;
    int pv = page_of(entry_of(kb + 16 * g), kb + 16 * g);
    load_k(kb + 16 * gk, page_of(entry_of(kb + 16 * gk), kb + 16 * gk));
    bf16x8 qf[NS][2 * U];
    {
        const int64_t q0 = (int64_t)(t.tok0 + tok) * a.ldq + (int64_t)head * a.ldq_head;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int d = 64 * u + 16 * g;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.0f;
            if (row_ok && d < D) {
                if constexpr (DT == DT_BF16) {
                    const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.q) + q0 + d);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const u32x4 w = p[v];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[8 * v + 2 * i] = bf16_lo(w[i]);
                            x[8 * v + 2 * i + 1] = bf16_hi(w[i]);
                        }
                    }
                } else {
                    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(a.q) + q0 + d);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const f32x4 w = p[v];
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * v + i] = w[i];
                    }
                }
            }
            if (a.flip) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = -x[i];
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                bf16x8 f[NS];
                split8<NS, true>(x + 8 * w, f);
#pragma unroll
                for (int n = 0; n < NS; ++n) qf[n][2 * u + w] = f[n];
            }
        }
    }

#pragma unroll 1
    for (; kb < end; kb += 64 * NW) {
        const int tv = kb + 16 * g, tk_next = kb + 64 * NW + 16 * gk, tv_next = kb + 64 * NW + 16 * g;
        // (loads return in order: asked for after V, the pages and the scales would wait for it)
        const int ek = entry_of(tk_next), ev = entry_of(tv_next);
        const int64_t sb = (int64_t)max(pv, 0) * c.H + h;
        const uint32_t ks = c.ks[sb];
        uint32_t vs = c.vs[sb];
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t* vp = c.vc + (((int64_t)max(pv, 0) * c.H + h) * D + li) * P + (tv & (P - 1));
#pragma unroll
        for (int i = 0; i < 4 * U; ++i) vraw[i] = *reinterpret_cast<const u32x4*>(vp + (FULL || 16 * i < D ? 16 * i * P : 0));
        // q.k of this lane's row and keys kb + 16 g + 0 .. 15; times kscale: scores in log2 units
        float s[16];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f32x4 acc = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const bool in = FULL || 64 * u + 16 * g < D;
                    const bf16x8 kf = cvt8(in ? kraw[e][u][2 * w] : 0u, in ? kraw[e][u][2 * w + 1] : 0u, 1.0f);
#pragma unroll
                    for (int n = 0; n < NS; ++n) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[n][2 * u + w], acc, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * e + i] = acc[i];
        }
        __builtin_amdgcn_sched_barrier(0);
        const int pv_next = page_of(ev, tv_next);
        load_k(tk_next, page_of(ek, tk_next));
        __builtin_amdgcn_sched_barrier(0);

        // masks, where the step holds a key that some row may not attend or that is not there
        if (kb < t.flo || kb + 64 > t.fhi || __ballot(pv < 0)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = tv + i;
                if (!(pv >= 0 && key >= row_lo && key < row_hi)) s[i] = kNegInf;
            }
            // V where no row may attend is whatever memory held: made zero, as 0 * NaN is not 0; and so is
            // the scale of a block of which no row may attend any key (code 255 would make 0 * inf)
            if (pv < 0 || tv >= t.hi || tv + 16 <= t.lo) vs = 127;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n1 = pv < 0 ? 0 : min(max(t.hi - tv - 4 * j, 0), 4), n0 = min(max(t.lo - tv - 4 * j, 0), 4);
                uint32_t keep = n1 == 4 ? 0xFFFFFFFFu : (1u << (8 * n1)) - 1u;
                keep &= n0 == 4 ? 0u : 0xFFFFFFFFu << (8 * n0);
#pragma unroll
                for (int i = 0; i < 4 * U; ++i) vraw[i][j] &= keep;
            }
        }

        __builtin_amdgcn_sched_barrier(0);
        // one factor for all of a lane's scores, made positive and finite: the largest score is that of
        // the largest product, a masked product stays -inf
        const float kscale = __builtin_amdgcn_fmed3f(e8m0_value(ks) * a.scale_log2, 1e-37f, 3.40282347e38f);
        const float vscale = e8m0_value(vs);
        // m is a reference that no score exceeds by more than kSlack: weights stay below 2^kSlack, and
        // only where one would not are the row's lanes asked for the maximum and the sums rescaled
        float mx = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
        mx *= kscale;
        if (__ballot(mx > m + kSlack)) {
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = fmaxf(m, mx);
            const float f = __builtin_amdgcn_exp2f(m - (mn == kNegInf ? 0.0f : mn));
            l *= f;
#pragma unroll
            for (int i = 0; i < 4 * U; ++i) o[i] *= f;
            m = mn;
        }
        const float ms = m == kNegInf ? 0.0f : m;  // a row with no key so far: exp2(-inf) = 0
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], kscale, -ms));
            l += s[i];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            bf16x8 pf[NP];
            split8<NP, false>(s + 8 * w, pf);
#pragma unroll
            for (int i = 0; i < 4 * U; ++i) {
                const bf16x8 vf = cvt8(vraw[i][2 * w], vraw[i][2 * w + 1], vscale);
#pragma unroll
                for (int n = 0; n < NP; ++n) o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[n], o[i], 0, 0, 0);
            }
        }
        pv = pv_next;
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the waves' keys: the upper half into the lower until one is left
    __shared__ float sm[NW / 2][64], sl[NW / 2][64];
    __shared__ f32x4 so[NW / 2][4 * U][64];
#pragma unroll
    for (int half = NW / 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
            sm[wave - half][lane] = m;
            sl[wave - half][lane] = l;
#pragma unroll
            for (int i = 0; i < 4 * U; ++i) so[wave - half][i][lane] = o[i];
        }
        __syncthreads();
        if (wave < half) {
            const float m2 = sm[wave][lane], mn = fmaxf(m, m2);
            const float ms = mn == kNegInf ? 0.0f : mn;
            const float f = __builtin_amdgcn_exp2f(m - ms), f2 = __builtin_amdgcn_exp2f(m2 - ms);
            l = l * f + sl[wave][lane] * f2;
#pragma unroll
            for (int i = 0; i < 4 * U; ++i) o[i] = o[i] * f + so[wave][i][lane] * f2;
            m = mn;
        }
        __syncthreads();
    }
    if (wave != 0 || !row_ok) return;
    if (part < 0) {
        const float inv = safe_rcp(l);
        const int64_t o0 = (int64_t)(t.tok0 + tok) * a.ldo + (int64_t)head * a.ldo_head + 4 * g;
#pragma unroll
        for (int i = 0; i < 4 * U; ++i)
            if (16 * i < D) store_out4<DT>(a.out, o0 + 16 * i, o[i] * inv);
        if (a.lse && g == 0) a.lse[(int64_t)(t.tok0 + tok) * a.Hq + head] = lse_of(m, l);
    } else {
        const int64_t row = (int64_t)part * kRows + li;
#pragma unroll
        for (int i = 0; i < 4 * U; ++i)
            if (16 * i < D) *reinterpret_cast<f32x4*>(a.part_o + row * D + 16 * i + 4 * g) = o[i];
        if (g == 0) {
            a.part_ml[2 * row] = m;
            a.part_ml[2 * row + 1] = l;
        }
    }
}

template <int DT, int U, bool FULL, int NW>
__global__ __launch_bounds__(64 * NW, rows_waves(DT, U)) void k_kv_attn_rows(KvAttnArgs a) {
    Units q = count_units(a);
    // Workgroups go to the XCDs in turn: where a head has several tiles, shares that follow one another
    // stay on one XCD, so that those tiles meet in its L2 (8 sequences of 64 tokens, 32 heads on 8, over
    // 4000 keys: 162 -> 97 us). Tiles that share no keys stay in turn (64 sequences of 4127 tokens: 121 us
    // in turn, 127 us so).
    int w = blockIdx.x;
    if (a.near) {
        const int used = (q.total + q.share - 1) / q.share, x = w & 7;
        if (w >= used) return;
        w = x * (used >> 3) + min(x, used & 7) + (w >> 3);
    }
    int at = w * q.share;
    const int stop = min(at + q.share, q.total);
    while (at < stop) {
        const UnitPlace p = find_unit(a, q, at);
        const int u1 = min(p.units, p.u + stop - at);
        const AttnTile t = attn_tile<kRows>(a, p.s, p.tile);
        const int lo = units_from(a, t.p0, t.keys);
        const int begin = min(max(lo + p.u * (int)a.unit, t.lo & ~63), kMaxKeys);
        const int end = u1 == p.units ? t.hi : min(t.hi, lo + u1 * (int)a.unit);
        const bool whole = p.u == 0 && u1 == p.units;
        attn_rows<DT, U, FULL, NW>(a, t, p.h, begin, end, whole ? -1 : 2 * w + (p.u == 0));
        at += u1 - p.u;
    }
}

// The partial results of a row's key splits joined: workgroups (., w) for the tile that share w ends in, if
// it begins there too, a row each and the others of its rows in turn (as many workgroups as a tile is
// promised to have rows; it may have more). A workgroup's threads take 4 channels each and the splits in
// turn (all loads of a thread are independent of one another), then join over LDS, always in the same order.
template <int DT>
__global__ __launch_bounds__(256) void k_kv_attn_join(KvAttnArgs a) {
    const KvView& c = a.c;
    const int w = blockIdx.y, D = c.D;
    Units q = count_units(a);
    const int cut = (w + 1) * q.share;
    if (cut >= q.total) return;
    const UnitPlace p = find_unit(a, q, cut);
    const int first = cut - p.u;
    if (p.u == 0 || first < w * q.share) return;
    const AttnTile t = attn_tile<kRows>(a, p.s, p.tile);
    const int h = p.h, splits = (first + p.units - 1) / q.share - w + 1;
    const int tid = threadIdx.x;
    const int per = D >> 2, lanes = 256 / per;  // threads of one split; splits at once
    const int mine = tid / per, d = (tid - mine * per) * 4;
    __shared__ float sf[256];  // each split's factor exp2(m_z - m), 256 splits at a time
    __shared__ float sm[4];
    __shared__ f32x4 so[256];
#pragma unroll 1
    for (int rr = blockIdx.x; rr < t.r1 - t.r0; rr += gridDim.x) {
        // row of split z: place 1 of share w, then place 0 of those after it
        const auto row = [&](int z) { return ((int64_t)(2 * (w + z)) + (z == 0)) * kRows + rr; };
        float m = kNegInf;
        for (int z = tid; z < splits; z += 256) m = fmaxf(m, a.part_ml[2 * row(z)]);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
        if ((tid & 63) == 0) sm[tid >> 6] = m;
        __syncthreads();
        m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
        const float ms = m == kNegInf ? 0.0f : m;

        float l = 0.0f;
        f32x4 o = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        for (int z0 = 0; z0 < splits; z0 += 256) {
            const int n = min(256, splits - z0);
            __syncthreads();
            if (tid < n) {
                const float* ml = a.part_ml + 2 * row(z0 + tid);
                const float f = __builtin_amdgcn_exp2f(ml[0] - ms);
                sf[tid] = f;
                l += ml[1] * f;
            }
            __syncthreads();
            if (mine < lanes) {
#pragma unroll 4
                for (int z = mine; z < n; z += lanes)
                    o += *reinterpret_cast<const f32x4*>(a.part_o + row(z0 + z) * D + d) * sf[z];
            }
        }
        so[tid] = o;
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) l += __shfl_xor(l, i);
        if ((tid & 63) == 0) sm[tid >> 6] = l;  // every thread has read sm's maxima: two barriers since
        __syncthreads();
        if (mine == 0) {
            l = (sm[0] + sm[1]) + (sm[2] + sm[3]);
            for (int i = 1; i < lanes; ++i) o += so[i * per + tid];
            const int r = t.r0 + rr, tok = r / a.G, head = h * a.G + r - tok * a.G;
            store_out4<DT>(a.out, (int64_t)(t.tok0 + tok) * a.ldo + (int64_t)head * a.ldo_head + d, o * safe_rcp(l));
            if (a.lse && d == 0) a.lse[(int64_t)(t.tok0 + tok) * a.Hq + head] = lse_of(m, l);
        }
        __syncthreads();  // sm and so are the next row's
    }
}

// ---------------------------------------------------------------------------------------------
// Many rows: tiles of 32 rows for each of eight (or four) waves. The workgroup brings 64 keys at a time
// into LDS, once for all its rows, as bf16 under their blocks' scales (exact), converted on the way. A
// wave multiplies with 32x32x16 instructions; as above the accumulator of S^T is, once exponentials are
// taken, the second operand of O^T's product: 16 consecutive keys in a lane. Weights enter as sums of two
// bf16 (fp32 queries: three), cut and rounded next to the products, where the vector unit has time.
// A prompt of 4096 tokens and 32 heads of 128 takes 203 us, 680 TFLOP/s of attention (1020 of products),
// bound by the vector instructions of the softmax: a wave's step has 48 products (1536 clk) and over 300
// vector instructions, which beside a wave that multiplies take 7 to 12 clk each, so that a half step lasts
// 3400 clk and the matrix cores are busy 45 % of the time that CUs work.
// (Weights as one fp16 each take 160 us instead of 206 for a prompt of 4096 tokens and 32 heads, but lose channels to which
// only keys of small weight contribute: fp16 ends 2^-24 below 1.)
// ---------------------------------------------------------------------------------------------
constexpr int kTileKeys = 64;
constexpr int kAheadK = 2, kAheadV = 3;  // products whose operands are read from LDS ahead of their turn

// 16-byte pieces of a row of K (a key) and of V (a channel) in LDS, one more than its data so that rows
// next to one another begin 4 banks apart: eight lanes of any access reach 32 banks.
constexpr int tile_kp(int u) { return 8 * u + 1; }
constexpr int kTileVp = kTileKeys / 8 + 1;

// What one of 256 threads brings of each 64 keys of K (a key, and every fourth 16-byte piece of it) or
// of V (16 keys of every 64th channel): from memory to registers, and a step later to LDS, converted.
template <int U, bool FULL>
struct TileStager {
    const uint8_t* codes;
    const uint8_t* scales;
    const int32_t* row;  // the sequence's pages, from the one of key `tok` on
    u32x4* dst;
    uint32_t at, at_tok, at_u, page_bytes;
    int tok;   // first key of the 64 that the thread brings
    int need;  // its first channel
    int last;  // index from `row` of the table's last page
    bool is_v, there;
    u32x4 raw[U];
    uint32_t code;

    __device__ __forceinline__ void init(const KvView& c, int D, int s, bool v, int id, u32x4* kt, u32x4* vt) {
        const int r = id >> 2, q = id & 3;
        is_v = v;
        codes = v ? c.vc : c.kc;
        scales = v ? c.vs : c.ks;
        tok = v ? 16 * q : r;
        need = v ? r : 16 * q;
        row = c.table + (int64_t)s * c.table_ld;
        last = c.W - 1;
        const int srow = (r & 32) + 8 * ((r >> 2) & 3) + 4 * ((r >> 4) & 1) + (r & 3);  // S^T's row of key r
        dst = v ? vt + r * kTileVp + 2 * q : kt + srow * tile_kp(U) + 2 * q;
        page_bytes = (uint32_t)(c.P * D);
        at_tok = v ? 1 : D;
        at_u = v ? 64 * c.P : 64;
        at = (v ? r * c.P : 16 * q) + (tok & (c.P - 1)) * at_tok;
    }
    // (kb is a multiple of 64 and tok below 64: the page index and the place in the page are each the
    // sum of one of kb and one of tok)
    __device__ __forceinline__ int entry(const KvView& c, int kb) const {
        return row[min((kb >> c.pshift) + (tok >> c.pshift), last)];
    }
    __device__ __forceinline__ void load(const KvView& c, int h, int hi, int kb, int e, int D) {
        there = kb + tok < hi && (uint32_t)e < (uint32_t)c.pages;
        const uint32_t blk = (there ? (uint32_t)e : 0u) * (uint32_t)c.H + h;
        code = scales[blk];
        const uint8_t* p = codes + (uint64_t)blk * page_bytes + (at + (kb & (c.P - 1)) * at_tok);
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = *reinterpret_cast<const u32x4*>(p + (FULL || 64 * u + need < D ? (int)(u * at_u) : -(int)at));
    }
    __device__ __forceinline__ void stage(int D, const AttnTile& t, int kb, int buf, int* some, int id) {
        float scale = e8m0_value(code);
        if (is_v) {
            const int tv = kb + tok;
            if (kb < t.lo || kb + kTileKeys > t.hi || __ballot(!there)) {
                // what no row may attend is made zero, and its block's scale one (0 * inf is not 0)
                if (!there || tv + 16 <= t.lo) scale = 1.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n1 = there ? min(max(t.hi - tv - 4 * j, 0), 4) : 0, n0 = min(max(t.lo - tv - 4 * j, 0), 4);
                    uint32_t keep = n1 == 4 ? 0xFFFFFFFFu : (1u << (8 * n1)) - 1u;
                    keep &= n0 == 4 ? 0u : 0xFFFFFFFFu << (8 * n0);
#pragma unroll
                    for (int u = 0; u < U; ++u) raw[u][j] &= keep;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4* d = dst + buf * (64 * U * kTileVp) + 64 * u * kTileVp;
                d[0] = __builtin_bit_cast(u32x4, cvt8(raw[u][0], raw[u][1], scale));
                d[1] = __builtin_bit_cast(u32x4, cvt8(raw[u][2], raw[u][3], scale));
            }
            if (id < 4) some[4 * buf + id] = there;
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4 w = raw[u];
                if (!FULL && 64 * u + need >= D) w = (u32x4){0, 0, 0, 0};
                u32x4* d = dst + buf * (kTileKeys * tile_kp(U)) + 8 * u;
                d[0] = __builtin_bit_cast(u32x4, cvt8(w[0], w[1], scale));
                d[1] = __builtin_bit_cast(u32x4, cvt8(w[2], w[3], scale));
            }
        }
    }
};

// Eight waves, half of them bringing K and half V; four that bring both where registers ask for it, or
// where tiles of 256 rows would leave CUs without one.
constexpr int tile_nw(int dt, int u) { return (dt == DT_BF16 ? u <= 2 : u == 1) ? 8 : 4; }

template <int DT, int U, bool FULL, int NW>
__global__ __launch_bounds__(64 * NW, tile_nw(DT, U) / 4) void k_kv_attn_tiles(KvAttnArgs a) {
    constexpr int NS = DT == DT_BF16 ? 1 : 3, NP = DT == DT_BF16 ? 2 : 3, TR = 32 * NW;
    constexpr int KP = tile_kp(U), VP = kTileVp;
    const KvView& c = a.c;
    const int D = FULL ? 64 * U : c.D;
    // kv head fastest: workgroups go to the XCDs in turn, so the tiles of a head meet in one L2; the
    // tiles at a sequence's end, with the most keys, first
    const int h = blockIdx.x % c.H, slot = (int)a.slots - 1 - (int)(blockIdx.x / c.H);
    int first;
    const int s = find_sequence(c, slot, a.G, TR, 1, &first);
    if (s < 0) return;
    const AttnTile t = attn_tile<TR>(a, s, slot - first);
    if (t.r0 >= t.r1) return;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 31, hf = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    __shared__ u32x4 kt[2][kTileKeys * KP];
    constexpr int NV = NW == 8 ? 3 : 2;  // buffers of V
    __shared__ u32x4 vt[NV][64 * U * VP];
    __shared__ int there[NV][4];  // whether each 16 keys have a page
    constexpr int NB = NW == 8 ? 1 : 2;
    TileStager<U, FULL> st[NB];
    int entry[NB];
    const int id = tid & 255;
#pragma unroll
    for (int i = 0; i < NB; ++i) st[i].init(c, D, t.s, NW == 8 ? wave >= 4 : i == 1, id, &kt[0][0], &vt[0][0]);
    const auto entries = [&](int kb) {
#pragma unroll
        for (int i = 0; i < NB; ++i) entry[i] = st[i].entry(c, kb);
    };
    const auto load = [&](int kb) {
#pragma unroll
        for (int i = 0; i < NB; ++i) st[i].load(c, h, t.hi, kb, entry[i], D);
    };
    const auto stage = [&](int buf, int vbuf, int kb) {
#pragma unroll
        for (int i = 0; i < NB; ++i) st[i].stage(D, t, kb, st[i].is_v ? vbuf : buf, &there[0][0], id);
    };

    int kb = min(t.lo, t.keys) & ~(kTileKeys - 1);
    entries(kb);
    load(kb);
    entries(kb + kTileKeys);

    // the wave's 32 query rows, and the keys that some and that all of them may attend
    const int r = t.r0 + 32 * wave + li;
    const bool ok = r < t.r1;
    const int tok = ok ? r / a.G : 0, head = h * a.G + (ok ? r - tok * a.G : 0), pos = t.p0 + tok;
    const int row_hi = !ok ? 0 : a.causal ? min(t.keys, pos + 1) : t.keys;
    const int row_lo = a.window ? window_from(pos, a.window) : 0;
    const int ra = t.r0 + 32 * wave, rb = min(ra + 32, t.r1) - 1;
    const int pa = t.p0 + ra / a.G, pb = t.p0 + rb / a.G;
    const int w_hi = ra > rb ? 0 : a.causal ? min(t.keys, pb + 1) : t.keys, w_lo = a.window ? window_from(pa, a.window) : 0;
    const int w_fhi = a.causal ? min(t.keys, pa + 1) : t.keys, w_flo = a.window ? window_from(pb, a.window) : 0;
    bf16x8 qf[NS][4 * U];
    {
        const int64_t q0 = (int64_t)(t.tok0 + tok) * a.ldq + (int64_t)head * a.ldq_head;
#pragma unroll
        for (int k = 0; k < 4 * U; ++k) {
            const int d = 16 * k + 8 * hf;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.0f;
            if (ok && (FULL || d < D)) {
                if constexpr (DT == DT_BF16) {
                    const u32x4 w = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.q) + q0 + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[2 * i] = bf16_lo(w[i]);
                        x[2 * i + 1] = bf16_hi(w[i]);
                    }
                } else {
                    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(a.q) + q0 + d);
                    const f32x4 w0 = p[0], w1 = p[1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = w0[i], x[4 + i] = w1[i];
                }
            }
            if (a.flip) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = -x[i];
            }
            bf16x8 f[NS];
            split8<NS, true>(x, f);
#pragma unroll
            for (int n = 0; n < NS; ++n) qf[n][k] = f[n];
        }
    }
    f32x16 o[2 * U];
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) o[i] = (f32x16)(0.0f);
    float m = kNegInf, l = 0.0f;
    const float scale = __builtin_amdgcn_fmed3f(a.scale_log2, 1e-37f, 3.40282347e38f);

    stage(0, 0, kb);
    load(kb + kTileKeys);
    entries(kb + 2 * kTileKeys);
    __syncthreads();
    int buf = 0, vbuf = 0;  // of this step
    // Of eight waves the two halves (a wave of each on every SIMD) work half a step apart: while one
    // multiplies (the weights of the step before with V, then K with q), the other is at its softmax, and
    // the barriers between the halves of a step keep it so: waves of one SIMD in the same half compete
    // for one unit and leave the other idle. In the half in
    // which they multiply the first four waves write the next step's K to LDS and the last four its V: K
    // takes the place of the K before this step's, which every wave is done with by then, and V, still
    // wanted half a step longer, has three places. (Four waves write in the other half, all at once.)
    const auto meet = [] {
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x16 x[2];  // q.k, then weights
    const auto qk = [&](int buf) {
        bf16x8 kf[4 * U][2];
        const auto read_k = [&](int k) {
#pragma unroll
            for (int j = 0; j < 2; ++j) kf[k][j] = __builtin_bit_cast(bf16x8, kt[buf][(32 * j + li) * KP + 2 * k + hf]);
        };
#pragma unroll
        for (int k = 0; k < kAheadK; ++k) read_k(k);
#pragma unroll
        for (int k = 0; k < 4 * U; ++k) {
            if (k + kAheadK < 4 * U) read_k(k + kAheadK);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    x[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[k][j], qf[n][k], k + n ? x[j] : (f32x16)(0.0f), 0, 0, 0);
        }
    };
    const auto pv = [&](int buf) {
        bf16x8 vf[8 * U];
        const auto read_v = [&](int n) {  // n: channels 32 (n % 2U) .., 8 keys n / 2U
            const int i = n % (2 * U), w = n / (2 * U);
            vf[n] = __builtin_bit_cast(bf16x8, vt[buf][(32 * i + li) * VP + 4 * (w >> 1) + 2 * hf + (w & 1)]);
        };
#pragma unroll
        for (int n = 0; n < kAheadV; ++n) read_v(n);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[w >> 1][8 * (w & 1) + i];
            bf16x8 pf[NP];
            split8<NP, false>(p, pf);
#pragma unroll
            for (int i = 0; i < 2 * U; ++i) {
                const int n = 2 * U * w + i;
                if (n + kAheadV < 8 * U) read_v(n + kAheadV);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int q = 0; q < NP; ++q) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[n], pf[q], o[i], 0, 0, 0);
            }
        }
    };
    const auto softmax = [&](int buf, int kb, const bool masked) {
        if (masked) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool page = there[buf][2 * j + hf] != 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = kb + 32 * j + 16 * hf + i;
                    if (!(page && key >= row_lo && key < row_hi)) x[j][i] = kNegInf;
                }
            }
        }
        float mx = x[0][0];
#pragma unroll
        for (int i = 1; i < 32; ++i) mx = fmaxf(mx, x[i >> 4][i & 15]);
        mx *= scale;
        if (__ballot(mx > m + kSlack)) {
            const float mn = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32)));
            const float f = __builtin_amdgcn_exp2f(m - (mn == kNegInf ? 0.0f : mn));
            l *= f;
#pragma unroll
            for (int i = 0; i < 2 * U; ++i) o[i] *= f;
            m = mn;
        }
        const float ms = m == kNegInf ? 0.0f : m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i >> 4][i & 15], scale, -ms));
            x[i >> 4][i & 15] = p;
            sum[i & 3] += p;
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    };
    bool weights = false;  // whether the step before left any to multiply with V
    if (NW == 8 && wave >= 4) meet();
#pragma unroll 1
    for (; kb < t.hi; kb += kTileKeys) {
        const bool some = kb < w_hi && kb + kTileKeys > w_lo;
        const int vlast = vbuf == 0 ? NV - 1 : vbuf - 1, vnext = vbuf == NV - 1 ? 0 : vbuf + 1;
        if (weights) pv(vlast);
        if (some) qk(buf);
        if constexpr (NW == 8) stage(buf ^ 1, vnext, kb + kTileKeys);
        meet();
        weights = some;
        if (some) {
            const int* at = there[vbuf];
            softmax(vbuf, kb, kb < w_flo || kb + kTileKeys > w_fhi || !(at[0] && at[1] && at[2] && at[3]));
        }
        if constexpr (NW == 4) stage(buf ^ 1, vnext, kb + kTileKeys);
        load(kb + 2 * kTileKeys);
        entries(kb + 3 * kTileKeys);
        meet();
        buf ^= 1;
        vbuf = vnext;
    }
    if (weights) pv(vbuf == 0 ? NV - 1 : vbuf - 1);
    if (NW == 8 && wave < 4) meet();

    l += __shfl_xor(l, 32);
    if (!ok) return;
    const float inv = safe_rcp(l);
    const int64_t o0 = (int64_t)(t.tok0 + tok) * a.ldo + (int64_t)head * a.ldo_head + 4 * hf;
#pragma unroll
    for (int i = 0; i < 2 * U; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!FULL && 32 * i + 8 * e >= D) continue;
            const f32x4 y = {o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
            store_out4<DT>(a.out, o0 + 32 * i + 8 * e, y * inv);
        }
    if (a.lse && hf == 0) a.lse[(int64_t)(t.tok0 + tok) * a.Hq + head] = lse_of(m, l);
}

static int cu_count() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
        return 256;
    return n;
}

KvAttnPlan plan_kv_attention(const KvView& c, int Hq, int window, int dtype, int max_tokens, int max_context) {
    KvAttnPlan p{};
    const int G = Hq / c.H, U = (c.D + 63) / 64, cus = cu_count();
    dtype = dtype == DT_BF16 ? DT_BF16 : DT_F32;
    // keys that one tile goes through, at most
    const int64_t room = (int64_t)c.W << c.pshift;
    int64_t keys = room;
    if (max_context > 0) keys = std::min<int64_t>(keys, max_context);
    if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window + std::max(max_tokens, 1) + 64);
    // tiles of r rows that have any, at most
    const auto tiles_of = [&](int r) {
        int64_t n = (int64_t)c.T * G / r + c.S;
        if (max_tokens > 0) n = std::min(n, c.S * (((int64_t)max_tokens * G + r - 1) / r));
        return n * c.H;
    };
    const int64_t tiles = tiles_of(kRows);

    // Which kernel: by the time of their steps of 64 keys, as measured, every tile taken to go through all
    // keys. In rows of 16 a wave's step takes 3 us (2.5 us where tiles of a head meet in L2, 5 to 7 us where
    // every step comes from memory, as only few rows do), with 4 or 8 waves on a CU at a time whatever the
    // number of tiles, and splitting and joining take about 15 us; in tiles a workgroup goes through all of
    // its tile's keys: a step of four waves takes 2.1 us alone on a CU, 2.7 us with a second workgroup there,
    // one of eight waves 3.0 us, and more where a lane holds more. (4096 tokens of 32 heads: 203 us in
    // tiles, 639 us in rows; 500 over 500 tokens of 32 heads on 8: 23 and 44 us; 512 rows of one head over
    // 32000 keys: 1.0 ms in tiles, 52 us in rows; 512 rows of 32 heads over 4096 keys: 134 and 96 us; wrong
    // for prompts of fp32 heads of 256, whose causal tiles have half the steps: 2048 tokens of 32 heads go
    // to rows, 422 us, and would take 270 us in tiles.) Tiles are of 128 rows unless there are more of them
    // than two for a CU.
    const bool wide = tile_nw(dtype, U) == 8;  // the variants of which two workgroups fit a CU
    const int nw = wide && tiles_of(128) > 2 * cus ? 8 : 4;
    const auto steps_of = [&](int r) {
        const int64_t k = window > 0 ? std::min<int64_t>(keys, (int64_t)window + r / G + 64) : keys;
        return (double)((k + 63) / 64);
    };
    const int64_t at_once = (int64_t)cus * (wide && nw == 4 ? 2 : 1), ntiles = tiles_of(32 * nw);
    const double step_us = wide ? (nw == 8 ? 3.0 : ntiles <= cus ? 2.1 : 2.7) : dtype == DT_BF16 ? 3.9 : U == 2 ? 3.0 : 7.6;
    const double tiles_us = step_us * steps_of(32 * nw) * (double)((ntiles + at_once - 1) / at_once);
    const double rows_us = 15.0 + 3.0 * steps_of(kRows) * (double)tiles / (4.0 * rows_waves(dtype, U) * cus);
    const int64_t slots = (int64_t)c.T * G / (32 * nw) + c.S;
    if ((int64_t)c.T * G >= 2 * kRows * (int64_t)c.S && tiles_us < rows_us && slots * c.H <= kMaxGrid) {
        p.tile_slots = (int)slots;
        p.nw = nw;
        return p;
    }
    const int64_t most = ((int64_t)c.T * G / kRows + c.S) * c.H;  // tiles, whatever the hints were
    const int waves = rows_waves(dtype, U);
    if (keys <= 2048) {
        // Short contexts: a workgroup for each tile, of eight waves where registers allow, and one launch
        // (600 tokens of 8 kv heads: 11.7 us, in shares 13.5 + 4.2 us for the join; 64 sequences of up to
        // 2000 tokens: 41 us against 50, all of 2000: 60 us against 57).
        p.nw = 4 * waves;
        p.unit = kWholeTiles;
        p.share_min = 1;
        p.grid = (int)std::min(std::min(tiles, most), kMaxGrid);
    } else {
        // Shares: four waves, so that a CU has a second workgroup to read for while one changes tiles or
        // joins its waves (64 sequences of 4127 tokens on average: 115 us, with one of eight 140 us).
        // Units of 256 keys, or of as many more as keep their number, and the places that shares begin and
        // end at, within 32 bits for whatever contexts the table has room for.
        p.nw = 4;
        p.unit = 256;
        while (most * (room / p.unit + 1) > kMaxUnits) p.unit *= 2;
        p.share_min = 2;
        p.near = (int64_t)c.T * G > kRows * (int64_t)c.S;
        p.grid = cus * waves;
        // (workgroups of the join for a tile: its rows, if the hint holds; each goes on to further rows)
        p.join_rows = (int)std::min<int64_t>(max_tokens > 0 ? (int64_t)max_tokens * G : kRows, kRows);
        p.ws = (int64_t)p.grid * 2 * kRows * (c.D + 2) * 4;
    }
    return p;
}

template <int DT, int U, int NW>
static void launch_rows_nw(const KvAttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.grid);
    if (a.c.D == 64 * U) hipLaunchKernelGGL((k_kv_attn_rows<DT, U, true, NW>), grid, dim3(64 * NW), 0, s, a);
    else hipLaunchKernelGGL((k_kv_attn_rows<DT, U, false, NW>), grid, dim3(64 * NW), 0, s, a);
}

template <int DT, int U, int NW>
static void launch_tiles(const KvAttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.slots * a.c.H);
    if (a.c.D == 64 * U) hipLaunchKernelGGL((k_kv_attn_tiles<DT, U, true, NW>), grid, dim3(64 * NW), 0, s, a);
    else hipLaunchKernelGGL((k_kv_attn_tiles<DT, U, false, NW>), grid, dim3(64 * NW), 0, s, a);
}

template <int DT, int U>
static void launch_one(const KvAttnArgs& a, int nw, hipStream_t s) {
    if (a.slots) {
        if constexpr (tile_nw(DT, U) == 8) {
            if (nw == 8) return launch_tiles<DT, U, 8>(a, s);
        }
        return launch_tiles<DT, U, 4>(a, s);
    }
    if constexpr (rows_waves(DT, U) == 2) {
        if (nw == 8) return launch_rows_nw<DT, U, 8>(a, s);
    }
    launch_rows_nw<DT, U, 4>(a, s);
}

template <int DT>
static hipError_t launch_dt(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
    switch ((a.c.D + 63) / 64) {
        case 1: launch_one<DT, 1>(a, p.nw, s); break;
        case 2: launch_one<DT, 2>(a, p.nw, s); break;
        case 3: launch_one<DT, 3>(a, p.nw, s); break;
        default: launch_one<DT, 4>(a, p.nw, s); break;
    }
    if (p.join_rows)
        hipLaunchKernelGGL((k_kv_attn_join<DT>), dim3((unsigned)p.join_rows, (unsigned)a.grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_attention(KvAttnArgs a, const KvAttnPlan& p, int dtype, void* ws, hipStream_t s) {
    a.slots = p.tile_slots;
    a.grid = p.grid;
    a.unit = p.unit;
    a.share_min = p.share_min;
    a.near = p.near;
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = a.part_o + (int64_t)p.grid * 2 * kRows * a.c.D;
    return dtype == DT_BF16 ? launch_dt<DT_BF16>(a, p, s) : launch_dt<DT_F32>(a, p, s);
}

}  // namespace bgf
