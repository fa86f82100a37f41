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

// 8 floats as sums of NS bf16. NS = 1: rounded. NS = 2: cut after 8 significant bits, the rest rounded:
// 2^-17 off at most, which keeps softmax weights (rounded to one bf16 they would add as much error as
// the bf16 output's own rounding) out of the result for one more product. NS = 3: exact (the 24
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
    int lo, hi;       // keys that some row may attend
    int flo, fhi;     // keys that every row may attend
};

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
    t.lo = a.window ? max(pa - a.window + 1, 0) : 0;
    t.flo = a.window ? pb - a.window + 1 : 0;
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
// What there is to do is counted in units of a.unit keys of a tile of a kv head, sequence by sequence;
// every workgroup takes the same number of consecutive units (a.share_min at least), wherever in a tile
// they begin and end. However uneven the contexts, all CUs read as much: a step of 64 sequences of 4127
// tokens on average takes 104 us so, and 126 us with one workgroup for each tile. A tile that lies
// within one workgroup's share is written as output. Of the others each workgroup leaves at most two
// partial results, of the tile that its share begins in (place 0) and of the one that it ends in
// (place 1), which k_kv_attn_join puts together.
// ---------------------------------------------------------------------------------------------
constexpr int kRows = 16;

// tiles of a sequence, units of each of them, and its units in all
__device__ __forceinline__ int seq_units(const KvAttnArgs& a, int s, int* tiles, int* units) {
    const KvView& c = a.c;
    const int n = cu_at(c, s + 1) - cu_at(c, s), ctx = max(c.ctx[s], 0);
    const int keys = (int)min((int64_t)ctx, (int64_t)c.W << c.pshift);
    const int lo = a.window ? max(ctx - n - a.window + 1, 0) & ~63 : 0;
    *tiles = max(n * a.G + kRows - 1, 0) / kRows;
    *units = keys > lo ? (keys - lo + a.unit - 1) / a.unit : 1;
    return c.H * *tiles * *units;
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
    for (int s0 = 0; s0 < a.c.S; s0 += 64) {
        count_64(a, s0, &q);
        q.total += __builtin_amdgcn_readlane(q.upto, 63);
    }
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
    const int row_lo = a.window ? pos - a.window + 1 : 0;
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
        const uint32_t ks = c.ks[sb], vs = c.vs[sb];
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
            // V where no row may attend is whatever memory held: made zero, as 0 * NaN is not 0
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
    int at = (int)blockIdx.x * q.share;
    const int stop = min(at + q.share, q.total);
    while (at < stop) {
        const UnitPlace p = find_unit(a, q, at);
        const int u1 = min(p.units, p.u + stop - at);
        const AttnTile t = attn_tile<kRows>(a, p.s, p.tile);
        const int lo = a.window ? max(t.p0 - a.window + 1, 0) & ~63 : 0;  // where the sequence's units begin
        const int begin = max(lo + p.u * a.unit, t.lo & ~63);
        const int end = u1 == p.units ? t.hi : min(t.hi, lo + u1 * a.unit);
        const bool whole = p.u == 0 && u1 == p.units;
        attn_rows<DT, U, FULL, NW>(a, t, p.h, begin, end, whole ? -1 : 2 * (int)blockIdx.x + (p.u == 0));
        at += u1 - p.u;
    }
}

// The partial results of a row's key splits joined: workgroup (r, w) for row r of the tile that share w
// ends in, if it begins there too. Its threads take 4 channels each and the splits in turn (all loads
// of a thread are independent of one another), then join over LDS, always in the same order.
template <int DT>
__global__ __launch_bounds__(256) void k_kv_attn_join(KvAttnArgs a) {
    const KvView& c = a.c;
    const int rr = blockIdx.x, w = blockIdx.y, D = c.D;
    Units q = count_units(a);
    const int cut = (w + 1) * q.share;
    if (cut >= q.total) return;
    const UnitPlace p = find_unit(a, q, cut);
    const int first = cut - p.u;
    if (p.u == 0 || first < w * q.share) return;
    const AttnTile t = attn_tile<kRows>(a, p.s, p.tile);
    if (rr >= t.r1 - t.r0) return;
    const int h = p.h, splits = (first + p.units - 1) / q.share - w + 1;
    // row of split z: place 1 of share w, then place 0 of those after it
    const auto row = [&](int z) { return ((int64_t)(2 * (w + z)) + (z == 0)) * kRows + rr; };
    const int tid = threadIdx.x;
    __shared__ float sf[256];  // each split's factor exp2(m_z - m), 256 splits at a time
    __shared__ float sm[4];
    __shared__ f32x4 so[256];
    float m = kNegInf;
    for (int z = tid; z < splits; z += 256) m = fmaxf(m, a.part_ml[2 * row(z)]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((tid & 63) == 0) sm[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const float ms = m == kNegInf ? 0.0f : m;

    const int per = D >> 2, lanes = 256 / per;  // threads of one split; splits at once
    const int mine = tid / per, d = (tid - mine * per) * 4;
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
    l = (sm[0] + sm[1]) + (sm[2] + sm[3]);
    if (mine != 0) return;
    for (int i = 1; i < lanes; ++i) o += so[i * per + tid];
    const int r = t.r0 + rr, tok = r / a.G, head = h * a.G + r - tok * a.G;
    store_out4<DT>(a.out, (int64_t)(t.tok0 + tok) * a.ldo + (int64_t)head * a.ldo_head + d, o * safe_rcp(l));
    if (a.lse && d == 0) a.lse[(int64_t)(t.tok0 + tok) * a.Hq + head] = lse_of(m, l);
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
    const int G = Hq / c.H;
    // tiles that have rows, and keys that one of them goes through, at most
    int64_t tiles = (int64_t)c.T * G / kRows + c.S;
    if (max_tokens > 0) tiles = std::min(tiles, c.S * (((int64_t)max_tokens * G + kRows - 1) / kRows));
    tiles *= c.H;
    const int64_t room = (int64_t)c.W << c.pshift;
    int64_t keys = room;
    if (max_context > 0) keys = std::min<int64_t>(keys, max_context);
    if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window + std::max(max_tokens, 1) + 64);
    // (the kernels count units in 32 bits, whatever the hints were)
    const int64_t most = ((int64_t)c.T * G / kRows + c.S) * c.H;
    const int64_t unit = 256;
    const int waves = rows_waves(dtype == DT_BF16 ? DT_BF16 : DT_F32, (c.D + 63) / 64);
    if (keys <= 1024 || most * (room / unit + 1) >= (int64_t(1) << 31)) {
        // Short contexts: a workgroup for each tile, of eight waves where registers allow. 600 tokens of 8
        // kv heads: 11.7 us, against 13.5 + 4.2 us for shares and their join.
        p.nw = 4 * waves;
        p.unit = 1 << 30;
        p.share_min = 1;
        p.grid = (int)std::min<int64_t>(std::min(tiles, most), 1 << 30);
    } else {
        // Shares: four waves, so that a CU has a second workgroup to read for while one changes tiles or
        // joins its waves (64 sequences of 4127 tokens on average: 115 us, with one of eight 140 us).
        p.nw = 4;
        p.unit = (int)unit;
        p.share_min = 2;
        p.grid = cu_count() * waves;
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

template <int DT, int U>
static void launch_rows(const KvAttnArgs& a, int nw, hipStream_t s) {
    if constexpr (rows_waves(DT, U) == 2) {
        if (nw == 8) return launch_rows_nw<DT, U, 8>(a, s);
    }
    launch_rows_nw<DT, U, 4>(a, s);
}

template <int DT>
static hipError_t launch_dt(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
    switch ((a.c.D + 63) / 64) {
        case 1: launch_rows<DT, 1>(a, p.nw, s); break;
        case 2: launch_rows<DT, 2>(a, p.nw, s); break;
        case 3: launch_rows<DT, 3>(a, p.nw, s); break;
        default: launch_rows<DT, 4>(a, p.nw, s); break;
    }
    if (p.join_rows)
        hipLaunchKernelGGL((k_kv_attn_join<DT>), dim3((unsigned)p.join_rows, (unsigned)a.grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_attention(KvAttnArgs a, const KvAttnPlan& p, int dtype, void* ws, hipStream_t s) {
    a.grid = p.grid;
    a.unit = p.unit;
    a.share_min = p.share_min;
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = a.part_o + (int64_t)p.grid * 2 * kRows * a.c.D;
    return dtype == DT_BF16 ? launch_dt<DT_BF16>(a, p, s) : launch_dt<DT_F32>(a, p, s);
}

}  // namespace bgf
