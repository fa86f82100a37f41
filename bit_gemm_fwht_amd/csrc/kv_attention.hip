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
template <int NS>
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
                const uint32_t a = __float_as_uint(y[2 * i]) & 0xFFFF0000u, b = __float_as_uint(y[2 * i + 1]) & 0xFFFF0000u;
                r[n][i] = (a >> 16) | b;
                // an infinity has no rest (inf - inf would be NaN)
                y[2 * i] = (a & 0x7F800000u) == 0x7F800000u ? 0.0f : y[2 * i] - __uint_as_float(a);
                y[2 * i + 1] = (b & 0x7F800000u) == 0x7F800000u ? 0.0f : y[2 * i + 1] - __uint_as_float(b);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) out[n] = __builtin_bit_cast(bf16x8, r[n]);
}

// One tile of TR query rows (a row = a token and one of the G query heads of a kv head, token major)
// and the keys that any of them may attend.
struct AttnTile {
    int s;            // sequence, -1: no such tile
    int tok0;         // first row of the sequence in the batch
    int r0, r1;       // its rows [r0, r1) of n * G
    int p0;           // position of the sequence's first row
    int keys;         // keys that exist: min(context, table)
    int lo, hi;       // keys that some row may attend
    int flo, fhi;     // keys that every row may attend
    int splits;       // key splits of this tile
};

template <int TR>
__device__ __forceinline__ AttnTile attn_tile(const KvAttnArgs& a, int slot) {
    const KvView& c = a.c;
    AttnTile t;
    int first;
    t.s = find_sequence(c, slot, a.G, TR, 1, &first);
    if (t.s < 0) return t;
    t.tok0 = cu_at(c, t.s);
    const int n = cu_at(c, t.s + 1) - t.tok0;
    t.r0 = (slot - first) * TR;
    t.r1 = min(t.r0 + TR, n * a.G);
    if (t.r0 >= t.r1) {
        t.s = -1;
        return t;
    }
    const int ctx = max(c.ctx[t.s], 0);
    t.keys = (int)min((int64_t)ctx, (int64_t)c.W << c.pshift);
    t.p0 = ctx - n;
    const int pa = t.p0 + t.r0 / a.G, pb = t.p0 + (t.r1 - 1) / a.G;  // positions of the first and last row
    t.hi = a.causal ? max(min(t.keys, pb + 1), 0) : t.keys;
    t.fhi = a.causal ? min(t.keys, pa + 1) : t.keys;
    t.lo = a.window ? max(pa - a.window + 1, 0) : 0;
    t.flo = a.window ? pb - a.window + 1 : 0;
    const int len = t.hi - (t.lo & ~63);
    t.splits = max(1, min(a.Z, (int)(((int64_t)len + a.chunk - 1) / a.chunk)));
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
// Few rows: tiles of 16, the keys dealt to four waves in steps of 64 each, straight from memory to
// registers (no two waves read the same key).
// ---------------------------------------------------------------------------------------------
constexpr int kRows = 16;

// Waves a SIMD holds at once: as many as the registers of the variant allow without spills (a lane
// holds 16 U of K and V each on their way, 16 U of o, 8 U (fp32: 24 U) of q).
constexpr int rows_waves(int dt, int u) {
    return dt == DT_BF16 ? (u == 1 ? 4 : u == 2 ? 3 : u == 3 ? 2 : 1) : (u == 1 ? 3 : u == 2 ? 2 : 1);
}

template <int DT, int U, bool FULL>  // U: 64-channel pieces of a head; FULL: the head fills them
__global__ __launch_bounds__(256, rows_waves(DT, U)) void k_kv_attn_rows(KvAttnArgs a) {
    constexpr int NS = DT == DT_BF16 ? 1 : 3, NP = DT == DT_BF16 ? 2 : 3;  // bf16 a query and a weight take
    const KvView& c = a.c;
    const int h = blockIdx.y, z = blockIdx.z;
    const AttnTile t = attn_tile<kRows>(a, blockIdx.x);
    if (t.s < 0 || z >= t.splits) return;
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
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                bf16x8 f[NS];
                split8<NS>(x + 8 * w, f);
#pragma unroll
                for (int n = 0; n < NS; ++n) qf[n][2 * u + w] = f[n];
            }
        }
    }

    f32x4 o[4 * U];
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) o[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    float m = kNegInf, l = 0.0f;

    const int begin = (t.lo & ~63) + z * a.chunk;
    const int end = z == t.splits - 1 ? t.hi : min(t.hi, begin + a.chunk);
    const int gk = li >> 2;  // S^T row li of piece e is key 16 gk + 4 e + (li & 3) of the step
    // pages of the 16 keys this lane loads K for, and of the 16 it loads V for; the next step's are
    // looked up while this step's K and V are on their way
    const auto page_of = [&](int key) { return key < t.hi ? page_at(c, t.s, key >> c.pshift) : -1; };
    int kb = begin + 64 * wave;
    int pk_next = page_of(kb + 16 * gk), pv_next = page_of(kb + 16 * g);
#pragma unroll 1
    for (; kb < end; kb += 256) {
        const int tk = kb + 16 * gk, tv = kb + 16 * g;
        const int pk = pk_next, pv = pv_next;
        pk_next = page_of(tk + 256);
        pv_next = page_of(tv + 256);
        u32x4 kraw[4][U], vraw[4 * U];
        const uint8_t* kp = c.kc + ((((int64_t)max(pk, 0) * c.H + h) << c.pshift) + (tk & (P - 1)) + (li & 3)) * D + 16 * g;
        const uint8_t* vp = c.vc + (((int64_t)max(pv, 0) * c.H + h) * D + li) * P + (tv & (P - 1));
        // (loads are not conditional: a lane with nothing to load reads page 0 and is masked below, a
        // piece past the head's channels is read from its start and not used)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = FULL || 64 * u + 16 * g < D;
                const u32x4 w = *reinterpret_cast<const u32x4*>(kp + 4 * e * D + (in ? 64 * u : -16 * g));
                kraw[e][u] = in ? w : (u32x4){0, 0, 0, 0};
            }
#pragma unroll
        for (int i = 0; i < 4 * U; ++i) vraw[i] = *reinterpret_cast<const u32x4*>(vp + (FULL || 16 * i < D ? 16 * i * P : 0));
        const int64_t sb = (int64_t)max(pv, 0) * c.H + h;
        const float kscale = fminf(e8m0_value(c.ks[sb]) * a.scale_log2, 3.40282347e38f);
        const float vscale = e8m0_value(c.vs[sb]);

        // scores of this lane's row and keys kb + 16 g + 0 .. 15, in log2 units
        float s[16];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f32x4 acc = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const bf16x8 kf = cvt8(kraw[e][u][2 * w], kraw[e][u][2 * w + 1], 1.0f);
#pragma unroll
                    for (int n = 0; n < NS; ++n) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[n][2 * u + w], acc, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * e + i] = acc[i] * kscale;
        }

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
        float mx = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, mx);
        const float ms = mn == kNegInf ? 0.0f : mn;  // a row with no key so far: exp2(-inf) = 0 below
        if (__ballot(mn > m)) {
            const float f = __builtin_amdgcn_exp2f(m - ms);
            l *= f;
#pragma unroll
            for (int i = 0; i < 4 * U; ++i) o[i] *= f;
            m = mn;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = __builtin_amdgcn_exp2f(s[i] - ms);
            l += s[i];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            bf16x8 pf[NP];
            split8<NP>(s + 8 * w, pf);
#pragma unroll
            for (int i = 0; i < 4 * U; ++i) {
                const bf16x8 vf = cvt8(vraw[i][2 * w], vraw[i][2 * w + 1], vscale);
#pragma unroll
                for (int n = 0; n < NP; ++n) o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[n], o[i], 0, 0, 0);
            }
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the four waves' keys: 2 and 3 into 0 and 1, then 1 into 0
    __shared__ float sm[2][64], sl[2][64];
    __shared__ f32x4 so[2][4 * U][64];
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
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
    if (t.splits == 1) {
        const float inv = safe_rcp(l);
        const int64_t o0 = (int64_t)(t.tok0 + tok) * a.ldo + (int64_t)head * a.ldo_head + 4 * g;
#pragma unroll
        for (int i = 0; i < 4 * U; ++i)
            if (16 * i < D) store_out4<DT>(a.out, o0 + 16 * i, o[i] * inv);
        if (a.lse && g == 0) a.lse[(int64_t)(t.tok0 + tok) * a.Hq + head] = lse_of(m, l);
    } else {
        const int64_t row = (((int64_t)z * c.H + h) * a.slots + blockIdx.x) * kRows + li;
#pragma unroll
        for (int i = 0; i < 4 * U; ++i)
            if (16 * i < D) *reinterpret_cast<f32x4*>(a.part_o + row * D + 16 * i + 4 * g) = o[i];
        if (g == 0) {
            a.part_ml[2 * row] = m;
            a.part_ml[2 * row + 1] = l;
        }
    }
}

// The partial results of a tile's key splits joined, in the splits' order: one workgroup for each
// (tile, kv head), a thread for 4 channels of a row.
template <int DT, int TR>
__global__ __launch_bounds__(256) void k_kv_attn_join(KvAttnArgs a) {
    const KvView& c = a.c;
    const int h = blockIdx.y, D = c.D;
    const AttnTile t = attn_tile<TR>(a, blockIdx.x);
    if (t.s < 0 || t.splits == 1) return;
    const int per = D >> 2;
    const int64_t step = (int64_t)c.H * a.slots * TR, base = ((int64_t)h * a.slots + blockIdx.x) * TR;
    for (int i = threadIdx.x; i < (t.r1 - t.r0) * per; i += 256) {
        const int rr = i / per, d = (i - rr * per) * 4;
        float m = kNegInf;
        for (int z = 0; z < t.splits; ++z) m = fmaxf(m, a.part_ml[2 * (z * step + base + rr)]);
        const float ms = m == kNegInf ? 0.0f : m;
        float l = 0.0f;
        f32x4 o = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        for (int z = 0; z < t.splits; ++z) {
            const int64_t row = z * step + base + rr;
            const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * row] - ms);
            l += a.part_ml[2 * row + 1] * f;
            o += *reinterpret_cast<const f32x4*>(a.part_o + row * D + d) * f;
        }
        const int r = t.r0 + rr, tok = r / a.G, head = h * a.G + r - tok * a.G;
        store_out4<DT>(a.out, (int64_t)(t.tok0 + tok) * a.ldo + (int64_t)head * a.ldo_head + d, o * safe_rcp(l));
        if (a.lse && d == 0) a.lse[(int64_t)(t.tok0 + tok) * a.Hq + head] = lse_of(m, l);
    }
}

KvAttnPlan plan_kv_attention(const KvView& c, int Hq, int window, int dtype, int max_tokens, int max_context) {
    KvAttnPlan p{};
    const int G = Hq / c.H;
    p.rows = kRows;
    p.slots = (unsigned)((int64_t)c.T * G / p.rows + c.S);
    // keys that one tile may have to go through
    int64_t keys = (int64_t)c.W << c.pshift;
    if (max_context > 0 && max_context < keys) keys = max_context;
    if (window > 0) {
        const int64_t w = (int64_t)window + p.rows / G + 64;
        if (w < keys) keys = w;
    }
    // enough workgroups for two on every CU, at least one 64-key step for each of the four waves
    const int64_t tiles = (int64_t)p.slots * c.H;
    int64_t z = (512 + tiles - 1) / tiles;
    const int64_t most = (keys + 255) / 256;
    if (z > most) z = most;
    if (z < 1) z = 1;
    int64_t chunk = (keys + z - 1) / z;
    chunk = (chunk + 255) / 256 * 256;
    z = (keys + chunk - 1) / chunk;
    p.Z = (int)(z < 1 ? 1 : z);
    p.chunk = (int)chunk;
    p.ws = p.Z == 1 ? 0 : (int64_t)p.Z * c.H * p.slots * p.rows * (c.D + 2) * 4;
    return p;
}

template <int DT, int U>
static void launch_rows(const KvAttnArgs& a, hipStream_t s) {
    const dim3 grid(a.slots, (unsigned)a.c.H, (unsigned)a.Z);
    if (a.c.D == 64 * U) hipLaunchKernelGGL((k_kv_attn_rows<DT, U, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_kv_attn_rows<DT, U, false>), grid, dim3(256), 0, s, a);
}

template <int DT>
static hipError_t launch_dt(const KvAttnArgs& a, hipStream_t s) {
    switch ((a.c.D + 63) / 64) {
        case 1: launch_rows<DT, 1>(a, s); break;
        case 2: launch_rows<DT, 2>(a, s); break;
        case 3: launch_rows<DT, 3>(a, s); break;
        default: launch_rows<DT, 4>(a, s); break;
    }
    if (a.Z > 1) hipLaunchKernelGGL((k_kv_attn_join<DT, kRows>), dim3(a.slots, (unsigned)a.c.H), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_attention(KvAttnArgs a, const KvAttnPlan& p, int dtype, void* ws, hipStream_t s) {
    a.slots = p.slots;
    a.Z = p.Z;
    a.chunk = p.chunk;
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = a.part_o + (int64_t)p.Z * a.c.H * p.slots * p.rows * a.c.D;
    return dtype == DT_BF16 ? launch_dt<DT_BF16>(a, s) : launch_dt<DT_F32>(a, s);
}

}  // namespace bgf
