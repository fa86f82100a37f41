// Rotary positions: the channels of a head turned in pairs by position * inv_freq[i].
//
// A workgroup takes a few tokens. First it computes their angles' sines and cosines, one (token, pair) a
// thread and for all heads at once, into LDS; then its threads walk over the tokens' heads in units of 16 bytes
// (half layout: 16 and their partners). The angle is fp64 and so is its reduction to a quarter turn (an fp32 product of a position past
// 2^17 is off by 2^-7 radians); sine and cosine of what is left, |r| <= pi / 4, are fp32 Taylor sums.
#include "device.h"
#include "kv_device.h"
#include "layer_internal.h"

namespace bgf {

constexpr int kRopeThreads = 256, kRopePairs = 512, kRopeTokens = 64, kRopeGroups = 512;

// cos and sin of an angle in radians, |t| < 2^45. pi / 2 as one fp64 is 6e-17 off, which n quarter turns add up: 8e-8
// at position 2^31 for a frequency of 1, past 2^-22 for one above 3 (a table may hold any), so its rest comes along.
__device__ __forceinline__ float2 cos_sin(double t) {
    const double n = rint(t * 0.63661977236758134);  // quarter turns: 2 / pi
    const float r = (float)fma(-n, 6.123233995736766e-17, fma(-n, 1.5707963267948966, t)), z = r * r;
    // sin r = r - r^3/3! + .. - r^11/11!, cos r = 1 - r^2/2! + .. - r^10/10!: the next terms are below 2^-32
    float s = __builtin_fmaf(z, -2.50521083854e-8f, 2.75573192240e-6f);
    s = __builtin_fmaf(z, s, -1.98412698413e-4f);
    s = __builtin_fmaf(z, s, 8.33333333333e-3f);
    s = __builtin_fmaf(z, s, -1.66666666667e-1f);
    s = __builtin_fmaf(r * z, s, r);
    float c = __builtin_fmaf(z, -2.75573192240e-7f, 2.48015873016e-5f);
    c = __builtin_fmaf(z, c, -1.38888888889e-3f);
    c = __builtin_fmaf(z, c, 4.16666666667e-2f);
    c = __builtin_fmaf(z, c, -0.5f);
    c = __builtin_fmaf(z, c, 1.0f);
    const int q = (int)(long long)n & 3;
    const float cs = (q & 1) ? s : c, sn = (q & 1) ? c : s;
    return make_float2(q == 1 || q == 2 ? -cs : cs, q >= 2 ? -sn : sn);
}

// V consecutive values in one access of V * size bytes
template <int DT, int V>
struct Words {
    typedef uint32_t type __attribute__((ext_vector_type(DT == DT_BF16 ? V / 2 : V)));
};
template <int DT, int V, bool NT>
__device__ __forceinline__ void load_values(const void* base, int64_t at, float (&v)[V]) {
    if constexpr (DT == DT_BF16 && V == 1) {
        v[0] = __uint_as_float((uint32_t)(reinterpret_cast<const uint16_t*>(base)[at]) << 16);
    } else if constexpr (V == (DT == DT_BF16 ? 2 : 1)) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(base) + at * (DT == DT_BF16 ? 2 : 4));
        if constexpr (DT == DT_BF16) v[0] = bf16_lo(w), v[1] = bf16_hi(w);
        else v[0] = __uint_as_float(w);
    } else {
        typedef typename Words<DT, V>::type words;
        const words* s = reinterpret_cast<const words*>(reinterpret_cast<const char*>(base) + at * (DT == DT_BF16 ? 2 : 4));
        const words w = NT ? __builtin_nontemporal_load(s) : *s;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (DT == DT_BF16) v[i] = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
            else v[i] = __uint_as_float(w[i]);
        }
    }
}

template <int DT, int V, bool NT>
__device__ __forceinline__ void store_values(void* base, int64_t at, const float (&v)[V]) {
    if constexpr (DT == DT_BF16 && V == 1) {
        reinterpret_cast<uint16_t*>(base)[at] = (uint16_t)pack_bf16x2_rne(v[0], 0.0f);
    } else if constexpr (V == (DT == DT_BF16 ? 2 : 1)) {
        uint32_t* d = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(base) + at * (DT == DT_BF16 ? 2 : 4));
        if constexpr (DT == DT_BF16) *d = pack_bf16x2_rne(v[0], v[1]);
        else *d = __float_as_uint(v[0]);
    } else {
        typedef typename Words<DT, V>::type words;
        words* d = reinterpret_cast<words*>(reinterpret_cast<char*>(base) + at * (DT == DT_BF16 ? 2 : 4));
        words w;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            if constexpr (DT == DT_BF16) w[i >> 1] = pack_bf16x2_rne(v[i], v[i + 1]);
            else w[i] = __float_as_uint(v[i]), w[i + 1] = __float_as_uint(v[i + 1]);
        }
        if constexpr (NT) __builtin_nontemporal_store(w, d);
        else *d = w;
    }
}

// HALF: pairs (i, i + rot / 2), a unit is V channels and their V partners; else (2 i, 2 i + 1), a unit is V channels
// (V even). Units past the turned ones copy V channels (where they are not in place already).
template <int DT, bool HALF, int V, bool NT>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeArgs a, int per, int hper) {
    __shared__ float2 turn[kRopePairs];
    __shared__ int pos[kRopeTokens];
    __shared__ int there[kRopeTokens];
    const int half = a.rot >> 1, h0 = blockIdx.y * hper, heads = min(hper, a.heads[0] + a.heads[1] - h0);
    const int turned = (HALF ? half : a.rot) / V, units = turned + (a.dim - a.rot) / V;
    // a thread's unit, head and token; kRopeThreads units further on it is (step_u, step_h, step_t) more
    const int u0 = threadIdx.x % units, r0 = threadIdx.x / units;
    const int step_u = kRopeThreads % units, step_r = kRopeThreads / units, step_h = step_r % heads, step_t = step_r / heads;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.tokens; t0 += (int64_t)gridDim.x * per) {
        const int n = (int)min((int64_t)per, a.tokens - t0);
        __syncthreads();  // the last tokens' values have been read
        if (a.pos) {
            if ((int)threadIdx.x < n) {
                pos[threadIdx.x] = a.pos[t0 + threadIdx.x];
                there[threadIdx.x] = 1;
            }
        } else {
            for (int i = threadIdx.x >> 6; i < n; i += kRopeThreads / 64) {  // a wave a token
                const int t = (int)(t0 + i);
                int first;
                const int s = find_sequence(a.batch, t, 1, 1, 0, &first);
                int64_t p = -1;
                if (s >= 0) {
                    const int end = cu_at(a.batch, s + 1);
                    if (t < end) p = (int64_t)a.batch.ctx[s] - end + t;
                }
                if ((threadIdx.x & 63) == 0) {
                    pos[i] = (int)p;
                    there[i] = p >= 0;
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
            float2 cs = cos_sin((double)pos[i / half] * a.inv_freq[i % half]);
            cs.x *= a.scale;
            cs.y *= a.backward ? -a.scale : a.scale;
            turn[i] = cs;
        }
        __syncthreads();
        int u = u0, h = r0 % heads, tok = r0 / heads;
        while (tok < n) {
            const int k = h0 + h >= a.heads[0], hk = h0 + h - (k ? a.heads[0] : 0);
            const int64_t t = t0 + tok;
            const int64_t xi = t * a.ldx[k] + hk * a.ldx_head[k], oi = t * a.ldo[k] + hk * a.ldo_head[k];
            // lanes that turn and lanes that copy load and store together
            const bool turns = u < turned, same = a.out[k] == a.x[k];
            if (there[tok] && (turns || !same)) {
                const int c = HALF && !turns ? a.rot + (u - turned) * V : u * V;
                float x[V], y[V];
                load_values<DT, V, NT>(a.x[k], xi + c, x);
                if constexpr (HALF) {
                    float z[V] = {};
                    if (turns) load_values<DT, V, NT>(a.x[k], xi + half + c, z);
                    const float2* cs = turn + (turns ? tok * half + c : 0);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float2 s = cs[turns ? j : 0];
                        y[j] = turns ? __builtin_fmaf(x[j], s.x, -(z[j] * s.y)) : x[j];
                        z[j] = __builtin_fmaf(z[j], s.x, x[j] * s.y);
                    }
                    store_values<DT, V, NT>(a.out[k], oi + c, y);
                    if (turns) store_values<DT, V, NT>(a.out[k], oi + half + c, z);
                } else {
                    const float2* cs = turn + (turns ? tok * half + c / 2 : 0);
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float2 s = cs[turns ? j / 2 : 0];
                        y[j] = turns ? __builtin_fmaf(x[j], s.x, -(x[j + 1] * s.y)) : x[j];
                        y[j + 1] = turns ? __builtin_fmaf(x[j + 1], s.x, x[j] * s.y) : x[j + 1];
                    }
                    store_values<DT, V, NT>(a.out[k], oi + c, y);
                }
            }
            u += step_u;
            h += step_h;
            tok += step_t;
            if (u >= units) {
                u -= units;
                ++h;
            }
            if (h >= heads) {  // h < 2 heads: one step is enough
                h -= heads;
                ++tok;
            }
        }
    }
}

template <int DT, bool HALF, bool NT>
static hipError_t launch_rope_k(const RopeArgs& a, hipStream_t s) {
    const int half = a.rot / 2;
    // a unit: 16 bytes, or as many as divide both parts of a head (whose places are then multiples of it too)
    constexpr int most = DT == DT_BF16 ? 8 : 4;
    int v = most;
    while ((HALF ? half : a.rot) % v || (a.dim - a.rot) % v) v /= 2;
    // Up to four tokens a workgroup. Where that leaves it few workgroups, fewer tokens, then a part of the heads, while
    // each thread has a unit (the angles are computed again for each part; 40 heads of 128: 64 tokens 4.3 us against
    // 6.2, 600 tokens 6.0 and 7.7)
    int per = kRopePairs / half;
    if (per > 4) per = 4;
    while (per > 1 && a.tokens < kRopeGroups * (int64_t)per) per /= 2;
    const int heads = a.heads[0] + a.heads[1], units = ((HALF ? half : a.rot) + a.dim - a.rot) / v;
    const int64_t need = (a.tokens + per - 1) / per;
    int parts = 1;
    while (need * parts < kRopeGroups && per * (heads / (2 * parts)) * units >= kRopeThreads) parts *= 2;
    const int hper = (heads + parts - 1) / parts;
    const dim3 grid((unsigned)(need < kMaxGrid ? need : kMaxGrid), (unsigned)((heads + hper - 1) / hper)), block(kRopeThreads);
    if (v == most) hipLaunchKernelGGL((k_rope<DT, HALF, most, NT>), grid, block, 0, s, a, per, hper);
    else if (v == most / 2) hipLaunchKernelGGL((k_rope<DT, HALF, most / 2, NT>), grid, block, 0, s, a, per, hper);
    else if constexpr (DT == DT_BF16) {
        if (v == 2) hipLaunchKernelGGL((k_rope<DT, HALF, 2, NT>), grid, block, 0, s, a, per, hper);
        else if constexpr (HALF) hipLaunchKernelGGL((k_rope<DT, HALF, 1, NT>), grid, block, 0, s, a, per, hper);
    } else if constexpr (HALF) {
        hipLaunchKernelGGL((k_rope<DT, HALF, 1, NT>), grid, block, 0, s, a, per, hper);
    }
    return hipGetLastError();
}

template <int DT, bool HALF>
static hipError_t launch_rope_h(const RopeArgs& a, hipStream_t s) {
    // past the caches where the call is larger than what they keep and a unit's runs are whole cache lines, which
    // partly written ones would not be twice (16384 tokens of 40 heads of 128: half layout 61.2 us against 67.3,
    // interleaved 62.8 against 69.7; heads of 80, half layout: 61.3 against 48.7, interleaved 42.1 against 47.8)
    const int64_t bytes = a.tokens * (a.heads[0] + a.heads[1]) * a.dim * (DT == DT_BF16 ? 2 : 4);
    const bool lines = !HALF || (a.rot / 2) * (DT == DT_BF16 ? 2 : 4) % 128 == 0;
    return bytes >= (int64_t(64) << 20) && lines ? launch_rope_k<DT, HALF, true>(a, s) : launch_rope_k<DT, HALF, false>(a, s);
}

hipError_t launch_rope(const RopeArgs& a, int dtype, int layout, hipStream_t s) {
    if (dtype == DT_BF16) return layout ? launch_rope_h<DT_BF16, false>(a, s) : launch_rope_h<DT_BF16, true>(a, s);
    return layout ? launch_rope_h<DT_F32, false>(a, s) : launch_rope_h<DT_F32, true>(a, s);
}

}  // namespace bgf
