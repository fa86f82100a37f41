// Rotary positions: the channels of a head turned in pairs by position * inv_freq[i].
//
// A workgroup takes a few tokens. First it computes their angles' sines and cosines, one (token, pair) a
// thread and for all heads at once, into LDS; then its threads walk over the tokens' heads, a unit of V pairs
// at a time. The angle is fp64 and so is its reduction to a quarter turn (an fp32 product of a position past
// 2^17 is off by 2^-7 radians); sine and cosine of what is left, |r| <= pi / 4, are fp32 Taylor sums.
#include "device.h"
#include "kv_device.h"
#include "layer_internal.h"

namespace bgf {

constexpr int kRopeThreads = 256, kRopePairs = 512, kRopeTokens = 64;

// cos and sin of an angle in radians
__device__ __forceinline__ float2 cos_sin(double t) {
    const double n = rint(t * 0.63661977236758134);  // quarter turns: 2 / pi
    const float r = (float)fma(-n, 1.5707963267948966, t), z = r * r;
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

// V consecutive values, in accesses of 16 bytes or V * size where that is less
template <int DT, int V>
__device__ __forceinline__ void load_values(const void* base, int64_t at, float (&v)[V]) {
    if constexpr (DT == DT_BF16) {
        constexpr int S = V > 8 ? 8 : V;
        typedef uint16_t words __attribute__((ext_vector_type(S)));
        const uint16_t* s = reinterpret_cast<const uint16_t*>(base) + at;
        if constexpr (V == 1) {
            v[0] = __uint_as_float((uint32_t)s[0] << 16);
        } else {
#pragma unroll
            for (int k = 0; k < V; k += S) {
                const words w = *reinterpret_cast<const words*>(s + k);
#pragma unroll
                for (int i = 0; i < S; ++i) v[k + i] = __uint_as_float((uint32_t)w[i] << 16);
            }
        }
    } else {
        constexpr int S = V > 4 ? 4 : V;
        typedef float words __attribute__((ext_vector_type(S)));
        const float* s = reinterpret_cast<const float*>(base) + at;
        if constexpr (V == 1) {
            v[0] = s[0];
        } else {
#pragma unroll
            for (int k = 0; k < V; k += S) {
                const words w = *reinterpret_cast<const words*>(s + k);
#pragma unroll
                for (int i = 0; i < S; ++i) v[k + i] = w[i];
            }
        }
    }
}

template <int DT, int V>
__device__ __forceinline__ void store_values(void* base, int64_t at, const float (&v)[V]) {
    if constexpr (DT == DT_BF16) {
        uint16_t* d = reinterpret_cast<uint16_t*>(base) + at;
        if constexpr (V == 1) {
            d[0] = (uint16_t)pack_bf16x2_rne(v[0], 0.0f);
        } else {
            constexpr int S = V > 8 ? 8 : V;
            typedef uint32_t words __attribute__((ext_vector_type(S / 2)));
#pragma unroll
            for (int k = 0; k < V; k += S) {
                words w;
#pragma unroll
                for (int i = 0; i < S / 2; ++i) w[i] = pack_bf16x2_rne(v[k + 2 * i], v[k + 2 * i + 1]);
                *reinterpret_cast<words*>(d + k) = w;
            }
        }
    } else {
        constexpr int S = V > 4 ? 4 : V;
        typedef float words __attribute__((ext_vector_type(S)));
        float* d = reinterpret_cast<float*>(base) + at;
        if constexpr (V == 1) {
            d[0] = v[0];
        } else {
#pragma unroll
            for (int k = 0; k < V; k += S) {
                words w;
#pragma unroll
                for (int i = 0; i < S; ++i) w[i] = v[k + i];
                *reinterpret_cast<words*>(d + k) = w;
            }
        }
    }
}

// HALF: pairs (i, i + rot / 2), else (2 i, 2 i + 1). A unit is V pairs of one head of one token. Channels
// past rot are copied V at a time (where they are not in place already).
template <int DT, bool HALF, int V>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeArgs a, int per) {
    __shared__ float2 turn[kRopePairs];
    __shared__ int pos[kRopeTokens];
    __shared__ int there[kRopeTokens];
    const int half = a.rot >> 1, heads = a.heads[0] + a.heads[1];
    const int units = half / V, rest = (a.dim - a.rot) / V;
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
        for (int i = threadIdx.x; i < n * heads * units; i += kRopeThreads) {
            const int u = i % units, h = (i / units) % heads, tok = i / units / heads;
            if (!there[tok]) continue;
            const int k = h >= a.heads[0], hk = h - (k ? a.heads[0] : 0);
            const int64_t t = t0 + tok;
            const int64_t xi = t * a.ldx[k] + hk * a.ldx_head[k], oi = t * a.ldo[k] + hk * a.ldo_head[k];
            const float2* cs = turn + tok * half + u * V;
            if constexpr (HALF) {
                float x1[V], x2[V], y1[V], y2[V];
                load_values<DT, V>(a.x[k], xi + u * V, x1);
                load_values<DT, V>(a.x[k], xi + half + u * V, x2);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 c = cs[j];
                    y1[j] = __builtin_fmaf(x1[j], c.x, -(x2[j] * c.y));
                    y2[j] = __builtin_fmaf(x2[j], c.x, x1[j] * c.y);
                }
                store_values<DT, V>(a.out[k], oi + u * V, y1);
                store_values<DT, V>(a.out[k], oi + half + u * V, y2);
            } else {
                float x[2 * V], y[2 * V];
                load_values<DT, 2 * V>(a.x[k], xi + 2 * u * V, x);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 c = cs[j];
                    y[2 * j] = __builtin_fmaf(x[2 * j], c.x, -(x[2 * j + 1] * c.y));
                    y[2 * j + 1] = __builtin_fmaf(x[2 * j + 1], c.x, x[2 * j] * c.y);
                }
                store_values<DT, 2 * V>(a.out[k], oi + 2 * u * V, y);
            }
        }
        for (int i = threadIdx.x; i < n * heads * rest; i += kRopeThreads) {
            const int u = i % rest, h = (i / rest) % heads, tok = i / rest / heads;
            const int k = h >= a.heads[0], hk = h - (k ? a.heads[0] : 0);
            if (!there[tok] || a.out[k] == a.x[k]) continue;
            const int64_t t = t0 + tok;
            float x[V];
            load_values<DT, V>(a.x[k], t * a.ldx[k] + hk * a.ldx_head[k] + a.rot + u * V, x);
            store_values<DT, V>(a.out[k], t * a.ldo[k] + hk * a.ldo_head[k] + a.rot + u * V, x);
        }
    }
}

template <int DT, bool HALF>
static hipError_t launch_rope_k(const RopeArgs& a, hipStream_t s) {
    const int half = a.rot / 2;
    int per = kRopePairs / half;
    if (per > 4) per = 4;
    const int64_t need = (a.tokens + per - 1) / per;
    const unsigned grid = (unsigned)(need < kMaxGrid ? need : kMaxGrid);
    // pairs of a unit: as many as fill 16-byte accesses and divide both parts of a head (their places then are
    // multiples of the access too)
    if (half % 8 == 0 && (a.dim - a.rot) % 8 == 0) hipLaunchKernelGGL((k_rope<DT, HALF, 8>), dim3(grid), dim3(kRopeThreads), 0, s, a, per);
    else hipLaunchKernelGGL((k_rope<DT, HALF, 1>), dim3(grid), dim3(kRopeThreads), 0, s, a, per);
    return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, int dtype, int layout, hipStream_t s) {
    if (dtype == DT_BF16) return layout ? launch_rope_k<DT_BF16, false>(a, s) : launch_rope_k<DT_BF16, true>(a, s);
    return layout ? launch_rope_k<DT_F32, false>(a, s) : launch_rope_k<DT_F32, true>(a, s);
}

}  // namespace bgf
