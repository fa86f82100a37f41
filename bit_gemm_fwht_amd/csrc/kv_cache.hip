// The key / value cache: rows of K and V quantized into their pages as they are written, and read
// back. One wave works for one block (page x kv head) of K or of V; grid: pages that the batch may
// touch (kMaxGrid at a time), kv heads by four, K and V (and again for the next kMaxGrid pages).
//
// A lane takes 4 channels of 16 tokens at a time: the rows' side is then read and written in pieces of 4
// values a token next to one another across the lanes, K's pages in 4 bytes a token likewise, and V's
// pages, where a channel's tokens lie together, in 16 bytes a channel after a transposition in registers.
// Nothing goes through LDS and no wave waits for another. Bound by memory: two prompts of 4096 tokens and
// 32 heads (201 MB) are written in 48.7 us, 4.1 TB/s, 8 contexts (108 MB) read in 22.6 us, 4.8 TB/s, where
// a large copy reaches 5.2; single tokens by the loads that hang on one another (sequence, page, row).
#include <algorithm>

#include "fp4_internal.h"
#include "kv_device.h"

namespace bgf {

constexpr int kKvThreads = 256;

// Which tokens of the batch a workgroup's block holds.
struct KvBlock {
    int page;      // -1: nothing to do
    int t0, t1;    // places of the page that the batch's rows take
    int row0;      // row of place t0
    bool begun;    // the page also holds older tokens (places before t0)
};

__device__ __forceinline__ KvBlock kv_block(const KvView& c, int slot) {
    KvBlock b;
    b.page = -1;
    int first;
    const int s = find_sequence(c, slot, 1, c.P, 2, &first);
    if (s < 0) return b;
    const int r0 = cu_at(c, s), n = cu_at(c, s + 1) - r0;
    if (n <= 0) return b;
    const int ctx = c.ctx[s];
    if (ctx <= 0) return b;
    const int64_t p0 = (int64_t)ctx - n;  // the first row's token; rows before token 0 have none
    const int64_t a0 = p0 > 0 ? p0 : 0;
    const int64_t j = (a0 >> c.pshift) + (slot - first);
    const int64_t lo = j << c.pshift;
    if (lo >= ctx || j >= c.W) return b;
    b.t0 = (int)max(a0 - lo, (int64_t)0);
    b.t1 = (int)min((int64_t)ctx - lo, (int64_t)c.P);
    b.row0 = (int)(r0 + (lo + b.t0 - p0));
    b.begun = b.t0 > 0 && p0 > 0;
    b.page = page_at(c, s, (int)j);
    return b;
}

// 4 values of a row, as they are in memory
template <int DT>
struct Row4 {
    static constexpr int N = DT == DT_BF16 ? 2 : 4;
    uint32_t w[N];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (DT == DT_BF16) {
            const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
            w[0] = v.x, w[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + at);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        if constexpr (DT == DT_BF16) {
            v[0] = bf16_lo(w[0]), v[1] = bf16_hi(w[0]), v[2] = bf16_lo(w[1]), v[3] = bf16_hi(w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
        }
    }
};

// four E4M3 codes under a smaller scale: c * f, f = 2^(old - e) <= 1/2, nearest even
__device__ __forceinline__ uint32_t requant4(uint32_t w, float f) {
    const v2f a = fp8x2_to_f32<false>(w), b = fp8x2_to_f32<true>(w);
    uint32_t r = cvt_fp8x2<false>(0u, a[0] * f, a[1] * f, 1.0f);
    return cvt_fp8x2<true>(r, b[0] * f, b[1] * f, 1.0f);
}

// a 4 x 4 byte block transposed: byte j of word i becomes byte i of word j
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    w[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    w[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    w[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
    w[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

template <int DT>
__global__ __launch_bounds__(kKvThreads) void k_kv_append(KvRowsArgs a) {
    const KvView& c = a.c;
    const int lane = threadIdx.x & 63;
    const int h = blockIdx.y * (kKvThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (h >= c.H) return;
    const bool is_v = blockIdx.z & 1;
    const KvBlock b = kv_block(c, (int)(blockIdx.x + (blockIdx.z >> 1) * gridDim.x));
    if (b.page < 0) return;
    const int D = c.D, P = c.P, quads = D >> 2;
    const int64_t blk = (int64_t)b.page * c.H + h;
    uint8_t* codes = (is_v ? c.vc : c.kc) + blk * P * D;
    uint8_t* scales = (is_v ? c.vs : c.ks) + blk;
    const void* x = is_v ? a.v : a.k;
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const int64_t x0 = (int64_t)b.row0 * ld + h * (is_v ? a.ldv_head : a.ldk_head);
    // tasks: a lane's 4 channels of 16 tokens; those that hold new tokens
    const int g0 = b.t0 >> 4, tasks = (((b.t1 + 15) >> 4) - g0) * quads;
    const bool held = tasks <= 64;  // one for a lane: read once

    const int old = (int)*scales - 127;
    Row4<DT> r[16];
    const auto load = [&](int i) {
        const int g = g0 + i / quads, d = (i % quads) * 4;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const int at = 16 * g + t;
            if (at >= b.t0 && at < b.t1) r[t].load(x, x0 + (int64_t)(at - b.t0) * ld + d);
            else r[t].zero();
        }
    };
    // amax of the new tokens (as integers: |x| orders like its bits)
    uint32_t m = 0;
    for (int i = lane; i < tasks; i += 64) {
        load(i);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float v[4];
            r[t].get(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    int e = e8m0_exp<8, 0x600000u>(__uint_as_float(m), a.ceil_rule != 0);
    if (b.begun) e = max(e, old);
    const bool grown = b.begun && e > old;  // the older tokens get the block's new scale
    const float f = __builtin_amdgcn_ldexpf(1.0f, grown ? old - e : 0);
    if (lane == 0) *scales = (uint8_t)(e + 127);

    // the new tokens: x * 2^-e by the scaled convert, which divides by 2^e exactly; 2^-127 is not a
    // normal fp32, so that exponent is reached by doubling x
    const float dbl = e == -127 ? 2.0f : 1.0f;
    const float sc = pow2f(max(e, -126));
    const float lim = fminf(448.0f * sc, 3.40282347e38f);
    for (int i = lane; i < tasks; i += 64) {
        if (!held) load(i);
        const int g = g0 + i / quads, d = (i % quads) * 4;
        uint32_t w[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float v[4];
            r[t].get(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __builtin_amdgcn_fmed3f(v[j] * dbl, -lim, lim);
            w[t] = cvt_fp8x2<false>(0u, v[0], v[1], sc);
            w[t] = cvt_fp8x2<true>(w[t], v[2], v[3], sc);
        }
        const int lo = b.t0 - 16 * g, hi = b.t1 - 16 * g;  // new places of these 16: [lo, hi)
        if (!is_v) {
#pragma unroll
            for (int t = 0; t < 16; ++t)
                if (t >= lo && t < hi) *reinterpret_cast<uint32_t*>(codes + (16 * g + t) * D + d) = w[t];
            continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t s4[4] = {w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
            transpose4(s4);  // s4[j]: channel d + j of tokens 4 q .. 4 q + 3
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * q + j] = s4[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4* p = reinterpret_cast<uint4*>(codes + (d + j) * P + 16 * g);
            uint32_t n[4] = {w[j], w[4 + j], w[8 + j], w[12 + j]};
            if (lo > 0 || hi < 16) {  // places before lo: older tokens; from hi on: left as they are
                const uint4 v = *p;
                const uint32_t was[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int nl = min(max(lo - 4 * q, 0), 4), nh = min(max(hi - 4 * q, 0), 4);
                    const uint32_t before = nl == 4 ? 0xFFFFFFFFu : (1u << (8 * nl)) - 1u;
                    const uint32_t upto = nh == 4 ? 0xFFFFFFFFu : (1u << (8 * nh)) - 1u;
                    const uint32_t older = grown ? requant4(was[q], f) : was[q];
                    n[q] = (older & before) | (n[q] & upto & ~before) | (was[q] & ~(upto | before));
                }
            }
            *p = make_uint4(n[0], n[1], n[2], n[3]);
        }
    }
    if (!grown) return;
    // older tokens elsewhere in the block: K's rows, V's groups of 16 without a new token
    const int pieces = is_v ? D * g0 : b.t0 * (D >> 4);
    for (int i = lane; i < pieces; i += 64) {
        uint4* p = reinterpret_cast<uint4*>(is_v ? codes + (i / g0) * P + 16 * (i % g0) : codes + 16 * i);
        const uint4 w = *p;
        *p = make_uint4(requant4(w.x, f), requant4(w.y, f), requant4(w.z, f), requant4(w.w, f));
    }
}

// y = code * 2^e for four codes
__device__ __forceinline__ void decode4(uint32_t w, int e, float (&y)[4]) {
    const v2f a = fp8x2_to_f32<false>(w), b = fp8x2_to_f32<true>(w);
    y[0] = __builtin_amdgcn_ldexpf(a[0], e);
    y[1] = __builtin_amdgcn_ldexpf(a[1], e);
    y[2] = __builtin_amdgcn_ldexpf(b[0], e);
    y[3] = __builtin_amdgcn_ldexpf(b[1], e);
}

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t at, const float (&y)[4]) {
    if constexpr (DT == DT_BF16) {
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + at) =
            make_uint2(pack_bf16x2_rne(y[0], y[1]), pack_bf16x2_rne(y[2], y[3]));
    } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at) = make_float4(y[0], y[1], y[2], y[3]);
    }
}

template <int DT>
__global__ __launch_bounds__(kKvThreads) void k_kv_read(KvRowsArgs a) {
    const KvView& c = a.c;
    const int lane = threadIdx.x & 63;
    const int h = blockIdx.y * (kKvThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (h >= c.H) return;
    const bool is_v = blockIdx.z & 1;
    const KvBlock b = kv_block(c, (int)(blockIdx.x + (blockIdx.z >> 1) * gridDim.x));
    if (b.page < 0) return;
    const int D = c.D, P = c.P, quads = D >> 2;
    const int64_t blk = (int64_t)b.page * c.H + h;
    const uint8_t* codes = (is_v ? c.vc : c.kc) + blk * P * D;
    const int e = (int)(is_v ? c.vs : c.ks)[blk] - 127;
    void* y = const_cast<void*>(is_v ? a.v : a.k);
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const int64_t y0 = (int64_t)b.row0 * ld + h * (is_v ? a.ldv_head : a.ldk_head);
    const int g0 = b.t0 >> 4, tasks = (((b.t1 + 15) >> 4) - g0) * quads;
    for (int i = lane; i < tasks; i += 64) {
        const int g = g0 + i / quads, d = (i % quads) * 4;
        uint32_t w[16];  // 4 channels of each of the 16 tokens
        if (is_v) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 v = *reinterpret_cast<const uint4*>(codes + (d + j) * P + 16 * g);
                w[j] = v.x, w[4 + j] = v.y, w[8 + j] = v.z, w[12 + j] = v.w;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t s4[4] = {w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
                transpose4(s4);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * q + j] = s4[j];
            }
        } else {
#pragma unroll
            for (int t = 0; t < 16; ++t) w[t] = *reinterpret_cast<const uint32_t*>(codes + (16 * g + t) * D + d);
        }
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const int at = 16 * g + t;
            if (at < b.t0 || at >= b.t1) continue;
            float v[4];
            decode4(w[t], e, v);
            store4<DT>(y, y0 + (int64_t)(at - b.t0) * ld + d, v);
        }
    }
}

static dim3 kv_grid(const KvView& c) {
    const int64_t slots = c.T / c.P + 2 * (int64_t)c.S, rounds = (slots + kMaxGrid - 1) / kMaxGrid;
    return dim3((unsigned)std::min(slots, kMaxGrid), (unsigned)((c.H + kKvThreads / 64 - 1) / (kKvThreads / 64)),
                (unsigned)(2 * rounds));
}

hipError_t launch_kv_append(const KvRowsArgs& a, int dtype, hipStream_t s) {
    if (dtype == DT_BF16) hipLaunchKernelGGL(k_kv_append<DT_BF16>, kv_grid(a.c), dim3(kKvThreads), 0, s, a);
    else hipLaunchKernelGGL(k_kv_append<DT_F32>, kv_grid(a.c), dim3(kKvThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvRowsArgs& a, int dtype, hipStream_t s) {
    if (dtype == DT_BF16) hipLaunchKernelGGL(k_kv_read<DT_BF16>, kv_grid(a.c), dim3(kKvThreads), 0, s, a);
    else hipLaunchKernelGGL(k_kv_read<DT_F32>, kv_grid(a.c), dim3(kKvThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace bgf
