// The key / value cache: rows of K and V quantized into their pages as they are written, and read
// back. One workgroup works for one block (page x kv head) of K or of V (grid z).
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

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (DT == DT_BF16) {
        const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(q[i]);
            v[2 * i + 1] = bf16_hi(q[i]);
        }
    } else {
        const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
        const float4 a = f[0], b = f[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// four E4M3 codes under a smaller scale: c * f, f = 2^(old - e) <= 1/2, nearest even
__device__ __forceinline__ uint32_t requant4(uint32_t w, float f) {
    const v2f a = fp8x2_to_f32<false>(w), b = fp8x2_to_f32<true>(w);
    uint32_t r = cvt_fp8x2<false>(0u, a[0] * f, a[1] * f, 1.0f);
    return cvt_fp8x2<true>(r, b[0] * f, b[1] * f, 1.0f);
}

template <int DT>
__global__ __launch_bounds__(kKvThreads) void k_kv_append(KvRowsArgs a) {
    const KvView& c = a.c;
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const KvBlock b = kv_block(c, blockIdx.x);
    if (b.page < 0) return;
    const int tid = threadIdx.x, D = c.D, P = c.P;
    const int64_t blk = (int64_t)b.page * c.H + h;
    uint8_t* codes = (is_v ? c.vc : c.kc) + blk * P * D;
    uint8_t* scales = (is_v ? c.vs : c.ks) + blk;
    const void* x = is_v ? a.v : a.k;
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const int64_t x0 = (int64_t)b.row0 * ld + h * (is_v ? a.ldv_head : a.ldk_head);
    const int per = D >> 3, chunks = (b.t1 - b.t0) * per;
    __shared__ uint32_t smax[kKvThreads / 64];
    __shared__ uint32_t tile[128 * 256 / 4];  // V: the new codes, [token][D], before their transposition

    const uint32_t old_code = *scales;
    // amax of the new tokens (as integers: |x| orders like its bits)
    uint32_t m = 0;
    for (int i = tid; i < chunks; i += kKvThreads) {
        const int t = i / per, d = (i - t * per) * 8;
        float v[8];
        load8<DT>(x, x0 + t * ld + d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if ((tid & 63) == 0) smax[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKvThreads / 64; ++i) m = max(m, smax[i]);
    int e = e8m0_exp<8, 0x600000u>(__uint_as_float(m), a.ceil_rule != 0);
    if (b.begun) e = max(e, (int)old_code - 127);
    if (tid == 0) *scales = (uint8_t)(e + 127);

    if (b.begun && e + 127 > (int)old_code) {  // the older tokens under the block's new scale
        const int diff = (int)old_code - 127 - e;
        const float f = __builtin_amdgcn_ldexpf(1.0f, diff);
        if (is_v) {
            const int groups = (b.t0 + 15) >> 4;
            for (int i = tid; i < D * groups; i += kKvThreads) {
                const int d = i / groups, g = i - d * groups;
                uint4* p = reinterpret_cast<uint4*>(codes + d * P + 16 * g);
                const uint4 v = *p;
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // bytes of the places before t0 only
                    const int n = min(max(b.t0 - 16 * g - 4 * j, 0), 4);
                    const uint32_t old = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
                    w[j] = (requant4(w[j], f) & old) | (w[j] & ~old);
                }
                *p = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            for (int i = tid; i < b.t0 * (D >> 4); i += kKvThreads) {
                uint4* p = reinterpret_cast<uint4*>(codes) + i;
                uint4 w = *p;
                w = make_uint4(requant4(w.x, f), requant4(w.y, f), requant4(w.z, f), requant4(w.w, f));
                *p = w;
            }
        }
        __syncthreads();
    }

    // the new tokens: x * 2^-e by the scaled convert, which divides by 2^e exactly; 2^-127 is not a
    // normal fp32, so that exponent is reached by doubling x
    const float dbl = e == -127 ? 2.0f : 1.0f;
    const float sc = pow2f(max(e, -126));
    const float lim = fminf(448.0f * sc, 3.40282347e38f);
    uint8_t* const tb = reinterpret_cast<uint8_t*>(tile);
    for (int i = tid; i < chunks; i += kKvThreads) {
        const int t = i / per, d = (i - t * per) * 8;
        float v[8];
        load8<DT>(x, x0 + t * ld + d, v);
        uint32_t r[2];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_fmed3f(v[j] * dbl, -lim, lim);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            r[j] = cvt_fp8x2<false>(0u, v[4 * j], v[4 * j + 1], sc);
            r[j] = cvt_fp8x2<true>(r[j], v[4 * j + 2], v[4 * j + 3], sc);
        }
        uint8_t* dst = is_v ? tb + t * D + d : codes + (b.t0 + t) * D + d;
        *reinterpret_cast<uint2*>(dst) = make_uint2(r[0], r[1]);
    }
    if (!is_v) return;
    __syncthreads();
    // V goes to the page channel by channel: 16 tokens at once where all 16 are new, else bytes
    const int g0 = b.t0 >> 4, groups = ((b.t1 + 15) >> 4) - g0;
    for (int i = tid; i < D * groups; i += kKvThreads) {
        const int g = i / D, d = i - g * D;
        const int lo = (g0 + g) * 16;
        uint8_t* dst = codes + d * P + lo;
        if (lo >= b.t0 && lo + 16 <= b.t1) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) w[j] |= (uint32_t)tb[(lo - b.t0 + 4 * j + k) * D + d] << (8 * k);
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int t = max(lo, b.t0); t < min(lo + 16, b.t1); ++t) dst[t - lo] = tb[(t - b.t0) * D + d];
        }
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
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const KvBlock b = kv_block(c, blockIdx.x);
    if (b.page < 0) return;
    const int tid = threadIdx.x, D = c.D, P = c.P;
    const int64_t blk = (int64_t)b.page * c.H + h;
    const uint8_t* codes = (is_v ? c.vc : c.kc) + blk * P * D;
    const int e = (int)(is_v ? c.vs : c.ks)[blk] - 127;
    void* y = const_cast<void*>(is_v ? a.v : a.k);
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const int64_t y0 = (int64_t)b.row0 * ld + h * (is_v ? a.ldv_head : a.ldk_head);
    const int per = D >> 2, n = b.t1 - b.t0;
    __shared__ uint32_t tile[256 * (128 / 4 + 1)];  // V: the page, channels 4 bytes apart beyond P
    const int pitch = P + 4;
    const uint8_t* tb = reinterpret_cast<const uint8_t*>(tile);
    if (is_v) {
        const int groups = P >> 4;
        for (int i = tid; i < D * groups; i += kKvThreads) {
            const int d = i / groups, g = i - d * groups;
            const uint4 w = *reinterpret_cast<const uint4*>(codes + d * P + 16 * g);
            uint32_t* dst = tile + (d * pitch + 16 * g) / 4;
            dst[0] = w.x, dst[1] = w.y, dst[2] = w.z, dst[3] = w.w;
        }
        __syncthreads();
    }
    for (int i = tid; i < n * per; i += kKvThreads) {
        const int t = i / per, d = (i - t * per) * 4;
        uint32_t w;
        if (is_v) {
            const uint8_t* p = tb + d * pitch + b.t0 + t;
            w = (uint32_t)p[0] | ((uint32_t)p[pitch] << 8) | ((uint32_t)p[2 * pitch] << 16) | ((uint32_t)p[3 * pitch] << 24);
        } else {
            w = *reinterpret_cast<const uint32_t*>(codes + (b.t0 + t) * D + d);
        }
        float v[4];
        decode4(w, e, v);
        store4<DT>(y, y0 + t * ld + d, v);
    }
}

static dim3 kv_grid(const KvView& c) {
    return dim3((unsigned)(c.T / c.P + 2 * c.S), (unsigned)c.H, 2);
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
