// Rows in pieces of 8 consecutive elements, one piece a lane and consecutive pieces in consecutive lanes:
// loads and stores of a wave are whole runs of memory, no transposition is needed, and a stochastic rounding's
// random words are one call a piece. An MX group of 32 is four lanes, a rotated chunk of n elements n / 8.
// The rotation's stages h = 1, 2, 4 run in registers, h = 8 .. 128 pair lane l with l ^ 1 .. l ^ 16, in the
// order and with the roundings of fwht_segment, so that the codes are the same as fp4_quantize's.
#pragma once

#include <type_traits>

#include "device.h"
#include "layer_internal.h"
#include "quant_block.h"

namespace bgf {

// raw words of a piece: 16 bytes of bf16, 32 of fp32
template <int DT>
struct Piece {
    static constexpr int N = DT == DT_BF16 ? 1 : 2;
    u32x4 w[N];
};

// NT: read once, not to be kept in the caches
template <int DT, bool NT = false>
__device__ __forceinline__ void piece_load(Piece<DT>& p, const void* base, int64_t elem) {
    const u32x4* s = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(base) + elem * (DT == DT_BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < Piece<DT>::N; ++i) p.w[i] = NT ? __builtin_nontemporal_load(s + i) : s[i];
}

template <int DT>
__device__ __forceinline__ void piece_zero(Piece<DT>& p) {
#pragma unroll
    for (int i = 0; i < Piece<DT>::N; ++i) p.w[i] = (u32x4){0u, 0u, 0u, 0u};
}

template <int DT>
__device__ __forceinline__ void piece_values(const Piece<DT>& p, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (DT == DT_BF16) v[j] = (j & 1) ? bf16_hi(p.w[0][j >> 1]) : bf16_lo(p.w[0][j >> 1]);
        else v[j] = __uint_as_float(p.w[j >> 2][j & 3]);
    }
}

template <int DT>
__device__ __forceinline__ Piece<DT> piece_pack(const float (&v)[8]) {
    Piece<DT> p;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        if constexpr (DT == DT_BF16) {
            p.w[0][j >> 1] = pack_bf16x2_rne(v[j], v[j + 1]);
        } else {
            p.w[j >> 2][j & 3] = __float_as_uint(v[j]);
            p.w[j >> 2][(j & 3) + 1] = __float_as_uint(v[j + 1]);
        }
    }
    return p;
}

template <int DT, bool NT = false>
__device__ __forceinline__ void piece_store(void* base, int64_t elem, const Piece<DT>& p) {
    u32x4* d = reinterpret_cast<u32x4*>(reinterpret_cast<char*>(base) + elem * (DT == DT_BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < Piece<DT>::N; ++i) {
        if constexpr (NT) __builtin_nontemporal_store(p.w[i], d + i);
        else d[i] = p.w[i];
    }
}

// One stage of the rotation between lanes l and l ^ M: a + b in the lower lane, a - b in the upper.
template <int M>
__device__ __forceinline__ void fwht_lanes(float (&v)[8]) {
    const float sgn = (__lane_id() & M) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], sgn, lane_xor<M>(v[i]));
}

// Blockwise H_n / sqrt(n), n in {0, 16, .., 256} the same for the whole wave, every lane taking part.
__device__ __forceinline__ void fwht_piece(float (&v)[8], int n) {
    if (n == 0) return;
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & h)) {
                const float a = v[i], b = v[i + h];
                v[i] = a + b;
                v[i + h] = a - b;
            }
    fwht_lanes<1>(v);
    if (n >= 32) fwht_lanes<2>(v);
    if (n >= 64) fwht_lanes<4>(v);
    if (n >= 128) fwht_lanes<8>(v);
    if (n >= 256) fwht_lanes<16>(v);
    const float c = n == 16 ? inv_sqrt_n<16>() : n == 32 ? inv_sqrt_n<32>() : n == 64 ? inv_sqrt_n<64>()
                  : n == 128 ? inv_sqrt_n<128>() : inv_sqrt_n<256>();
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * c;
}

// Codes of a piece under the block exponent k: 4 bytes of E2M1 in out[0], 8 of E4M3 in out[0], out[1].
template <int ELEM, int RND>
__device__ __forceinline__ void piece_encode(float (&v)[8], int k, uint64_t seed, uint64_t idx, uint32_t (&out)[2]) {
    if (k == -127) {  // 2^-127 is not a normal fp32: 2^-126 after doubling (exact for such tiny values)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * 2.0f;
        k = -126;
    }
    const float scale = pow2f(k);
    if constexpr (RND == RND_RNE) {
        if constexpr (ELEM == ELEM_E2M1) {
            uint32_t r = cvt_fp4x2<0>(0u, v[0], v[1], scale);
            r = cvt_fp4x2<1>(r, v[2], v[3], scale);
            r = cvt_fp4x2<2>(r, v[4], v[5], scale);
            out[0] = cvt_fp4x2<3>(r, v[6], v[7], scale);
        } else {
            const float top = 448.0f * scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_fmed3f(v[i], -top, top);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t r = cvt_fp8x2<false>(0u, v[4 * w], v[4 * w + 1], scale);
                out[w] = cvt_fp8x2<true>(r, v[4 * w + 2], v[4 * w + 3], scale);
            }
        }
    } else {
        const float rcp = __builtin_amdgcn_ldexpf(1.0f, -k);
        uint32_t c[4];
        philox_group(SrSource{seed, idx}, 0, c);
        out[0] = out[1] = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (ELEM == ELEM_E2M1) out[0] |= e2m1_sr(v[j] * rcp, sr_u16(c, j)) << (4 * j);
            else out[j >> 2] |= e4m3_sr(v[j] * rcp, sr_u16(c, j)) << (8 * (j & 3));
        }
    }
}

// Rotate, scale and encode the wave's pieces and store those that are `valid`. idx: the piece's first
// element in the row-major output (a multiple of 8; pieces of a group in four lanes 4 i .. 4 i + 3).
template <int RND>
__device__ __forceinline__ void piece_quantize(const QuantOut& q, float (&v)[8], int64_t idx, bool valid) {
    fwht_piece(v, q.hn);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    m = fmaxf(m, lane_xor<1>(m));
    m = fmaxf(m, lane_xor<2>(m));
    uint32_t out[2];
    int k;
    if (q.elem == ELEM_E2M1) {
        k = e8m0_exp<2, 0x400000u>(m, q.ceil_rule != 0);
        piece_encode<ELEM_E2M1, RND>(v, k, q.seed, (uint64_t)idx, out);
        if (valid) *reinterpret_cast<uint32_t*>(q.codes + (idx >> 1)) = out[0];
    } else {
        k = e8m0_exp<8, 0x600000u>(m, q.ceil_rule != 0);
        piece_encode<ELEM_E4M3, RND>(v, k, q.seed, (uint64_t)idx, out);
        if (valid) *reinterpret_cast<u32x2*>(q.codes + idx) = (u32x2){out[0], out[1]};
    }
    if (valid && !(__lane_id() & 3)) q.scales[idx >> 5] = (uint8_t)(k + 127);
}

// The activation of a gated feed-forward and its derivative, in few operations and nowhere far from fp32's own
// rounding. Their number is what the tiles' epilogue and the coded backward pass last by: the sigmoid as
// rcp(1 + exp(-x)) of the hardware's two instructions is off by 64 half steps (2^-24) at -80 and 17 at -20, this
// one by 5 to -20 and 7 to -87, for 1 % of the tiles' time and of the backward pass's (4096 rows, K 4096, F 11008,
// 4 bits: 249.4 -> 251.9 us; backward with codes 95.7 -> 96.9); with the exact quotient alone a round of tiles takes
// 5 us more.

// e^-y for y >= 0: 2^t by the hardware (an ulp) with t = RN(-y log2 e), times 1 + d for what t leaves of the exponent,
// d = -y - t ln 2, which is less than 2^-17. ln 2 as one fp32 is 2^-29 off, which t passes on: a rounding at y = 20,
// four at 87. y past 104, infinity too, is taken as 104, where the result is 0; so are results below 2^-126.
__device__ __forceinline__ float exp_minus(float y) {
    y = __builtin_amdgcn_fmed3f(y, 0.0f, 104.0f);  // (fminf takes two instructions)
    const float t = -y * 1.44269504f;
    const float d = __builtin_fmaf(t, -0.69314718f, -y);
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, d, e);
}

// p = 1 / (1 + e^-x) and its derivative p (1 - p), both to a few roundings of themselves: with e = e^-|x| <= 1 they
// come from r = 1 / (1 + e) and s = e r, whose divisor lies in [1, 2] (the hardware's reciprocal: an ulp). p of positive
// x is 1 - s, whose error is a share of the smaller of the two (root mean square of normal arguments of size 1.5: 0.58
// half steps, with r 0.78; the exact exponential and quotient 0.68).
__device__ __forceinline__ float sigmoid(float x, float& slope) {
    const float e = exp_minus(fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e), s = e * r;
    slope = r * s;
    return x < 0.0f ? s : 1.0f - s;
}

// Phi(g) of the normal distribution, and e = e^(-g^2 / 2), both to a few roundings of themselves: (1 + erf(g / sqrt 2))
// / 2 cancels for negative g, 4 % off at -5 and 0 at -5.8. Up to |g| = 1 it is 1 / 2 + g R(g^2), past it the tail
// Phi(-a), a = |g|, or one minus that; the tail is e times Q(a) = erfcx(a / sqrt 2) / 2, a smooth function: s P(s) with
// s = 1 / (1 + 0.33 a). R of degree 5 and P of degree 7 are fitted for the least relative error over [0, 1] and [1,
// 14.6] (0.012 and 0.16 half steps). The square's own rounding, which the exponential would pass on a^2 / 2 times, goes
// into the exponent. All of it takes less than the two branches of erff do (4096 rows, K 4096, F 11008, 4 bits: 287 ->
// 267 us, backward with codes 117 -> 113).
__device__ __forceinline__ float normal_cdf(float g, float& e) {
    const float a = __builtin_amdgcn_fmed3f(fabsf(g), 0.0f, 14.5f), w = a * a;
    const float x = exp_minus(0.5f * w);
    e = __builtin_fmaf(-0.5f * x, __builtin_fmaf(a, a, -w), x);
    const float s = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.33f, 1.0f));
    float p = __builtin_fmaf(s, 0.043525774f, -0.13791771f);
    p = __builtin_fmaf(s, p, 0.108361416f);
    p = __builtin_fmaf(s, p, 0.006608054f);
    p = __builtin_fmaf(s, p, 0.10068161f);
    p = __builtin_fmaf(s, p, 0.115317486f);
    p = __builtin_fmaf(s, p, 0.13183379f);
    p = __builtin_fmaf(s, p, 0.13164388f);
    const float tail = e * (s * p);
    float r = __builtin_fmaf(w, -7.654211e-6f, 1.1348638e-4f);
    r = __builtin_fmaf(w, r, -1.18633e-3f);
    r = __builtin_fmaf(w, r, 9.973323e-3f);
    r = __builtin_fmaf(w, r, -6.649036e-2f);
    r = __builtin_fmaf(w, r, 0.3989423f);
    const float far = g < 0.0f ? tail : 1.0f - tail;
    return a < 1.0f ? __builtin_fmaf(g, r, 0.5f) : far;
}

// (1 + tanh z) / 2 = sigmoid(2 z): 2 z = g (2 sqrt(2 / pi) + 0.044715 * 2 sqrt(2 / pi) g^2)
constexpr float kTanhA = 1.5957691216057308f, kTanhB = 0.07135481627260025f;

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    float unused;
    if constexpr (ACT == ACT_SILU) return g * sigmoid(g, unused);
    else if constexpr (ACT == ACT_GELU) return g * normal_cdf(g, unused);
    else return g * sigmoid(g * __builtin_fmaf(g * g, kTanhB, kTanhA), unused);
}

template <int ACT>
__device__ __forceinline__ void act_slope(float g, float& a, float& d) {
    float dp;
    if constexpr (ACT == ACT_SILU) {
        const float p = sigmoid(g, dp);
        a = g * p;
        d = __builtin_fmaf(g, dp, p);
    } else if constexpr (ACT == ACT_GELU) {
        const float p = normal_cdf(g, dp);
        a = g * p;
        d = __builtin_fmaf(g * 0.39894228040143268f, dp, p);
    } else {
        const float w = g * g, p = sigmoid(g * __builtin_fmaf(w, kTanhB, kTanhA), dp);
        a = g * p;
        // (the square held finite: it meets a factor of 0 where it would not be)
        d = __builtin_fmaf(g * dp, __builtin_fmaf(fminf(w, 1e37f), 3.0f * kTanhB, kTanhA), p);
    }
}

// f(ACT) of the call's activation. Chosen once for all the values of a tile: value by value, each activation pays for
// the registers and the code of the others (SiLU, 4096 rows: 243.9 us chosen once, 9 more value by value).
template <typename F>
__device__ __forceinline__ void by_act(int act, F f) {
    if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
    else if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
    else f(std::integral_constant<int, ACT_GELU_TANH>{});
}

}  // namespace bgf
