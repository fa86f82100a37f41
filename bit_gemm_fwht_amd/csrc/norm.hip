// Root-mean-square norm of rows with the residual's addition and a low-bit output, and its backward pass.
//
// Forward, a row s = RN(x + r): y = s w / sqrt(mean s^2 + eps). One pass over memory: a row's pieces of 8
// elements (piece.h) stay in registers between the sum of squares and the output, so x and r are read once
// and s, y and the codes written once.
#include "device.h"
#include "layer_internal.h"
#include "piece.h"

namespace bgf {

constexpr int kNormThreads = 512;  // of a workgroup at most: rows of 32768 in 8 pieces a lane

// Sums of a and b over the `lanes` lanes of a row (a power of two; above 64 the whole workgroup), in a fixed
// order. red: 2 floats a wave; every thread of the workgroup calls it.
__device__ __forceinline__ void row_sums(float& a, float& b, int lanes, float* red) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        if (m < lanes) {
            a += __shfl_xor(a, m);
            b += __shfl_xor(b, m);
        }
    }
    if (lanes > 64) {
        const int nw = blockDim.x >> 6, wave = threadIdx.x >> 6;
        __syncthreads();  // the last row's sums have been read
        if ((threadIdx.x & 63) == 0) {
            red[2 * wave] = a;
            red[2 * wave + 1] = b;
        }
        __syncthreads();
        a = red[0];
        b = red[1];
        for (int i = 1; i < nw; ++i) {
            a += red[2 * i];
            b += red[2 * i + 1];
        }
    }
}

template <int IN, int NP, int FQ>
__global__ __launch_bounds__(kNormThreads) void k_rmsnorm(NormArgs a, int lanes) {
    __shared__ float red[2 * kNormThreads / 64];
    const int at = threadIdx.x & (lanes - 1), per = blockDim.x / lanes, sub = threadIdx.x / lanes;
    const int pieces = a.cols >> 3;
    const float inv_cols = 1.0f / (float)a.cols;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < a.rows; r0 += (int64_t)gridDim.x * per) {
        const int64_t row = r0 + sub;
        const bool in = row < a.rows;
        Piece<IN> x[NP], r[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = at + lanes * i;
            piece_zero<IN>(x[i]);
            piece_zero<IN>(r[i]);
            if (in && p < pieces) {
                piece_load<IN>(x[i], a.x, row * a.ldx + 8 * p);
                if (a.r) piece_load<IN>(r[i], a.r, row * a.ldr + 8 * p);
            }
        }
        float v[NP][8], ss = 0.0f, none = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = at + lanes * i;
            piece_values<IN>(x[i], v[i]);
            if (a.r) {
                float rv[8];
                piece_values<IN>(r[i], rv);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += rv[j];
                const Piece<IN> s = piece_pack<IN>(v[i]);
                piece_values<IN>(s, v[i]);  // what the sum holds is what is normed
                if (in && p < pieces) piece_store<IN>(a.sum, row * a.lds + 8 * p, s);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
        }
        row_sums(ss, none, lanes, red);
        const float rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = at + lanes * i;
            const bool here = in && p < pieces;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.0f;
            if (a.w && here) {
                if (a.w_bf16) {
                    Piece<DT_BF16> t;
                    piece_load<DT_BF16>(t, a.w, 8 * p);
                    piece_values<DT_BF16>(t, w);
                } else {
                    Piece<DT_F32> t;
                    piece_load<DT_F32>(t, a.w, 8 * p);
                    piece_values<DT_F32>(t, w);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
            if (a.y && here) piece_store<IN>(a.y, row * a.ldy + 8 * p, piece_pack<IN>(v[i]));
            // every lane takes part: a group's and a chunk's lanes exchange values
            if constexpr (FQ != 0)
                piece_quantize<FQ == 2 ? RND_SR : RND_RNE>(a.q, v[i], row * a.cols + 8 * p, here);
        }
    }
}

// lanes of a row: a power of two that covers its pieces, at most `most`
static int row_lanes(int cols, int most) {
    int lanes = 8;
    while (lanes < most && lanes < cols / 8) lanes *= 2;
    return lanes;
}

template <int IN, int FQ>
static hipError_t launch_rmsnorm_k(const NormArgs& a, hipStream_t s) {
    const int pieces = (a.cols + 7) / 8;
    const int lanes = row_lanes(a.cols, kNormThreads);
    const int threads = lanes > 64 ? lanes : 256, per = threads / lanes;  // above a wave: one row a workgroup
    const int64_t need = (a.rows + per - 1) / per;
    const unsigned grid = (unsigned)(need < kMaxGrid ? need : kMaxGrid);
    const int np = (pieces + lanes - 1) / lanes;
    if (np <= 1) hipLaunchKernelGGL((k_rmsnorm<IN, 1, FQ>), dim3(grid), dim3(threads), 0, s, a, lanes);
    else if (np <= 2) hipLaunchKernelGGL((k_rmsnorm<IN, 2, FQ>), dim3(grid), dim3(threads), 0, s, a, lanes);
    else if (np <= 4) hipLaunchKernelGGL((k_rmsnorm<IN, 4, FQ>), dim3(grid), dim3(threads), 0, s, a, lanes);
    else hipLaunchKernelGGL((k_rmsnorm<IN, 8, FQ>), dim3(grid), dim3(threads), 0, s, a, lanes);
    return hipGetLastError();
}

hipError_t launch_rmsnorm(const NormArgs& a, int dtype, int rnd, hipStream_t s) {
    const int fq = !a.q.codes ? 0 : rnd == RND_SR ? 2 : 1;
    if (dtype == DT_BF16)
        return fq == 0 ? launch_rmsnorm_k<DT_BF16, 0>(a, s) : fq == 1 ? launch_rmsnorm_k<DT_BF16, 1>(a, s) : launch_rmsnorm_k<DT_BF16, 2>(a, s);
    return fq == 0 ? launch_rmsnorm_k<DT_F32, 0>(a, s) : fq == 1 ? launch_rmsnorm_k<DT_F32, 1>(a, s) : launch_rmsnorm_k<DT_F32, 2>(a, s);
}

// ---------------------------------------------------------------------------------------------
// Backward: with r = 1 / sqrt(mean s^2 + eps), n = s r, a = dy w:
//   dx = dsum + r (a - n mean(a n)),  dw = sum over rows of dy n.
// Both means come from one pass over the row (sum s^2 and sum a s, then mean(a n) = r sum(a s) / cols). A
// workgroup keeps its rows' part of dw in registers and writes it once; k_sum_slots adds the parts.
// ---------------------------------------------------------------------------------------------
template <int IN, int NP>
__global__ __launch_bounds__(kNormThreads) void k_rmsnorm_grad(NormGradArgs a, int lanes) {
    __shared__ float red[2 * kNormThreads / 64];
    const int at = threadIdx.x & (lanes - 1), per = blockDim.x / lanes, sub = threadIdx.x / lanes;
    const int pieces = a.cols >> 3;
    const float inv_cols = 1.0f / (float)a.cols;
    float dw[NP][8], w[NP][8];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = at + lanes * i;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = 0.0f;
            w[i][j] = 1.0f;
        }
        if (a.w && p < pieces) {
            if (a.w_bf16) {
                Piece<DT_BF16> t;
                piece_load<DT_BF16>(t, a.w, 8 * p);
                piece_values<DT_BF16>(t, w[i]);
            } else {
                Piece<DT_F32> t;
                piece_load<DT_F32>(t, a.w, 8 * p);
                piece_values<DT_F32>(t, w[i]);
            }
        }
    }
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < a.rows; r0 += (int64_t)gridDim.x * per) {
        const int64_t row = r0 + sub;
        const bool in = row < a.rows;
        Piece<IN> s[NP], dy[NP], ds[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = at + lanes * i;
            piece_zero<IN>(s[i]);
            piece_zero<IN>(dy[i]);
            piece_zero<IN>(ds[i]);
            if (in && p < pieces) {
                piece_load<IN>(s[i], a.s, row * a.lds + 8 * p);
                piece_load<IN>(dy[i], a.dy, row * a.lddy + 8 * p);
                if (a.dsum) piece_load<IN>(ds[i], a.dsum, row * a.lddsum + 8 * p);
            }
        }
        float ss = 0.0f, as = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float sv[8], dv[8];
            piece_values<IN>(s[i], sv);
            piece_values<IN>(dy[i], dv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = __builtin_fmaf(sv[j], sv[j], ss);
                as = __builtin_fmaf(dv[j] * w[i][j], sv[j], as);
            }
        }
        row_sums(ss, as, lanes, red);
        const float rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
        const float c = as * inv_cols * rstd * rstd;  // mean(a n) r: dx = r (a - s c) + dsum
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = at + lanes * i;
            float sv[8], dv[8], o[8], base[8];
            piece_values<IN>(s[i], sv);
            piece_values<IN>(dy[i], dv);
            piece_values<IN>(ds[i], base);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = __builtin_fmaf(rstd, dv[j] * w[i][j] - sv[j] * c, base[j]);
                dw[i][j] = __builtin_fmaf(dv[j], sv[j] * rstd, dw[i][j]);
            }
            if (in && p < pieces) piece_store<IN>(a.dx, row * a.lddx + 8 * p, piece_pack<IN>(o));
        }
    }
    if (!a.part) return;
    // rows that share a wave are added lane by lane; then one slot a wave (rows of up to 64 lanes) or workgroup
    const int64_t slot = lanes > 64 ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = at + lanes * i;
#pragma unroll
        for (int m = 8; m < 64; m <<= 1) {
            if (m >= lanes) {
#pragma unroll
                for (int j = 0; j < 8; ++j) dw[i][j] += __shfl_xor(dw[i][j], m);
            }
        }
        if (p < pieces && (lanes > 64 || (threadIdx.x & 63) < lanes))
            piece_store<DT_F32>(a.part, slot * a.cols + 8 * p, piece_pack<DT_F32>(dw[i]));
    }
}

// dw[c] = sum of part[slot][c], slots in order within each of 64 runs, then the runs in order: 16 columns by 64 runs
// a workgroup.
__global__ __launch_bounds__(1024) void k_sum_slots(const float* part, int slots, int cols, float* dw) {
    __shared__ float run[64][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), g = threadIdx.x >> 4;
    const int each = (slots + 63) / 64, s0 = g * each, s1 = min(slots, s0 + each);
    float t = 0.0f;
    if (c < cols)
        for (int s = s0; s < s1; ++s) t += part[(int64_t)s * cols + c];
    run[g][threadIdx.x & 15] = t;
    __syncthreads();
    if (g == 0 && c < cols) {
        for (int i = 1; i < 64; ++i) t += run[i][threadIdx.x];
        dw[c] = t;
    }
}

NormGradPlan plan_rmsnorm_grad(int64_t rows, int cols, bool dw) {
    NormGradPlan p;
    p.lanes = row_lanes(cols, kNormThreads);
    p.threads = p.lanes > 64 ? p.lanes : 256;
    const int per = p.threads / p.lanes;
    const int64_t need = (rows + per - 1) / per, most = 512;
    p.grid = (int)(need < most ? need : most);
    p.slots = dw ? (p.lanes > 64 ? p.grid : p.grid * (p.threads / 64)) : 0;
    return p;
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& a, const NormGradPlan& p, int dtype, hipStream_t s) {
    if (p.grid > 0) {
        const int np = ((a.cols + 7) / 8 + p.lanes - 1) / p.lanes;
        const dim3 g(p.grid), t(p.threads);
        if (dtype == DT_BF16) {
            if (np <= 1) hipLaunchKernelGGL((k_rmsnorm_grad<DT_BF16, 1>), g, t, 0, s, a, p.lanes);
            else if (np <= 2) hipLaunchKernelGGL((k_rmsnorm_grad<DT_BF16, 2>), g, t, 0, s, a, p.lanes);
            else if (np <= 4) hipLaunchKernelGGL((k_rmsnorm_grad<DT_BF16, 4>), g, t, 0, s, a, p.lanes);
            else hipLaunchKernelGGL((k_rmsnorm_grad<DT_BF16, 8>), g, t, 0, s, a, p.lanes);
        } else {
            if (np <= 1) hipLaunchKernelGGL((k_rmsnorm_grad<DT_F32, 1>), g, t, 0, s, a, p.lanes);
            else if (np <= 2) hipLaunchKernelGGL((k_rmsnorm_grad<DT_F32, 2>), g, t, 0, s, a, p.lanes);
            else if (np <= 4) hipLaunchKernelGGL((k_rmsnorm_grad<DT_F32, 4>), g, t, 0, s, a, p.lanes);
            else hipLaunchKernelGGL((k_rmsnorm_grad<DT_F32, 8>), g, t, 0, s, a, p.lanes);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.dw) return hipSuccess;
    hipLaunchKernelGGL(k_sum_slots, dim3((a.cols + 15) / 16), dim3(1024), 0, s, a.part, p.slots, a.cols, a.dw);
    return hipGetLastError();
}

}  // namespace bgf
