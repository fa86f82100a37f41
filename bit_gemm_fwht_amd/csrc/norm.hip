// Root-mean-square norm of rows with the residual's addition and a low-bit output, and its backward pass.
//
// Forward, a row s = RN(x + r): y = s w / sqrt(mean s^2 + eps). One pass over memory: a row's pieces of 8
// elements (piece.h) stay in registers between the sum of squares and the output, so x and r are read once
// and s, y and the codes written once. Rows past 12288 columns nearly fill them: what would spill is worked out or read
// again (LEAN, again, apart below), and no instance uses scratch memory but one of the backward pass (bf16, 6 pieces a
// lane: 3 registers).
#include "device.h"
#include "launch.h"
#include "layer_internal.h"
#include "piece.h"

namespace bgf {

constexpr int kNormThreads = 512;  // of a workgroup at most: rows of 32768 in 8 pieces a lane

// Sums of a and b over the `lanes` lanes of a row (a power of two), in a fixed order. red: 2 floats a wave,
// another set for each of two calls that follow one another; every thread of the workgroup calls it.
__device__ __forceinline__ void row_sums(float& a, float& b, int lanes, float* red) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        if (m < lanes) {
            a += __shfl_xor(a, m);
            b += __shfl_xor(b, m);
        }
    }
    if (lanes > 64) {
        const int nw = lanes >> 6, wave = threadIdx.x >> 6, first = wave & -nw;  // the row's waves
        if ((threadIdx.x & 63) == 0) {
            red[2 * wave] = a;
            red[2 * wave + 1] = b;
        }
        __syncthreads();
        a = red[2 * first];
        b = red[2 * first + 1];
        for (int i = first + 1; i < first + nw; ++i) {
            a += red[2 * i];
            b += red[2 * i + 1];
        }
    }
}

// A piece of the weight as it is stored, and its values.
__device__ __forceinline__ void weight_load(Piece<DT_F32>& t, const void* w, int kind, int p) {
    if (kind == W_BF16) {
        Piece<DT_BF16> h;
        piece_load<DT_BF16>(h, w, 8 * p);
        t.w[0] = h.w[0];
    } else if (kind == W_F32) {
        piece_load<DT_F32>(t, w, 8 * p);
    }
}
__device__ __forceinline__ void weight_values(const Piece<DT_F32>& t, int kind, float (&v)[8]) {
    if (kind == W_BF16) {
        Piece<DT_BF16> h;
        h.w[0] = t.w[0];
        piece_values<DT_BF16>(h, v);
    } else if (kind == W_F32) {
        piece_values<DT_F32>(t, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    }
}

// The lane's place as if anew: what follows from it is worked out again, not held in registers.
__device__ __forceinline__ void again(int& at) { asm volatile("" : "+v"(at)); }

// Before a piece of a row that fills the registers: its loads are not moved up to those of the pieces before, and
// its places are worked out again, not held.
__device__ __forceinline__ void apart(int& at) { asm volatile("" : "+v"(at)::"memory"); }

// Loads are unconditional: lanes past the row's end or the last row read the last piece or row again, whose
// values count for nothing (a load behind a condition waits for the ones before it).
template <int IN, int NP, int FQ, bool RES, bool NT>
__global__ __launch_bounds__(kNormThreads) void k_rmsnorm(NormArgs a, int lanes) {
    __shared__ float red[2][2 * kNormThreads / 64];
    const int per = blockDim.x / lanes, sub = threadIdx.x / lanes;
    int at = threadIdx.x - sub * lanes;
    const int pieces = a.cols >> 3;
    const float inv_cols = 1.0f / (float)a.cols;
    Piece<IN> x[NP], r[NP];
    auto load = [&](int64_t r0, int i0, int i1) {
        const int64_t row = min(r0 + sub, a.rows - 1);
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            const int p = min(at + lanes * i, pieces - 1);
            piece_load<IN, NT>(x[i], a.x, row * a.ldx + 8 * p);
            if constexpr (RES) piece_load<IN, NT>(r[i], a.r, row * a.ldr + 8 * p);
        }
    };
    constexpr int W = 4 * Piece<IN>::N;  // registers of a piece as it is stored
    // Where a row's fp32 values, its weight and the next row nearly fill the registers, the addresses of its pieces,
    // which the compiler would hold from row to row, are worked out again for each (6000 rows with residual and codes,
    // held and worked out again: 20480 columns in bf16 330 and 275 us, in fp32 459 and 359). Without a residual to carry
    // that costs 2 to 3 % where nothing spills.
    constexpr bool LEAN = RES ? NP >= 6 : NP * (16 + W) + (FQ != 0) > 160;
    // The next row is loaded during the present one, but for fp32 of 8 pieces with a residual, where it has no room
    // (6000 rows of 32768: 671 us, spilled 1037).
    constexpr bool AHEAD = NP * (16 + W * (RES ? 2 : 1)) <= 192;
    if constexpr (AHEAD) load((int64_t)blockIdx.x * per, 0, NP);
    // the weight stays in registers where there is room beside the next row, else it is read again for each row
    constexpr bool KEPT = NP <= 2;
    Piece<DT_F32> w[NP];
    auto load_weight = [&]() {
#pragma unroll
        for (int i = 0; i < NP; ++i) weight_load(w[i], a.w, a.w_kind, min(at + lanes * i, pieces - 1));
    };
    if constexpr (KEPT) load_weight();
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < a.rows; r0 += (int64_t)gridDim.x * per, turn ^= 1) {
        const int64_t row = r0 + sub;
        const bool in = row < a.rows;
        if constexpr (LEAN) again(at);
        float v[NP][8], ss = 0.0f, none = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = at + lanes * i;
            if constexpr (!AHEAD) {
                if (i % 2 == 0) {
                    apart(at);
                    load(r0, i, i + 2);
                }
            }
            piece_values<IN>(x[i], v[i]);
            if constexpr (RES) {
                float rv[8];
                piece_values<IN>(r[i], rv);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += rv[j];
                const Piece<IN> s = piece_pack<IN>(v[i]);
                piece_values<IN>(s, v[i]);  // what the sum holds is what is normed
                if (in && p < pieces) piece_store<IN>(a.sum, row * a.lds + 8 * p, s);
            }
            if (p >= pieces) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
        }
        // the weight first: loads return in order; then the next row, on its way during this one's sums and codes
        if constexpr (LEAN) again(at);
        if constexpr (!KEPT) load_weight();
        if constexpr (AHEAD) load(r0 + (int64_t)gridDim.x * per, 0, NP);
        row_sums(ss, none, lanes, red[turn]);
        const float rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if constexpr (LEAN) again(at);
            const int p = at + lanes * i;
            const bool here = in && p < pieces;
            float wv[8];
            weight_values(w[i], a.w_kind, wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * wv[j];
            if (a.y && here) piece_store<IN>(a.y, row * a.ldy + 8 * p, piece_pack<IN>(v[i]));
            // every lane takes part: a group's and a chunk's lanes exchange values
            if constexpr (FQ != 0)
                piece_quantize<FQ == 2 ? RND_SR : RND_RNE>(a.q, v[i], row * a.cols + 8 * p, here);
        }
    }
}

// How a row's pieces are dealt: the lanes of a row and the pieces of a lane. Up to 64 pieces: a part of a wave, a
// power of two of lanes, one piece each. Above: one row a workgroup of 1, 2, 4 or 8 waves (5 on 4 SIMDs: 6000 rows of
// 5120 in 68.5 us, 4 waves with 3 pieces a lane 53.6), so that few lanes are idle, and then with 2 pieces a lane, which
// keep more of a row in flight (8192 rows of 4096: 52.6 us, with 1 piece 59.9, with 4 59.4), or 1 where all rows
// are resident at once and a row's latency counts (one row of 4096: 4.0 us against 5.1).
struct RowPlan {
    int lanes, np;
};
static RowPlan plan_row(int cols, bool few) {
    const int pieces = cols / 8;
    RowPlan best{8, 1};
    if (pieces <= 64) {
        while (best.lanes < pieces) best.lanes *= 2;
        return best;
    }
    const int nps[] = {few ? 1 : 2, few ? 2 : 1, 3, 4, 6, 8};
    int idle = 1 << 30;
    for (int np : nps)
        for (int lanes = 64; lanes <= kNormThreads; lanes *= 2)
            if (lanes * np >= pieces && lanes * np - pieces < idle) {
                idle = lanes * np - pieces;
                best = RowPlan{lanes, np};
            }
    return best;
}

template <int IN, int FQ, bool RES, bool NT>
static hipError_t launch_rmsnorm_r(const NormArgs& a, hipStream_t s) {
    int cus = 0;
    const hipError_t e = cu_count(&cus);
    if (e != hipSuccess) return e;
    const bool few = a.rows <= 4 * cus;
    const RowPlan r = plan_row(a.cols, few);
    const int threads = r.lanes > 64 ? r.lanes : 256, per = threads / r.lanes;
    // few rows: a workgroup each; else 1024 threads a CU, which go through several rows with the next one on its way
    // (8192 rows of 4096: 49.6 us, with 2048 threads a CU 51.9, a workgroup for each row 54.2)
    const int64_t need = (a.rows + per - 1) / per, most = few ? need : (int64_t)cus * (1024 / threads);
    const dim3 grid((unsigned)(need < most ? need : most)), block(threads);
    if (r.np == 1) hipLaunchKernelGGL((k_rmsnorm<IN, 1, FQ, RES, NT>), grid, block, 0, s, a, r.lanes);
    else if (r.np == 2) hipLaunchKernelGGL((k_rmsnorm<IN, 2, FQ, RES, NT>), grid, block, 0, s, a, r.lanes);
    else if (r.np == 3) hipLaunchKernelGGL((k_rmsnorm<IN, 3, FQ, RES, NT>), grid, block, 0, s, a, r.lanes);
    else if (r.np == 4) hipLaunchKernelGGL((k_rmsnorm<IN, 4, FQ, RES, NT>), grid, block, 0, s, a, r.lanes);
    else if (r.np == 6) hipLaunchKernelGGL((k_rmsnorm<IN, 6, FQ, RES, NT>), grid, block, 0, s, a, r.lanes);
    else hipLaunchKernelGGL((k_rmsnorm<IN, 8, FQ, RES, NT>), grid, block, 0, s, a, r.lanes);
    return hipGetLastError();
}

template <int IN, int FQ>
static hipError_t launch_rmsnorm_k(const NormArgs& a, hipStream_t s) {
    // bf16 that is more than the caches keep is not kept there (128 MiB read: 52.6 us, kept 54.4; 64 MiB: kept 35.1,
    // not kept 38.4). fp32 always is: a lane's two 16-byte halves touch the same cache line one after the other.
    if constexpr (IN == DT_BF16) {
        if (a.rows * a.cols * (a.r ? 4 : 2) >= (int64_t(96) << 20))
            return a.r ? launch_rmsnorm_r<IN, FQ, true, true>(a, s) : launch_rmsnorm_r<IN, FQ, false, true>(a, s);
    }
    return a.r ? launch_rmsnorm_r<IN, FQ, true, false>(a, s) : launch_rmsnorm_r<IN, FQ, false, false>(a, s);
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
template <int IN, int NP, bool NT>
__global__ __launch_bounds__(kNormThreads) void k_rmsnorm_grad(NormGradArgs a, int lanes) {
    __shared__ float red[2][2 * kNormThreads / 64];
    const int per = blockDim.x / lanes, sub = threadIdx.x / lanes;
    int at = threadIdx.x - sub * lanes;
    const int pieces = a.cols >> 3;
    const float inv_cols = 1.0f / (float)a.cols;
    // What a lane holds of a row from the sums to the result: all three inputs and the weight where they fit beside its
    // part of dw, else s and dy, or s alone; the others are read again where they are used (6000 rows, spilled and read
    // again: 32768 columns in bf16 578 and 424 us, in fp32 1272 and 712; 24576 in fp32 586 and 497).
    constexpr int W = 4 * Piece<IN>::N;
    constexpr bool ALL = NP * (16 + 3 * W) <= 168, DS = NP * (8 + 3 * W) <= 128, DY = NP * (8 + 2 * W) <= 160;
    constexpr int NW = ALL ? NP : 1, NS = DS ? NP : 1, ND = DY ? NP : 1;
    struct Row {
        Piece<IN> s[NP], dy[ND], ds[NS];
    };
    auto load_dy = [&](Piece<IN>& t, int64_t r0, int i) {
        piece_load<IN, NT>(t, a.dy, min(r0 + sub, a.rows - 1) * a.lddy + 8 * min(at + lanes * i, pieces - 1));
    };
    auto load = [&](Row& t, int64_t r0) {  // without conditions, as in the forward pass
        const int64_t row = min(r0 + sub, a.rows - 1);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int p = min(at + lanes * i, pieces - 1);
            piece_load<IN, NT>(t.s[i], a.s, row * a.lds + 8 * p);
            if constexpr (DY) load_dy(t.dy[i], r0, i);
            if constexpr (DS) {
                if (a.dsum) piece_load<IN, NT>(t.ds[i], a.dsum, row * a.lddsum + 8 * p);
                else piece_zero<IN>(t.ds[i]);
            }
        }
    };
    // the next row is loaded during the present one where both fit the registers
    constexpr bool AHEAD = NP * (IN == DT_BF16 ? 1 : 2) <= 3;
    const int64_t step = (int64_t)gridDim.x * per;
    Row next;
    if constexpr (AHEAD) load(next, (int64_t)blockIdx.x * per);
    float dw[NP][8];
    Piece<DT_F32> w[NW];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        if constexpr (ALL) weight_load(w[i], a.w, a.w_kind, min(at + lanes * i, pieces - 1));
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    auto weight = [&](int i, float (&v)[8]) {
        if constexpr (!ALL) weight_load(w[0], a.w, a.w_kind, min(at + lanes * i, pieces - 1));
        weight_values(w[ALL ? i : 0], a.w_kind, v);
    };
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < a.rows; r0 += step, turn ^= 1) {
        const int64_t row = r0 + sub;
        const bool in = row < a.rows;
        if constexpr (NP >= 4) again(at);
        Row t;
        if constexpr (AHEAD) {
            t = next;
            load(next, r0 + step);
        } else {
            load(t, r0);
        }
        float ss = 0.0f, as = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if constexpr (!ALL) apart(at);
            else if constexpr (NP >= 6) again(at);
            const bool here = in && at + lanes * i < pieces;
            float sv[8], dv[8], wv[8];
            piece_values<IN>(t.s[i], sv);
            if constexpr (!DY) load_dy(t.dy[0], r0, i);
            piece_values<IN>(t.dy[DY ? i : 0], dv);
            weight(i, wv);
            float q = 0.0f, d = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q = __builtin_fmaf(sv[j], sv[j], q);
                d = __builtin_fmaf(dv[j] * wv[j], sv[j], d);
            }
            ss += here ? q : 0.0f;
            as += here ? d : 0.0f;
            if constexpr (!ALL) asm volatile("" : "+v"(ss), "+v"(as));  // (added now: the piece's values are done with)
        }
        if constexpr (NP >= 4) again(at);
        row_sums(ss, as, lanes, red[turn]);
        const float rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
        const float c = as * inv_cols * rstd * rstd;  // mean(a n) r: dx = r (a - s c) + dsum
        if constexpr (NP >= 6) {  // as they were loaded: else their values and products are held from the sums to here
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int k = 0; k < Piece<IN>::N; ++k) asm volatile("" : "+v"(t.s[i].w[k]), "+v"(t.dy[DY ? i : 0].w[k]));
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if constexpr (!ALL) apart(at);
            else if constexpr (NP >= 6) again(at);
            const int p = at + lanes * i;
            const bool here = in && p < pieces;
            float sv[8], dv[8], wv[8], o[8], base[8];
            piece_values<IN>(t.s[i], sv);
            if constexpr (!DY) load_dy(t.dy[0], r0, i);
            piece_values<IN>(t.dy[DY ? i : 0], dv);
            if constexpr (!DS) {
                if (a.dsum) piece_load<IN, NT>(t.ds[0], a.dsum, min(row, a.rows - 1) * a.lddsum + 8 * min(p, pieces - 1));
                else piece_zero<IN>(t.ds[0]);
            }
            piece_values<IN>(t.ds[DS ? i : 0], base);
            weight(i, wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = __builtin_fmaf(rstd, dv[j] * wv[j] - sv[j] * c, base[j]);
                // (a row that is not there was read as another one)
                dw[i][j] = in ? __builtin_fmaf(dv[j], sv[j] * rstd, dw[i][j]) : dw[i][j];
            }
            if (here) piece_store<IN>(a.dx, row * a.lddx + 8 * p, piece_pack<IN>(o));
        }
    }
    if (!a.part) return;
    // the workgroup's rows are added: those that share a wave lane by lane, then the waves through LDS in their order;
    // a slot a workgroup
    __shared__ Piece<DT_F32> share[kNormThreads];
    const int wide = max(lanes, 64);
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
        if (wide < (int)blockDim.x) {
            share[threadIdx.x] = piece_pack<DT_F32>(dw[i]);
            __syncthreads();
            for (int k = threadIdx.x + wide; k < (int)blockDim.x; k += wide) {  // (of the first rows: all others)
                float v[8];
                piece_values<DT_F32>(share[k], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) dw[i][j] += v[j];
            }
            __syncthreads();
        }
        if (p < pieces && (int)threadIdx.x < lanes)
            piece_store<DT_F32>(a.part, (int64_t)blockIdx.x * a.cols + 8 * p, piece_pack<DT_F32>(dw[i]));
    }
}

// dw[c] = sum of part[slot][c] in a fixed order: 32 columns a workgroup, 4 a thread, the slots in 128 runs, then
// the runs by fours, then those 32.
__global__ __launch_bounds__(1024) void k_sum_slots(const float* part, int slots, int cols, float* dw) {
    __shared__ float run[128][33], four[32][33];
    const int k = threadIdx.x & 7, g = threadIdx.x >> 3, c = blockIdx.x * 32 + 4 * k;
    const int each = (slots + 127) / 128, s0 = g * each, s1 = min(slots, s0 + each);
    f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < cols)
        for (int s = s0; s < s1; ++s) t += *reinterpret_cast<const f32x4*>(part + (int64_t)s * cols + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) run[g][4 * k + i] = t[i];
    __syncthreads();
    const int col = threadIdx.x & 31, q = threadIdx.x >> 5;
    four[q][col] = (run[4 * q][col] + run[4 * q + 1][col]) + (run[4 * q + 2][col] + run[4 * q + 3][col]);
    __syncthreads();
    if (q == 0 && blockIdx.x * 32 + col < cols) {
        float v = four[0][col];
#pragma unroll
        for (int i = 1; i < 32; ++i) v += four[i][col];
        dw[blockIdx.x * 32 + col] = v;
    }
}

// 512 threads a CU: each carries its part of dw through many rows, so that the parts, which are written and
// read again, stay few (8192 rows of 4096: 52.7 us; with 1024 threads a CU 59.2, with 1 piece a lane 60.9). The
// number of CUs is the whole card's here and not asked of the device: it decides in which parts dw is added, and so the
// last bits, and the size of the workspace, which a program may ask for without a device.
constexpr int kGradGroups = 256;
NormGradPlan plan_rmsnorm_grad(int64_t rows, int cols, bool dw) {
    NormGradPlan p;
    const RowPlan r = plan_row(cols, rows <= 1024);
    p.lanes = r.lanes;
    p.np = r.np;
    // rows share a workgroup, and its part of dw, as soon as there is one for each CU (16384 rows of 1024: 29.5 us, a
    // part for each row in flight 34.4; 2048 rows of 2048: 12.9 and 17.0)
    p.threads = p.lanes > 64 ? p.lanes : 64;
    while (p.threads < kNormThreads && (rows * p.lanes + p.threads - 1) / p.threads > kGradGroups) p.threads *= 2;
    const int per = p.threads / p.lanes;
    const int64_t need = (rows + per - 1) / per;
    p.grid = (int)(need < kGradGroups ? need : kGradGroups);
    p.slots = dw ? p.grid : 0;
    return p;
}

template <int IN, bool NT>
static hipError_t launch_rmsnorm_grad_k(const NormGradArgs& a, const NormGradPlan& p, hipStream_t s) {
    const dim3 g(p.grid), t(p.threads);
    if (p.np == 1) hipLaunchKernelGGL((k_rmsnorm_grad<IN, 1, NT>), g, t, 0, s, a, p.lanes);
    else if (p.np == 2) hipLaunchKernelGGL((k_rmsnorm_grad<IN, 2, NT>), g, t, 0, s, a, p.lanes);
    else if (p.np == 3) hipLaunchKernelGGL((k_rmsnorm_grad<IN, 3, NT>), g, t, 0, s, a, p.lanes);
    else if (p.np == 4) hipLaunchKernelGGL((k_rmsnorm_grad<IN, 4, NT>), g, t, 0, s, a, p.lanes);
    else if (p.np == 6) hipLaunchKernelGGL((k_rmsnorm_grad<IN, 6, NT>), g, t, 0, s, a, p.lanes);
    else hipLaunchKernelGGL((k_rmsnorm_grad<IN, 8, NT>), g, t, 0, s, a, p.lanes);
    return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& a, const NormGradPlan& p, int dtype, hipStream_t s) {
    if (p.grid > 0) {
        const bool nt = a.rows * a.cols * (a.dsum ? 6 : 4) >= (int64_t(96) << 20);  // as in the forward pass
        const hipError_t e = dtype == DT_F32 ? launch_rmsnorm_grad_k<DT_F32, false>(a, p, s)
                             : nt            ? launch_rmsnorm_grad_k<DT_BF16, true>(a, p, s)
                                             : launch_rmsnorm_grad_k<DT_BF16, false>(a, p, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dw) return hipSuccess;
    hipLaunchKernelGGL(k_sum_slots, dim3((a.cols + 31) / 32), dim3(1024), 0, s, a.part, p.slots, a.cols, a.dw);
    return hipGetLastError();
}

}  // namespace bgf
