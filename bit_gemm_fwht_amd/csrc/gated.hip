// Gated feed-forward on block-scaled operands: h = act(A Wg^T) * (A Wu^T) in one launch, optionally with the
// two products kept (g | u) and h quantized along its columns; and its backward pass.
//
// Both products of a place are accumulated in the same lane's registers, so the activation and the product
// need no exchange and g and u never leave the chip unless they are asked for. Two kernels:
//  - k_gated_tile: the pipelined GEMM tile (gemm_tile.h) on B slabs that hold 32 rows of Wg and the same 32
//    of Wu in turn: 256 x 128 or 128 x 64 results a workgroup;
//  - k_gated_rows: few rows of A, and every K that the tiles do not take: 32 columns a workgroup, its waves
//    each multiply a share of K straight from memory (no LDS: no weight is used twice), the shares are added
//    through LDS in a fixed order.
#include "device.h"
#include "fp4_internal.h"
#include "gemm_tile.h"
#include "layer_internal.h"
#include "piece.h"

namespace bgf {

// Store a staged fp32 tile [ROWS][COLS] (row pitch `pitch` bytes in LDS) as dtype OUT at c[m0 ..][n0 ..],
// 16-byte pieces where the place allows; rows from M and columns from N on are not there.
template <int OUT, int ROWS, int COLS, int NTH>
__device__ __forceinline__ void store_staged(const uint8_t* lds, int pitch, char* c, int64_t ldc, int64_t m0, int64_t n0,
                                             int64_t M, int64_t N) {
    constexpr int ESZ = OUT == DT_F32 ? 4 : 2, EPC = 16 / ESZ, PPR = COLS / EPC;
    const bool vec_ok = ((reinterpret_cast<uintptr_t>(c) & 15) == 0) && ((ldc * ESZ) % 16 == 0);
#pragma unroll 2
    for (int t = threadIdx.x; t < ROWS * PPR; t += NTH) {
        const int r = t / PPR, k = (t % PPR) * EPC;
        const int64_t m = m0 + r, n = n0 + k;
        if (m >= M) break;
        const float* src = reinterpret_cast<const float*>(lds + r * pitch) + k;
        u32x4 val;
        if constexpr (OUT == DT_F32) {
            val = *reinterpret_cast<const u32x4*>(src);
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4*>(src), b = *reinterpret_cast<const f32x4*>(src + 4);
            val = (u32x4){pack_bf16x2_rne(a[0], a[1]), pack_bf16x2_rne(a[2], a[3]), pack_bf16x2_rne(b[0], b[1]),
                          pack_bf16x2_rne(b[2], b[3])};
        }
        char* cp = c + (m * ldc + n) * ESZ;
        if (vec_ok && n + EPC <= N) {
            *reinterpret_cast<u32x4*>(cp) = val;
        } else {
            for (int i = 0; i < EPC; ++i) {
                if (n + i < N) {
                    if constexpr (OUT == DT_F32) reinterpret_cast<uint32_t*>(cp)[i] = val[i];
                    else reinterpret_cast<uint16_t*>(cp)[i] = (uint16_t)(val[i >> 1] >> (16 * (i & 1)));
                }
            }
        }
    }
}

// Quantize 32 columns of row m from column n on (the lane's values; every lane of the wave takes part), nearest
// even: a stochastic rounding, which activations hardly use, is a pass of its own.
__device__ __forceinline__ void quantize_group(const GemmArgs& g, float (&v)[32], int64_t m, int64_t n) {
    fwht_groups(v, g.q_hn);
    uint32_t out[8];
    const float amax = block_amax<32, 0>(v);
    const SrSource sr{0, 0};
    const uint32_t s = g.q_elem == ELEM_E2M1 ? e8m0_block<ELEM_E2M1, RND_RNE, 32, 0>(v, amax, g.q_ceil != 0, sr, out)
                                             : e8m0_block<ELEM_E4M3, RND_RNE, 32, 0>(v, amax, g.q_ceil != 0, sr, out);
    if (m >= g.M || n >= g.N) return;
    if (g.q_elem == ELEM_E2M1) {
        *reinterpret_cast<u32x4*>(g.qcodes + m * (g.N / 2) + n / 2) = (u32x4){out[0], out[1], out[2], out[3]};
    } else {
        u32x4* d = reinterpret_cast<u32x4*>(g.qcodes + m * g.N + n);
        d[0] = (u32x4){out[0], out[1], out[2], out[3]};
        d[1] = (u32x4){out[4], out[5], out[6], out[7]};
    }
    g.qscales[m * (g.N / 32) + n / 32] = (uint8_t)s;
}

// Epilogue of big_tile<.., GATED>: acc[0] and acc[1] are g and u of TS rows x TS / 2 columns. Each of what
// is written is staged through LDS in fp32, so that stores are whole pieces of rows and a lane finds the 32
// columns of a group.
template <bool FP8, int OUT, int FQ, int TS>
__device__ __forceinline__ void gated_epilogue(const GemmArgs& g, v16f (&acc)[Big<FP8, TS>::WTN][Big<FP8, TS>::WTM],
                                               int64_t m0, int64_t n0, uint8_t* smem) {
    using C = Big<FP8, TS>;
    constexpr int COLS = TS / 2, EP = 4 * COLS + 16;  // staged row pitch
    static_assert(C::TM * EP <= C::NST * C::STAGE, "staging buffer exceeds the stage buffers");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int fr = lane & 31, fg = lane >> 5;
    auto stage = [&](auto value) {
        barrier_only();  // every wave is done with the stage buffers / the last pass
#pragma unroll
        for (int im = 0; im < C::WTM; ++im)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = wm * 32 * C::WTM + 32 * im + fr;
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = value(im, 4 * q + i);
                *reinterpret_cast<f32x4*>(smem + row * EP + 4 * (32 * wn + 8 * q + 4 * fg)) = v;
            }
        wait_lgkm0();
        barrier_only();
    };
    if (g.gu) {
        char* const gu = reinterpret_cast<char*>(g.gu);
        constexpr int ESZ = OUT == DT_F32 ? 4 : 2;
        stage([&](int im, int i) { return acc[0][im][i]; });
        store_staged<OUT, C::TM, COLS, C::NTH>(smem, EP, gu, g.ldgu, m0, n0, g.M, g.N);
        stage([&](int im, int i) { return acc[1][im][i]; });
        store_staged<OUT, C::TM, COLS, C::NTH>(smem, EP, gu + g.N * ESZ, g.ldgu, m0, n0, g.M, g.N);
    }
    stage([&](int im, int i) { return act_value(acc[0][im][i], g.act) * acc[1][im][i]; });
    if constexpr (FQ != FQ_NONE) {
        constexpr int GPR = COLS / 32;  // groups of a row, in consecutive lanes
#pragma unroll 1
        for (int t = tid; t < C::TM * GPR; t += C::NTH) {  // every lane in every sweep
            const int r = t / GPR, j = t % GPR;
            float v[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(smem + r * EP + 4 * (32 * j + 4 * c));
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * c + i] = x[i];
            }
            quantize_group(g, v, m0 + r, n0 + 32 * j);
        }
    }
    if (g.c) store_staged<OUT, C::TM, COLS, C::NTH>(smem, EP, reinterpret_cast<char*>(g.c), g.ldc, m0, n0, g.M, g.N);
    if (g.h32) store_staged<DT_F32, C::TM, COLS, C::NTH>(smem, EP, reinterpret_cast<char*>(g.h32), g.N, m0, n0, g.M, g.N);
}

template <bool FP8, bool B2D, int OUT, int FQ, int TS>
__global__ __launch_bounds__(TS == 256 ? 512 : 256, TS == 256 ? 1 : 2) void k_gated_tile(GemmArgs g) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int ntm = (int)((g.M + TS - 1) / TS), ntn = (int)((g.N + TS / 2 - 1) / (TS / 2));
    int tm, tn;
    big_tile_coords(blockIdx.x, ntm, ntn, tm, tn);
    big_tile<FP8, B2D, OUT, false, FQ, TS, true>(g, tm, tn, smem);
}

// ---------------------------------------------------------------------------------------------
// Few rows: 32 rows of A by 32 columns of h a workgroup of 8 waves. K is cut into units of 128 bytes of a row
// (256 E2M1 or 128 E4M3 values); wave w takes the units w, w + 8, .. and multiplies them with 32x32x64 scaled
// products whose operands come straight from memory, a lane's 16 bytes at a time (lane l: row l % 32, as in
// the tiles). Rows past the last are those of the last (their results are not stored); bytes past a row's end
// are zeros.
// ---------------------------------------------------------------------------------------------
constexpr int kRowsWaves = 8;

// the scale bytes 2 j + fg of a row's unit, j = 0 .. STEPS - 1, in byte 0 (even j) and 2 (odd j) of s[j / 2]
template <int STEPS>
__device__ __forceinline__ void unit_scales(const uint8_t* row, int64_t kgroups, int64_t g0, int fg, int (&s)[(STEPS + 1) / 2]) {
    if (!(kgroups & 3)) {
#pragma unroll
        for (int d = 0; d < STEPS / 2; ++d)
            s[d] = g0 + 4 * d < kgroups ? (int)(*reinterpret_cast<const uint32_t*>(row + g0 + 4 * d) >> (8 * fg)) : 0;
    } else {
#pragma unroll
        for (int d = 0; d < STEPS / 2; ++d) {
            const int64_t a = g0 + 4 * d + fg;
            s[d] = (a < kgroups ? row[a] : 0) | (a + 2 < kgroups ? (int)row[a + 2] << 16 : 0);
        }
    }
}

template <bool FP8>
struct RowsUnit {
    static constexpr int VALUES = FP8 ? 128 : 256, STEPS = VALUES / 64;
    u32x4 c[8 / 2];  // 64 bytes of the row: chunks 2 i + fg of the unit's eight
    int s[STEPS / 2];
};

template <bool FP8>
__device__ __forceinline__ void load_unit(RowsUnit<FP8>& u, const uint8_t* codes, const uint8_t* scales, int64_t row,
                                          int64_t srow, int64_t rowbytes, int64_t kgroups, int unit, int fg) {
    const int64_t b0 = (int64_t)unit * 128;
    const uint8_t* p = codes + row * rowbytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = b0 + 16 * (2 * i + fg);
        u.c[i] = at < rowbytes ? *reinterpret_cast<const u32x4*>(p + at) : (u32x4){0u, 0u, 0u, 0u};
    }
    unit_scales<RowsUnit<FP8>::STEPS>(scales + srow * kgroups, kgroups, (int64_t)unit * (RowsUnit<FP8>::VALUES / 32), fg, u.s);
}

template <bool FP8>
__device__ __forceinline__ v8i unit_frag(const RowsUnit<FP8>& u, int j) {
    if constexpr (FP8) {
        const u32x4 a = u.c[2 * j], b = u.c[2 * j + 1];
        return (v8i){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
    } else {
        const u32x4 a = u.c[j];
        return (v8i){(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    }
}

template <bool FP8>
__device__ __forceinline__ v16f unit_product(const RowsUnit<FP8>& w, const RowsUnit<FP8>& a, v16f acc) {
    constexpr int F = FP8 ? 0 : 4;
#pragma unroll
    for (int j = 0; j < RowsUnit<FP8>::STEPS; ++j) {
        if (j & 1) acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(unit_frag<FP8>(w, j), unit_frag<FP8>(a, j), acc, F, F, 2, w.s[j >> 1], 2, a.s[j >> 1]);
        else acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(unit_frag<FP8>(w, j), unit_frag<FP8>(a, j), acc, F, F, 0, w.s[j >> 1], 0, a.s[j >> 1]);
    }
    return acc;
}

template <bool FP8, bool B2D, int OUT, int FQ>
__global__ __launch_bounds__(64 * kRowsWaves) void k_gated_rows(GemmArgs g) {
    // shares of K: [wave][g or u][row of A][column]; then h [row][column] in the first of them
    __shared__ __attribute__((aligned(16))) float part[kRowsWaves][2][32][33];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 31, fg = lane >> 5;
    const int64_t rowbytes = FP8 ? g.K : g.K / 2, kgroups = g.K / 32;
    const int units = (int)((rowbytes + 127) / 128);
    const int64_t mt = (g.M + 31) / 32, tiles = mt * ((g.N + 31) / 32);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t n0 = t / mt * 32, m0 = t % mt * 32;
        const int64_t m = min(m0 + fr, g.M - 1), n = min(n0 + fr, g.N - 1), sn = B2D ? n >> 5 : n;
        v16f ag, au;
#pragma unroll
        for (int i = 0; i < 16; ++i) ag[i] = au[i] = 0.0f;
        for (int u = wave; u < units; u += kRowsWaves) {
            RowsUnit<FP8> wg, wu, a;
            load_unit<FP8>(wg, g.b, g.sb, n, sn, rowbytes, kgroups, u, fg);
            load_unit<FP8>(wu, g.b_up, g.sb_up, n, sn, rowbytes, kgroups, u, fg);
            load_unit<FP8>(a, g.a, g.sa, m, m, rowbytes, kgroups, u, fg);
            ag = unit_product<FP8>(wg, a, ag);
            au = unit_product<FP8>(wu, a, au);
        }
        // lane (fr, fg), register i: column 8 (i / 4) + 4 fg + i % 4 of row fr
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int c = 8 * (i >> 2) + 4 * fg + (i & 3);
            part[wave][0][fr][c] = ag[i];
            part[wave][1][fr][c] = au[i];
        }
        __syncthreads();
        float hv[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int at = tid + 512 * k, r = at >> 5, c = at & 31;
            float gv = part[0][0][r][c], uv = part[0][1][r][c];
#pragma unroll
            for (int w = 1; w < kRowsWaves; ++w) {
                gv += part[w][0][r][c];
                uv += part[w][1][r][c];
            }
            hv[k] = act_value(gv, g.act) * uv;
            const int64_t row = m0 + r, col = n0 + c;
            if (row < g.M && col < g.N) {
                if constexpr (OUT == DT_F32) {
                    if (g.gu) {
                        float* d = reinterpret_cast<float*>(g.gu) + row * g.ldgu + col;
                        d[0] = gv;
                        d[g.N] = uv;
                    }
                    if (g.c) reinterpret_cast<float*>(g.c)[row * g.ldc + col] = hv[k];
                } else {
                    if (g.gu) {
                        uint16_t* d = reinterpret_cast<uint16_t*>(g.gu) + row * g.ldgu + col;
                        d[0] = (uint16_t)pack_bf16x2_rne(gv, 0.0f);
                        d[g.N] = (uint16_t)pack_bf16x2_rne(uv, 0.0f);
                    }
                    if (g.c) reinterpret_cast<uint16_t*>(g.c)[row * g.ldc + col] = (uint16_t)pack_bf16x2_rne(hv[k], 0.0f);
                }
                if (g.h32) g.h32[row * g.N + col] = hv[k];
            }
        }
        if constexpr (FQ != FQ_NONE) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 2; ++k) part[0][0][(tid + 512 * k) >> 5][tid & 31] = hv[k];
            __syncthreads();
            if (wave == 0) {  // a lane a row; the upper lanes repeat the last one's places without storing
                float v[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = part[0][0][fr][c];
                quantize_group(g, v, lane < 32 ? m0 + lane : g.M, n0);
            }
        }
        __syncthreads();  // the next tile's shares overwrite what is read here
    }
}

// ---------------------------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------------------------
hipError_t plan_gated(int64_t M, int64_t F, int64_t K, bool fp8, const fp4_qparams* q, GatedPlan* p) {
    const int64_t rowb = fp8 ? K : K / 2;
    const bool direct = K % (fp8 ? 128 : 256) == 0 && M * rowb < (1ll << 31) && F * rowb < (1ll << 31);
    p->tile = 0;
    if (direct && M > 64 && ((M + 127) / 128) * ((F + 63) / 64) <= kMaxGrid) {
        int cus = 0;
        const hipError_t e = cu_count(&cus);
        if (e != hipSuccess) return e;
        const int64_t big = ((M + 255) / 256) * ((F + 127) / 128);
        p->tile = M < 256 || F < 128 || 2 * big <= cus ? 128 : 256;
    }
    // a rotation has to lie within a tile's columns
    p->quant_pass = q && (q->round_mode == FP4_ROUND_SR || q->hadamard_n > (p->tile ? p->tile / 2 : 32));
    p->ws = p->quant_pass ? M * F * 4 : 0;
    return hipSuccess;
}

template <bool FP8, bool B2D, int OUT, int FQ, int TS>
static hipError_t launch_tile(const GemmArgs& g, hipStream_t s) {
    using C = Big<FP8, TS>;
    const size_t lds = (size_t)C::NST * C::STAGE;
    const hipError_t e = allow_lds<k_gated_tile<FP8, B2D, OUT, FQ, TS>>(lds);
    if (e != hipSuccess) return e;
    const unsigned tiles = (unsigned)(((g.M + TS - 1) / TS) * ((g.N + TS / 2 - 1) / (TS / 2)));
    hipLaunchKernelGGL((k_gated_tile<FP8, B2D, OUT, FQ, TS>), dim3(tiles), dim3(C::NTH), lds, s, g);
    return hipGetLastError();
}

template <bool FP8, bool B2D, int OUT, int FQ>
static hipError_t launch_gated_k(const GemmArgs& g, int tile, hipStream_t s) {
    if (tile == 256) return launch_tile<FP8, B2D, OUT, FQ, 256>(g, s);
    if (tile == 128) return launch_tile<FP8, B2D, OUT, FQ, 128>(g, s);
    const int64_t tiles = ((g.N + 31) / 32) * ((g.M + 31) / 32);
    hipLaunchKernelGGL((k_gated_rows<FP8, B2D, OUT, FQ>), dim3((unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid)),
                       dim3(64 * kRowsWaves), 0, s, g);
    return hipGetLastError();
}

template <int OUT, int FQ>
static hipError_t launch_gated_q(const GemmArgs& g, int kind, int tile, hipStream_t s) {
    if (kind == 1) return launch_gated_k<true, false, OUT, FQ>(g, tile, s);
    return g.b_2d ? launch_gated_k<false, true, OUT, FQ>(g, tile, s) : launch_gated_k<false, false, OUT, FQ>(g, tile, s);
}

template <int OUT>
static hipError_t launch_gated_o(const GemmArgs& g, int kind, int tile, int fused_q, hipStream_t s) {
    return fused_q ? launch_gated_q<OUT, FQ_RNE>(g, kind, tile, s) : launch_gated_q<OUT, FQ_NONE>(g, kind, tile, s);
}

hipError_t launch_gated(GemmArgs g, const GatedPlan& p, int kind, int dtype, int fused_q, void* ws, hipStream_t s) {
    g.h32 = p.quant_pass ? reinterpret_cast<float*>(ws) : nullptr;
    const int fused = fused_q && !p.quant_pass;
    const hipError_t e = dtype == DT_BF16 ? launch_gated_o<DT_BF16>(g, kind, p.tile, fused, s) : launch_gated_o<DT_F32>(g, kind, p.tile, fused, s);
    if (e != hipSuccess || !p.quant_pass) return e;
    SegArgs a{};
    a.x = ws;
    a.rows = g.M;
    a.cols = a.ldx = g.N;
    a.nseg = g.M * (g.N / 32);
    a.codes = g.qcodes;
    a.scales = g.qscales;
    a.seed = g.q_seed;
    a.ceil_rule = g.q_ceil;
    return launch_segment(a, DT_F32, g.q_hn, g.q_elem, SC_E8M0, g.q_round, 1, 32, PASS_QUANT, s);
}

// ---------------------------------------------------------------------------------------------
// Backward: dgu = (dh u act'(g), dh act(g)), a piece of 8 columns of both a lane.
// ---------------------------------------------------------------------------------------------
template <int DT, int FQ>
__global__ __launch_bounds__(256) void k_gated_grad(GatedGradArgs a) {
    const int pieces = a.F >> 3;
    const int64_t total = a.rows * pieces;
    for (int64_t b0 = (int64_t)blockIdx.x * 256; b0 < total; b0 += (int64_t)gridDim.x * 256) {
        const int64_t i = b0 + threadIdx.x;
        const bool in = i < total;
        const int64_t row = i / pieces;
        const int col = 8 * (int)(i - row * pieces);
        float dh[8], g[8], u[8];
        if (in) {
            Piece<DT> p;
            piece_load<DT>(p, a.dh, row * a.lddh + col);
            piece_values<DT>(p, dh);
            piece_load<DT>(p, a.gu, row * a.ldgu + col);
            piece_values<DT>(p, g);
            piece_load<DT>(p, a.gu, row * a.ldgu + a.F + col);
            piece_values<DT>(p, u);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) dh[j] = g[j] = u[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v, d;
            act_slope(g[j], a.act, v, d);
            g[j] = dh[j] * u[j] * d;
            u[j] = dh[j] * v;
        }
        if (a.dgu && in) {
            piece_store<DT>(a.dgu, row * a.lddgu + col, piece_pack<DT>(g));
            piece_store<DT>(a.dgu, row * a.lddgu + a.F + col, piece_pack<DT>(u));
        }
        if constexpr (FQ != FQ_NONE) {
            constexpr int RND = FQ == FQ_SR ? RND_SR : RND_RNE;
            piece_quantize<RND>(a.q, g, row * 2 * a.F + col, in);
            piece_quantize<RND>(a.q, u, row * 2 * a.F + a.F + col, in);
        }
    }
}

template <int DT>
static hipError_t launch_gated_grad_k(const GatedGradArgs& a, int rnd, hipStream_t s) {
    const int64_t need = (a.rows * (a.F / 8) + 255) / 256;
    const unsigned grid = (unsigned)(need < kMaxGrid ? need : kMaxGrid);
    if (!a.q.codes) hipLaunchKernelGGL((k_gated_grad<DT, FQ_NONE>), dim3(grid), dim3(256), 0, s, a);
    else if (rnd == RND_SR) hipLaunchKernelGGL((k_gated_grad<DT, FQ_SR>), dim3(grid), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_gated_grad<DT, FQ_RNE>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int dtype, int rnd, hipStream_t s) {
    return dtype == DT_BF16 ? launch_gated_grad_k<DT_BF16>(a, rnd, s) : launch_gated_grad_k<DT_F32>(a, rnd, s);
}

}  // namespace bgf
