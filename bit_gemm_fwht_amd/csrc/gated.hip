// Gated feed-forward on block-scaled operands: h = act(A Wg^T) * (A Wu^T) in one launch, optionally with the
// two products kept (g | u) and h quantized along its columns; and its backward pass.
//
// Both products of a place are accumulated in the same lane's registers, so the activation and the product
// need no exchange and g and u never leave the chip unless they are asked for. Sums are fp32; of
// E4M3 products the matrix core itself keeps 13 bits below the largest of each 8 (g at K 4096 is off by 1.6e-5 of its root
// mean square, as in the GEMM; E2M1 products lose nothing). Three kernels:
//  - k_gated_tile: the pipelined GEMM tile (gemm_tile.h) on B slabs that hold 32 rows of Wg and the same 32
//    of Wu in turn: 256 x 128 or 128 x 64 results a workgroup;
//  - k_gated_stream: up to 64 rows of A, or parts of so many where tiles would leave CUs idle, K a multiple of 128:
//    bound by the weights' bytes;
//  - k_gated_rows: what neither takes (few rows of any K, operands past 2 GiB): 32 columns a workgroup, its waves
//    each multiply a share of K straight from memory, the shares are added through LDS in a fixed order.
#include "device.h"
#include "fp4_internal.h"
#include "gemm_tile.h"
#include "layer_internal.h"
#include "piece.h"

namespace bgf {

// Store a staged tile [ROWS][COLS] of dtype OUT (SRC: as it is staged, OUT or fp32; row pitch `pitch` bytes in LDS)
// at c[m0 ..][n0 ..], 16-byte pieces where the place allows; rows from M and columns from N on are not there. A
// thread keeps its piece of the columns and walks down the rows. NT: past the caches, which then keep the operands
// that other tiles read again: g and u always (they wait for the backward pass), h where it would not stay in them
// until it is read either. 4096 rows, K 4096, F 11008 in 4 bits with the next quantize of h: 320 us with nothing past
// the caches, 320 with g and u, 278 with all three; 2048 rows: 170, 138, 143.
template <int OUT, int SRC, int ROWS, int COLS, int NTH, bool NT = false>
__device__ __forceinline__ void store_staged(const uint8_t* lds, int pitch, char* c, int64_t ldc, int64_t m0, int64_t n0,
                                             int64_t M, int64_t N) {
    constexpr int ESZ = OUT == DT_F32 ? 4 : 2, EPC = 16 / ESZ, PPR = COLS / EPC;
    static_assert(NTH % PPR == 0, "whole rows a sweep");
    const bool vec_ok = ((reinterpret_cast<uintptr_t>(c) & 15) == 0) && ((ldc * ESZ) % 16 == 0);
    const int k = ((int)threadIdx.x % PPR) * EPC;
    const int64_t n = n0 + k;
#pragma unroll 4
    for (int r = threadIdx.x / PPR; r < ROWS; r += NTH / PPR) {
        const int64_t m = m0 + r;
        if (m >= M) break;
        const uint8_t* src = lds + r * pitch + k * (SRC == DT_F32 ? 4 : 2);
        u32x4 val;
        if constexpr (SRC == OUT) {
            val = *reinterpret_cast<const u32x4*>(src);
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4*>(src), b = *reinterpret_cast<const f32x4*>(src + 16);
            val = (u32x4){pack_bf16x2_rne(a[0], a[1]), pack_bf16x2_rne(a[2], a[3]), pack_bf16x2_rne(b[0], b[1]),
                          pack_bf16x2_rne(b[2], b[3])};
        }
        char* cp = c + (m * ldc + n) * ESZ;
        if (vec_ok && n + EPC <= N) {
            if constexpr (NT) __builtin_nontemporal_store(val, reinterpret_cast<u32x4*>(cp));
            else *reinterpret_cast<u32x4*>(cp) = val;
        } else {
#pragma unroll
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

// Epilogue of big_tile<.., GATED>: acc[0] and acc[1] are g and u of TS rows x TS / 2 columns. What is written is
// staged through LDS first, so that stores are whole pieces of rows and a lane finds the 32 columns of a group:
// g and u side by side in bf16, everything else a tile at a time, h in fp32 where it is quantized.
template <bool FP8, int OUT, int FQ, int TS, int NS>
__device__ __forceinline__ void gated_epilogue(const GemmArgs& g, v16f (&acc)[Big<FP8, TS>::WTN][Big<FP8, TS>::WTM],
                                               int64_t m0, int64_t n0, uint8_t* smem) {
    using C = Big<FP8, TS, NS>;
    constexpr int COLS = TS / 2, ESZ = OUT == DT_F32 ? 4 : 2;
    constexpr int EP = 4 * COLS + 16, HP = 2 * COLS + 16;  // row pitches: fp32, or g and u in bf16; h in bf16
    static_assert(C::TM * EP <= C::NST * C::STAGE, "staging buffer exceeds the stage buffers");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int fr = lane & 31, fg = lane >> 5;
    // four consecutive columns of a row at a time: put(row, column, the four values of acc's index)
    auto each = [&](auto put) {
        barrier_only();  // every wave is done with the stage buffers / the last pass
#pragma unroll
        for (int im = 0; im < C::WTM; ++im)
#pragma unroll
            for (int q = 0; q < 4; ++q) put(wm * 32 * C::WTM + 32 * im + fr, 32 * wn + 8 * q + 4 * fg, im, 4 * q);
        wait_lgkm0();
        barrier_only();
    };
    auto put_f32 = [&](int row, int col, f32x4 v) { *reinterpret_cast<f32x4*>(smem + row * EP + 4 * col) = v; };
    auto put_bf16 = [&](int pitch, int row, int col, f32x4 v) {
        *reinterpret_cast<u32x2*>(smem + row * pitch + 2 * col) = (u32x2){pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
    };
    auto four = [&](int p, int im, int i) { return (f32x4){acc[p][im][i], acc[p][im][i + 1], acc[p][im][i + 2], acc[p][im][i + 3]}; };
    auto h_of = [&](auto act, int im, int i) {
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = act_value<decltype(act)::value>(acc[0][im][i + k]) * acc[1][im][i + k];
        return v;
    };
    if (g.gu) {
        char* const gu = reinterpret_cast<char*>(g.gu);
        if constexpr (OUT == DT_BF16) {
            each([&](int row, int col, int im, int i) {
                put_bf16(EP, row, col, four(0, im, i));
                put_bf16(EP, row, COLS + col, four(1, im, i));
            });
            store_staged<OUT, OUT, C::TM, COLS, C::NTH, true>(smem, EP, gu, g.ldgu, m0, n0, g.M, g.N);
            store_staged<OUT, OUT, C::TM, COLS, C::NTH, true>(smem + 2 * COLS, EP, gu + g.N * ESZ, g.ldgu, m0, n0, g.M, g.N);
        } else {
            each([&](int row, int col, int im, int i) { put_f32(row, col, four(0, im, i)); });
            store_staged<OUT, OUT, C::TM, COLS, C::NTH, true>(smem, EP, gu, g.ldgu, m0, n0, g.M, g.N);
            each([&](int row, int col, int im, int i) { put_f32(row, col, four(1, im, i)); });
            store_staged<OUT, OUT, C::TM, COLS, C::NTH, true>(smem, EP, gu + g.N * ESZ, g.ldgu, m0, n0, g.M, g.N);
        }
    }
    char* const h = reinterpret_cast<char*>(g.c);
    if constexpr (FQ == FQ_NONE) {
        if (!h && !g.h32) return;
        if (OUT == DT_BF16 && !g.h32) {
            by_act(g.act, [&](auto act) { each([&](int row, int col, int im, int i) { put_bf16(HP, row, col, h_of(act, im, i)); }); });
            if (g.c_nt) store_staged<OUT, OUT, C::TM, COLS, C::NTH, true>(smem, HP, h, g.ldc, m0, n0, g.M, g.N);
            else store_staged<OUT, OUT, C::TM, COLS, C::NTH>(smem, HP, h, g.ldc, m0, n0, g.M, g.N);
            return;
        }
    }
    by_act(g.act, [&](auto act) { each([&](int row, int col, int im, int i) { put_f32(row, col, h_of(act, im, i)); }); });
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
    if (h) {
        if (g.c_nt) store_staged<OUT, DT_F32, C::TM, COLS, C::NTH, true>(smem, EP, h, g.ldc, m0, n0, g.M, g.N);
        else store_staged<OUT, DT_F32, C::TM, COLS, C::NTH>(smem, EP, h, g.ldc, m0, n0, g.M, g.N);
    }
    if (g.h32) store_staged<DT_F32, DT_F32, C::TM, COLS, C::NTH>(smem, EP, reinterpret_cast<char*>(g.h32), g.N, m0, n0, g.M, g.N);
}

// Tile coordinates of workgroup b: each of the 8 XCDs, which receive ids in turn, owns a run of tiles that follow one
// another, walked in groups of 4 tile rows, so that what an XCD's CUs read at once stays in its L2 (2048 rows, K 4096, F
// 11008: 128 us; groups of 2 138, of 16 139; without runs of their own where 8 does not divide the tiles 300 rows take
// 39.3 us for 36.8).
__device__ __forceinline__ void gated_tile_coords(int b, int ntm, int ntn, int& tm, int& tn) {
    constexpr int GM = 4;
    const int T = ntm * ntn, xcd = b % 8, each = T / 8, more = T % 8;
    b = xcd * each + min(xcd, more) + b / 8;
    const int grp = b / (GM * ntn), first = grp * GM;
    const int gs = min(ntm - first, GM);
    tm = first + (b % (GM * ntn)) % gs;
    tn = (b % (GM * ntn)) / gs;
}

template <bool FP8, bool B2D, int OUT, int FQ, int TS, int NS, bool RAG>
__global__ __launch_bounds__(TS == 256 ? 512 : 256, TS == 256 || NS > 2 ? 1 : 2) void k_gated_tile(GemmArgs g) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int ntm = (int)((g.M + TS - 1) / TS), ntn = (int)((g.N + TS / 2 - 1) / (TS / 2));
    int tm, tn;
    gated_tile_coords(blockIdx.x, ntm, ntn, tm, tn);
    big_tile<FP8, B2D, OUT, false, FQ, TS, true, NS, RAG>(g, tm, tn, smem);
}

// Store one place's values: gu, h, and h for a quantize pass of its own.
template <int OUT>
__device__ __forceinline__ void store_gated(const GemmArgs& g, int64_t row, int64_t col, float gv, float uv, float h) {
    if constexpr (OUT == DT_F32) {
        if (g.gu) {
            float* d = reinterpret_cast<float*>(g.gu) + row * g.ldgu + col;
            d[0] = gv;
            d[g.N] = uv;
        }
        if (g.c) reinterpret_cast<float*>(g.c)[row * g.ldc + col] = h;
    } else {
        if (g.gu) {
            uint16_t* d = reinterpret_cast<uint16_t*>(g.gu) + row * g.ldgu + col;
            d[0] = (uint16_t)pack_bf16x2_rne(gv, 0.0f);
            d[g.N] = (uint16_t)pack_bf16x2_rne(uv, 0.0f);
        }
        if (g.c) reinterpret_cast<uint16_t*>(g.c)[row * g.ldc + col] = (uint16_t)pack_bf16x2_rne(h, 0.0f);
    }
    if (g.h32) g.h32[row * g.N + col] = h;
}

// ---------------------------------------------------------------------------------------------
// Few rows, K a multiple of 128: bound by the weights' bytes. A workgroup of NW waves takes 16 NC columns of
// both projections and up to 16 MT rows of A; wave w takes the 128-byte units w, w + NW, .. of K by itself: it
// copies a unit's codes and scales straight into a ring of D buffers of its own in LDS (whole 128-byte runs of
// memory a row, many in flight, no registers and no barrier) and multiplies them with 16x16x128 scaled products
// (lane layouts in gemm.hip). The waves' shares of K are added through LDS in the order of the waves. Rows past
// M and F lie past the buffers' extents and read as zeros without touching memory.
// ---------------------------------------------------------------------------------------------
constexpr int kStreamWaves = 4;

template <bool FP8, int NC, int MT, int NW, int D>
struct Stream {
    static constexpr int WR = 16 * NC, AR = 16 * MT;      // rows of a projection, of A
    static constexpr int SPR = FP8 ? 4 : 8;               // scale bytes of a row's unit
    static constexpr int STEPS = FP8 ? 1 : 2;             // products of a unit
    static constexpr int WSZ = (WR * SPR + 255) / 256 * 256;
    static constexpr int OFF_U = WR * 128, OFF_A = 2 * WR * 128, OFF_SG = OFF_A + AR * 128, OFF_SU = OFF_SG + WSZ;
    static constexpr int OFF_SA = OFF_SU + WSZ, ASZ = (AR * SPR + 255) / 256 * 256;
    static constexpr int UNIT = OFF_SA + ASZ;             // bytes of a buffer
    static constexpr int COPIES = 4 * NC + 2 * MT + (2 * WSZ + ASZ) / 256;  // vector-memory instructions of a unit
    static constexpr int HP = WR + 4;                     // row pitch of the shares, in values
    static constexpr int SHARE = 2 * AR * HP;             // values of a wave's share: g, then u
    static constexpr int RING = NW * D * UNIT, SUM = 4 * NW * SHARE;
    static constexpr int LDS = RING > SUM ? RING : SUM;
    static_assert(LDS <= 160 * 1024, "LDS budget");
};

template <bool FP8, int OUT, int FQ, int NC, int MT, int NW, int D>
__global__ __launch_bounds__(64 * NW) void k_gated_stream(GemmArgs g) {
    using S = Stream<FP8, NC, MT, NW, D>;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, fq = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * S::WR, m0 = (int64_t)blockIdx.y * S::AR;
    const int rowbytes = (int)(FP8 ? g.K : g.K / 2), kgroups = (int)(g.K / 32);
    const int units = (rowbytes + 127) / 128, mine = (units - wave + NW - 1) / NW;
    uint8_t* const ring = smem + wave * D * S::UNIT;

    const int64_t srows = g.b_2d ? (g.N + 31) / 32 : g.N;
    auto resource = [](const void* p, int64_t bytes) { return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000); };
    const __amdgpu_buffer_rsrc_t rG = resource(g.b, g.N * rowbytes), rU = resource(g.b_up, g.N * rowbytes);
    const __amdgpu_buffer_rsrc_t rA = resource(g.a, g.M * rowbytes), rSA = resource(g.sa, g.M * kgroups);
    const __amdgpu_buffer_rsrc_t rSG = resource(g.sb, srows * kgroups), rSU = resource(g.sb_up, srows * kgroups);
    // extent 0: units past the last read nothing, so that every unit is the same number of copies
    const __amdgpu_buffer_rsrc_t rZ = resource(g.a, 0);
    // copy i of an operand fills its LDS rows r = 8 i + lane / 8, slot lane % 8 with chunk slot ^ swz(r)
    int voW[2 * NC], voA[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * NC; ++i) {
        const int r = 8 * i + (lane >> 3);
        voW[i] = (int)((n0 + r) * rowbytes + 16 * ((lane & 7) ^ chunk_swz(r)));
    }
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        const int r = 8 * i + (lane >> 3);
        voA[i] = (int)((m0 + r) * rowbytes + 16 * ((lane & 7) ^ chunk_swz(r)));
    }
    constexpr int DPR = S::SPR / 4;  // scale dwords of a row
    const int sp = lane % DPR;
    int voSW[S::WSZ / 256], voSA[S::ASZ / 256];
#pragma unroll
    for (int i = 0; i < S::WSZ / 256; ++i) {
        const int r = (64 * i + lane) / DPR;
        voSW[i] = r < S::WR ? (int)((g.b_2d ? (n0 + r) >> 5 : n0 + r) * kgroups + 4 * sp) : -1;
    }
#pragma unroll
    for (int i = 0; i < S::ASZ / 256; ++i) {
        const int r = (64 * i + lane) / DPR;
        voSA[i] = r < S::AR ? (int)((m0 + r) * kgroups + 4 * sp) : -1;
    }

    auto issue = [&](int i) {  // the wave's unit i
        uint8_t* const st = ring + (i % D) * S::UNIT;
        const int u = wave + NW * i;
        const bool real = i < mine;
        const int so = real ? u * 128 : 0, ss = real ? u * S::SPR : 0;
        // the second half of the last unit of an E2M1 row whose K is an odd multiple of 128 is not there
        const bool half = !FP8 && real && u * 128 + 64 >= rowbytes;
#pragma unroll
        for (int j = 0; j < 2 * NC; ++j) {
            const int vo = half && (((lane & 7) ^ chunk_swz(8 * j + (lane >> 3))) >= 4) ? -1 : voW[j];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(real ? rG : rZ, (lds_ptr_t)(st + 1024 * j), 16, vo, so, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(real ? rU : rZ, (lds_ptr_t)(st + S::OFF_U + 1024 * j), 16, vo, so, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j) {
            const int vo = half && (((lane & 7) ^ chunk_swz(8 * j + (lane >> 3))) >= 4) ? -1 : voA[j];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(real ? rA : rZ, (lds_ptr_t)(st + S::OFF_A + 1024 * j), 16, vo, so, 0, 0);
        }
        const bool gone = half && sp;
#pragma unroll
        for (int j = 0; j < S::WSZ / 256; ++j) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(real ? rSG : rZ, (lds_ptr_t)(st + S::OFF_SG + 256 * j), 4, gone ? -1 : voSW[j], ss, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(real ? rSU : rZ, (lds_ptr_t)(st + S::OFF_SU + 256 * j), 4, gone ? -1 : voSW[j], ss, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < S::ASZ / 256; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(real ? rSA : rZ, (lds_ptr_t)(st + S::OFF_SA + 256 * j), 4, gone ? -1 : voSA[j], ss, 0, 0);
    };
    const int swz = chunk_swz(fr);
    auto frag = [&](const uint8_t* rows, int t, int j) -> v8i {  // rows 16 t + fr: (16 t + fr) swizzles like fr
        const uint8_t* const p = rows + (16 * t + fr) * 128;
        const u32x4 a = *reinterpret_cast<const u32x4*>(p + 16 * ((4 * j + fq) ^ swz));
        if constexpr (FP8) {
            const u32x4 b = *reinterpret_cast<const u32x4*>(p + 16 * ((4 + fq) ^ swz));
            return (v8i){(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
        } else {
            return (v8i){(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
        }
    };
    auto scale = [&](const uint8_t* s, int t, int j) {
        return (int)(*reinterpret_cast<const uint32_t*>(s + (16 * t + fr) * S::SPR + 4 * j) >> (8 * fq));
    };

    f32x4 acc[2][NC][MT];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[p][c][m] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i);
    for (int i = 0; i < mine; ++i) {
        issue(i + D - 1);                  // into the buffer that was read last
        wait_vm<(D - 1) * S::COPIES>();    // this wave's copies of unit i have landed
        asm volatile("" ::: "memory");
        const uint8_t* const st = ring + (i % D) * S::UNIT;
#pragma unroll
        for (int j = 0; j < S::STEPS; ++j) {
            v8i fa[MT];
            int sa[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                fa[m] = frag(st + S::OFF_A, m, j);
                sa[m] = scale(st + S::OFF_SA, m, j);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const v8i fw = frag(st + p * S::OFF_U, c, j);
                    const int sw = scale(st + (p ? S::OFF_SU : S::OFF_SG), c, j);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[p][c][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa[m], acc[p][c][m], FP8 ? 0 : 4,
                                                                                       FP8 ? 0 : 4, 0, sw, 0, sa[m]);
                }
        }
        wait_lgkm0();  // the buffer has been read
    }
    wait_vm<0>();  // the last copies (of nothing) have landed: the ring is free
    __syncthreads();
    // the shares: lane (fr, fq) holds columns 16 c + 4 fq + i of row 16 m + fr
    float* const part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                *reinterpret_cast<f32x4*>(part + wave * S::SHARE + (p * S::AR + 16 * m + fr) * S::HP + 16 * c + 4 * fq) = acc[p][c][m];
    __syncthreads();
    const int rows = (int)min((int64_t)S::AR, g.M - m0);
    by_act(g.act, [&](auto act) {
        for (int i = tid; i < rows * S::WR; i += 64 * NW) {
            const int r = i / S::WR, c = i % S::WR;
            float gv = part[r * S::HP + c], uv = part[(S::AR + r) * S::HP + c];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                gv += part[w * S::SHARE + r * S::HP + c];
                uv += part[w * S::SHARE + (S::AR + r) * S::HP + c];
            }
            const float h = act_value<decltype(act)::value>(gv) * uv;
            const int64_t row = m0 + r, col = n0 + c;
            if (col < g.N) store_gated<OUT>(g, row, col, gv, uv, h);
            if constexpr (FQ != FQ_NONE) part[r * S::HP + c] = h;  // read by this thread alone until now
        }
    });
    if constexpr (FQ != FQ_NONE) {
        static_assert(NC == 2 && MT <= 4, "a group of 32 columns, a lane a row");
        __syncthreads();
        if (wave == 0) {
            float v[32];
            const int r = min(lane, S::AR - 1);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(part + r * S::HP + 4 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * c + i] = x[i];
            }
            quantize_group(g, v, lane < rows ? m0 + lane : g.M, n0);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Any shape: 32 rows of A by 32 columns of h a workgroup of 8 waves. K is cut into units of 128 bytes of a row
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
            by_act(g.act, [&](auto act) { hv[k] = act_value<decltype(act)::value>(gv) * uv; });
            const int64_t row = m0 + r, col = n0 + c;
            if (row < g.M && col < g.N) store_gated<OUT>(g, row, col, gv, uv, hv[k]);
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
// Workgroups of 16 columns that k_gated_stream would have: rows of A in equal parts of at most 64.
static int64_t stream_parts(int64_t M) { return (M + 63) / 64; }
static int64_t stream_groups(int64_t M, int64_t F) { return stream_parts(M) * ((F + 15) / 16); }

// Which kernel, by the rows of A and the tiles that they give (times: F 11008, K 4096, 4 bits, bf16 h):
//  - up to 64 rows: k_gated_stream (64 rows 15.9 us, tiles 15.3 at 65; 8 bits 33 and 37);
//  - with more it reads the weights again for each 64 rows, but its waves share K, and few tiles are bound by how
//    long one takes for K: up to 2 3/4 workgroups of 16 columns a CU (F 1376: 128 rows 7.6 us, tiles 14.8; 512 rows
//    15.2 and 16.5, 1024 rows 24.8 and 16.9), 2 in 8 bits (F 1376: 256 rows 14.8 us and 23.8; 512 rows 25.2 and 23.9)
//    and where it codes h, which takes 32 columns a workgroup, and 1 where it alone would need a pass to code h;
//  - tiles of 256 rows from 256 rows on, where they fill more than half the CUs (300 rows 36.8 us, tiles of 128 rows
//    42; 4096 rows 242 and 398), else tiles of 128 rows;
//  - of those four stages deep where each tile has a CU to itself (65 rows 15.3 us, two stages and two workgroups a
//    CU 19.0; 200 rows, where it has not, 28.7 and 25.0);
//  - K off the multiples of 128: tiles of 128 rows with scales through registers, up to 32 rows k_gated_rows (K
//    2080: 64 rows 20.3 us, tiles 16.3);
//  - operands of 2 GiB and more, whose places leave 32 bits: k_gated_rows.
hipError_t plan_gated(int64_t M, int64_t F, int64_t K, bool fp8, const fp4_qparams* q, GatedPlan* p) {
    const int64_t rowb = fp8 ? K : K / 2;
    const bool direct = M * rowb < (1ll << 31) && F * rowb < (1ll << 31);
    int columns = 32;  // of a tile: a rotation has to lie within them
    p->kernel = GATED_ROWS;
    if (direct && K % 128 == 0 && M <= 64) {
        p->kernel = GATED_STREAM;
    } else if (direct && M > (K % 128 ? 32 : 64) && ((M + 127) / 128) * ((F + 63) / 64) <= kMaxGrid) {
        int cus = 0;
        const hipError_t e = cu_count(&cus);
        if (e != hipSuccess) return e;
        const int64_t big = ((M + 255) / 256) * ((F + 127) / 128);
        const bool mid = M < 256 || F < 128 || 2 * big <= cus;
        const bool deep = ((M + 127) / 128) * ((F + 63) / 64) <= cus;
        const bool nearest = q && q->round_mode != FP4_ROUND_SR;
        const bool alone = nearest && q->hadamard_n == 64, codes = nearest && q->hadamard_n <= 32;
        const int quarters = alone ? 4 : fp8 || codes ? 8 : 11;
        if (K % 128 == 0 && 4 * stream_groups(M, F) <= quarters * cus) {
            p->kernel = GATED_STREAM;
        } else {
            p->kernel = K % 128 ? GATED_TILE128_RAGGED : !mid ? GATED_TILE256 : deep ? GATED_TILE128_DEEP : GATED_TILE128;
            columns = p->kernel == GATED_TILE256 ? 128 : 64;
        }
    }
    p->quant_pass = q && (q->round_mode == FP4_ROUND_SR || q->hadamard_n > columns);
    p->ws = p->quant_pass ? M * F * 4 : 0;
    return hipSuccess;
}

template <bool FP8, int OUT, int FQ, int NC, int MT, int D>
static hipError_t launch_stream(const GemmArgs& g, hipStream_t s) {
    using S = Stream<FP8, NC, MT, kStreamWaves, D>;
    const hipError_t e = allow_lds<k_gated_stream<FP8, OUT, FQ, NC, MT, kStreamWaves, D>>(S::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_gated_stream<FP8, OUT, FQ, NC, MT, kStreamWaves, D>), dim3((unsigned)((g.N + S::WR - 1) / S::WR), (unsigned)stream_parts(g.M)),
                       dim3(64 * kStreamWaves), S::LDS, s, g);
    return hipGetLastError();
}

template <bool FP8, int OUT, int FQ, int NC, int MT>
static hipError_t launch_stream_d(const GemmArgs& g, int cus, hipStream_t s) {
    // two buffers where a wave has eight units or more to go through (one row, 8 bits, K 4096: 23.3 us against 24.5;
    // 4 bits, K 8192: 18.7 against 19.3), else one, which leaves room for more workgroups (4 bits, K 4096: 9.9
    // against 10.2). With more than 32 rows two buffers leave room for one workgroup a CU alone: only where there are
    // no more than that (48 rows, 4 bits, K 8192, F 11008: 31.0 us with one, 33.6 with two), and then for any K (128
    // rows, K 4096, F 1376: 7.6 against 8.7)
    const bool alone = stream_parts(g.M) * ((g.N + 16 * NC - 1) / (16 * NC)) <= cus;
    const bool deep = alone || (MT <= 2 && (FP8 ? g.K / 128 : g.K / 256) >= 8 * kStreamWaves);
    return deep ? launch_stream<FP8, OUT, FQ, NC, MT, 2>(g, s) : launch_stream<FP8, OUT, FQ, NC, MT, 1>(g, s);
}

// Whether 48 columns a workgroup are faster than 16 for 33 to 64 rows of A in 8 bits, where A's rows are most of a unit
// and one such workgroup fills a CU: only where their number fills the rounds that it takes, and K is long enough for
// their bare start and end (64 rows, us of 48 and of 16 columns; 256 CUs). One round from 3/4 full: K 4096, F 9216 22.4
// and 24.2, F 11008 29.6 and 32.6, K 8192, F 9216 52.5 and 67.7; F 12320, a second round for one workgroup, 50.2 and
// 42.5. Several from 7/8 full: K 4096, F 21504 62.0 and 66.1, F 24576 62.9 and 69.4; F 14336, 0.58 full, 56.6 and 45.7,
// F 28672, 0.78, 87.2 and 80.4. K from 8192 on from 3/4 full: F 28672 151.5 and 161.0; F 16384, 0.67, 99.7 and 92.7. K
// 2048: F 12288 16.3 and 14.1, F 24576 35.6 and 31.6.
static bool columns48(const GemmArgs& g, int cus) {
    const int64_t groups = (g.N + 47) / 48, places = (groups + cus - 1) / cus * cus;
    const int eighths = places == cus || g.K >= 8192 ? 6 : 7;
    return g.M > 32 && g.M <= 64 && g.K >= 4096 && 8 * groups >= eighths * places;
}

template <bool FP8, int OUT, int FQ>
static hipError_t launch_stream_m(const GemmArgs& g, hipStream_t s) {
    // 16 columns a workgroup, so that several fit a CU and all are resident at once; 32 where groups of 32 are
    // quantized; 48 in 8 bits by columns48; 32, two buffers deep, where that makes no more workgroups than CUs of what
    // would be up to twice as many, and a wave has two units (256 rows, K 4096, F 1376: 10.7 us against 11.8, 8 bits
    // 14.8 against 18.2; 64 rows of F 5504 10.4 and 11.5, 15.2 and 18.0; K 256, 512 rows of F 1024: 5.5 against 4.4)
    constexpr int NC = FQ != FQ_NONE ? 2 : 1;
    const int64_t rows = (g.M + stream_parts(g.M) - 1) / stream_parts(g.M);
    int cus = 0;
    const hipError_t e = cu_count(&cus);
    if (e != hipSuccess) return e;
    if constexpr (FP8 && FQ == FQ_NONE) {
        if (columns48(g, cus))
            return g.M <= 48 ? launch_stream<FP8, OUT, FQ, 3, 3, 2>(g, s) : launch_stream<FP8, OUT, FQ, 3, 4, 1>(g, s);
    }
    if constexpr (FQ == FQ_NONE) {
        const int64_t groups = stream_groups(g.M, g.N);
        if (rows > 32 && groups > cus && groups <= 2 * cus && (FP8 ? g.K / 128 : g.K / 256) >= 2 * kStreamWaves)
            return rows <= 48 ? launch_stream_d<FP8, OUT, FQ, 2, 3>(g, cus, s) : launch_stream_d<FP8, OUT, FQ, 2, 4>(g, cus, s);
    }
    if (rows <= 16) return launch_stream_d<FP8, OUT, FQ, NC, 1>(g, cus, s);
    if (rows <= 32) return launch_stream_d<FP8, OUT, FQ, NC, 2>(g, cus, s);
    if (rows <= 48) return launch_stream_d<FP8, OUT, FQ, NC, 3>(g, cus, s);
    return launch_stream_d<FP8, OUT, FQ, NC, 4>(g, cus, s);
}

template <bool FP8, bool B2D, int OUT, int FQ, int TS, int NS, bool RAG = false>
static hipError_t launch_tile(const GemmArgs& g, hipStream_t s) {
    using C = Big<FP8, TS, NS>;
    const size_t lds = (size_t)C::NST * C::STAGE;
    const hipError_t e = allow_lds<k_gated_tile<FP8, B2D, OUT, FQ, TS, NS, RAG>>(lds);
    if (e != hipSuccess) return e;
    const unsigned tiles = (unsigned)(((g.M + TS - 1) / TS) * ((g.N + TS / 2 - 1) / (TS / 2)));
    hipLaunchKernelGGL((k_gated_tile<FP8, B2D, OUT, FQ, TS, NS, RAG>), dim3(tiles), dim3(C::NTH), lds, s, g);
    return hipGetLastError();
}

template <bool FP8, bool B2D, int OUT, int FQ>
static hipError_t launch_gated_k(const GemmArgs& g, int kernel, hipStream_t s) {
    if (kernel == GATED_TILE256) return launch_tile<FP8, B2D, OUT, FQ, 256, 2>(g, s);
    if (kernel == GATED_TILE128) return launch_tile<FP8, B2D, OUT, FQ, 128, 2>(g, s);
    if (kernel == GATED_TILE128_RAGGED) return launch_tile<FP8, B2D, OUT, FQ, 128, 2, true>(g, s);
    if (kernel == GATED_TILE128_DEEP) return launch_tile<FP8, B2D, OUT, FQ, 128, 4>(g, s);
    if (kernel == GATED_STREAM) return launch_stream_m<FP8, OUT, FQ>(g, s);
    const int64_t tiles = ((g.N + 31) / 32) * ((g.M + 31) / 32);
    hipLaunchKernelGGL((k_gated_rows<FP8, B2D, OUT, FQ>), dim3((unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid)),
                       dim3(64 * kRowsWaves), 0, s, g);
    return hipGetLastError();
}

template <int OUT, int FQ>
static hipError_t launch_gated_q(const GemmArgs& g, int kind, int kernel, hipStream_t s) {
    if (kind == 1) return launch_gated_k<true, false, OUT, FQ>(g, kernel, s);
    return g.b_2d ? launch_gated_k<false, true, OUT, FQ>(g, kernel, s) : launch_gated_k<false, false, OUT, FQ>(g, kernel, s);
}

template <int OUT>
static hipError_t launch_gated_o(const GemmArgs& g, int kind, int kernel, int fused_q, hipStream_t s) {
    return fused_q ? launch_gated_q<OUT, FQ_RNE>(g, kind, kernel, s) : launch_gated_q<OUT, FQ_NONE>(g, kind, kernel, s);
}

hipError_t launch_gated(GemmArgs g, const GatedPlan& p, int kind, int dtype, int fused_q, void* ws, hipStream_t s) {
    g.h32 = p.quant_pass ? reinterpret_cast<float*>(ws) : nullptr;
    g.c_nt = g.M * g.N * (dtype == DT_BF16 ? 2 : 4) >= (int64_t(64) << 20);
    const int fused = fused_q && !p.quant_pass;
    const hipError_t e = dtype == DT_BF16 ? launch_gated_o<DT_BF16>(g, kind, p.kernel, fused, s) : launch_gated_o<DT_F32>(g, kind, p.kernel, fused, s);
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
// Backward: dgu = (dh u act'(g), dh act(g)), a piece of 8 columns of both a lane; bound by memory. NT (bf16): what
// is read and dgu go past the caches, where the call is larger than what they keep (4096 rows, F 11008: 93.5 us
// against 99.4; 1024 rows 27.1 against 27.7, but then dgu is still there for the calls that read it next).
// ---------------------------------------------------------------------------------------------
template <int DT, int FQ, bool NT>
__global__ __launch_bounds__(256) void k_gated_grad(GatedGradArgs a) {
    const int pieces = a.F >> 3;
    const int64_t total = a.rows * pieces;
    for (int64_t b0 = (int64_t)blockIdx.x * 256; b0 < total; b0 += (int64_t)gridDim.x * 256) {
        const bool in = b0 + threadIdx.x < total;
        // one 64-bit division a wave, a 32-bit one a lane
        const int64_t row0 = b0 / pieces;
        const uint32_t i = (uint32_t)(b0 - row0 * pieces) + threadIdx.x, down = i / (uint32_t)pieces;
        const int64_t row = row0 + down;
        const int col = 8 * (int)(i - down * (uint32_t)pieces);
        float dh[8], g[8], u[8];
        if (in) {
            Piece<DT> p, q, r;
            piece_load<DT, NT>(p, a.dh, row * a.lddh + col);
            piece_load<DT, NT>(q, a.gu, row * a.ldgu + col);
            piece_load<DT, NT>(r, a.gu, row * a.ldgu + a.F + col);
            piece_values<DT>(p, dh);
            piece_values<DT>(q, g);
            piece_values<DT>(r, u);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) dh[j] = g[j] = u[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v, d;
            // (chosen for each value: for all eight at once the loads are waited for together, 97.6 -> 103.0 us)
            by_act(a.act, [&](auto act) { act_slope<decltype(act)::value>(g[j], v, d); });
            g[j] = dh[j] * u[j] * d;
            u[j] = dh[j] * v;
        }
        if (a.dgu && in) {
            piece_store<DT, NT>(a.dgu, row * a.lddgu + col, piece_pack<DT>(g));
            piece_store<DT, NT>(a.dgu, row * a.lddgu + a.F + col, piece_pack<DT>(u));
        }
        if constexpr (FQ != FQ_NONE) {
            constexpr int RND = FQ == FQ_SR ? RND_SR : RND_RNE;
            piece_quantize<RND>(a.q, g, row * 2 * a.F + col, in);
            piece_quantize<RND>(a.q, u, row * 2 * a.F + a.F + col, in);
        }
    }
}

template <int DT, bool NT>
static hipError_t launch_gated_grad_k(const GatedGradArgs& a, int rnd, hipStream_t s) {
    const int64_t need = (a.rows * (a.F / 8) + 255) / 256;
    const unsigned grid = (unsigned)(need < kMaxGrid ? need : kMaxGrid);
    if (!a.q.codes) hipLaunchKernelGGL((k_gated_grad<DT, FQ_NONE, NT>), dim3(grid), dim3(256), 0, s, a);
    else if (rnd == RND_SR) hipLaunchKernelGGL((k_gated_grad<DT, FQ_SR, NT>), dim3(grid), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_gated_grad<DT, FQ_RNE, NT>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int dtype, int rnd, hipStream_t s) {
    if (dtype == DT_F32) return launch_gated_grad_k<DT_F32, false>(a, rnd, s);
    return a.rows * a.F * 6 >= (int64_t(96) << 20) ? launch_gated_grad_k<DT_BF16, true>(a, rnd, s) : launch_gated_grad_k<DT_BF16, false>(a, rnd, s);
}

}  // namespace bgf
