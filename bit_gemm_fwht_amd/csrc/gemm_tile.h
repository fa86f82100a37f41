// The pipelined tile of the block-scaled GEMM (256 x 256 or 128 x 128 results a workgroup, operands copied
// straight into LDS, scaled matrix instructions) with its epilogue, shared by the GEMM kernels and the gated
// feed-forward.
#pragma once

#include "device.h"
#include "fp4_internal.h"
#include "launch.h"
#include "quant_block.h"

namespace bgf {

typedef int v8i __attribute__((ext_vector_type(8)));

// FQ: fused output quantize, 0 none, FQ_RNE or FQ_SR (a template argument, so that the nearest-even
// variant carries no stochastic-rounding registers)
constexpr int FQ_NONE = 0, FQ_RNE = 1, FQ_SR = 2;

// ---------------------------------------------------------------------------------------------
// Large-tile pipelined kernel: 256 x 256 workgroup tile, 8 waves (two per SIMD, so one wave's
// waits are covered by the other's matrix work), each wave a 128 x 64 quadrant of 4 x 2 tiles of
// the 32x32x64 scaled MFMA (lane l: row l % 32, 32 K values of group l / 32 of the instruction's
// 64; result lane l, register i: D[8 (i / 4) + 4 (l / 32) + i % 4][l % 32]).
// A multi-stage LDS ring is filled by direct global->LDS 128-bit loads (no VGPR staging): each
// wave writes 1 KB contiguous blocks, so a row's 16-byte chunks are placed by choosing which
// chunk each lane fetches. The chunk slot is XOR-swizzled with bits of the row so that the
// 16-byte fragment reads of consecutive rows hit distinct LDS banks (for 32 and 64 banks).
// Scales: one dword (4 K groups) per row per 128-deep step, shifted per lane so that a fixed
// OPSEL byte selects the lane's group.
// Workgroups are renumbered so that each of the 8 XCDs (which receive workgroup ids round-robin)
// owns a contiguous run of tiles, walked in groups of 4 tile rows for L2 reuse.
// ---------------------------------------------------------------------------------------------
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// TS = 256: 8 waves of 128 x 64 (one workgroup per CU: two 68 KB stages); TS = 128: 4 waves of
// 64 x 64 (two workgroups per CU: two 34 KB stages each), for grids of 256 x 256 tiles that would
// leave most CUs idle. NS stages: with 4 of them three are on their way while one is multiplied (TS = 128, one
// workgroup per CU), for grids of so few tiles that each has a CU to itself.
template <bool FP8, int TS = 256, int NS = 2>
struct Big {
    static constexpr int TM = TS, TN = TS, NW = TS == 256 ? 8 : 4, NTH = 64 * NW;
    static constexpr int WTM = TS == 256 ? 4 : 2, WTN = 2;  // 32x32 tiles per wave (M x N)
    static constexpr int WN = TN / (32 * WTN);        // waves along N
    // One stage covers 128 bytes of every row (full 128-byte cache lines): 256 K values of FP4
    // or 128 of FP8.
    static constexpr int KSTEP = FP8 ? 128 : 256;
    static constexpr int RB = 128;                    // bytes per row per stage
    static constexpr int CPR = RB / 16;               // 16-byte chunks per row
    static constexpr int NKK = KSTEP / 64;            // 64-deep MFMA steps per stage
    static constexpr int SPR = KSTEP / 32;            // scale bytes per row per stage
    static constexpr int NST = NS;                    // pipeline stages
    static constexpr int OPB = TM * RB;               // operand bytes per stage
    static constexpr int SB = TM * SPR;               // scale bytes per operand per stage
    // stage layout: A's scales, B's scales, A's codes, B's codes (scales first, so that the
    // scale reads of a stage reach every tile with one base register and 16-bit offsets)
    static constexpr int OFF_SB = SB, OFF_A = 2 * SB, OFF_B = 2 * SB + OPB;
    static constexpr int STAGE = 2 * OPB + 2 * SB;
    static constexpr int IPW = OPB / 1024 / NW;       // 1 KB code loads per wave per operand
    static constexpr int SPW = 2 * SB / 256 / NW;     // 256 B scale loads per wave (both operands)
    static constexpr int LOADS = 2 * IPW + SPW;       // vector-memory instructions per thread per stage
};

// 16-byte chunk slot of chunk c in row r: c ^ swz(r), distinct over any 8 consecutive rows and over
// any 8 rows of equal parity (conflict-free 16-byte fragment reads for 32 or 64 LDS banks)
__device__ __forceinline__ int chunk_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }


// s_waitcnt with vmcnt = N (gfx9 encoding: vmcnt bits [3:0] and [15:14]); expcnt and lgkmcnt at
// their maximum, i.e. not waited for
template <int N>
__device__ __forceinline__ void wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Workgroup barrier without the memory fence of __syncthreads (which waits for every outstanding
// vector-memory operation, including the next stage's prefetch). The empty asm statements keep
// the compiler from moving LDS or memory accesses across it; the caller waits for what must have
// completed.
__device__ __forceinline__ void barrier_only() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// s_waitcnt lgkmcnt(0): this wave's LDS reads and writes have completed
__device__ __forceinline__ void wait_lgkm0() {
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));
}

// ---------------------------------------------------------------------------------------------
// NVFP4 -> MXFP8 re-expression of one 32-wide K group of a row: q holds its 32 E2M1 codes (element
// k in nibble k % 8 of word k / 8), s01 its two E4M3 block scales (byte 0: elements 0-15). With S
// the larger block scale, E is the smallest exponent with 448 * 2^E >= 6 S, and every element
// becomes E4M3(val(q) * s_blk * 2^-E): val(q) * s_blk is exact in fp32 and the scaled convert
// divides it by 2^E exactly before rounding to nearest even. o: 32 E4M3 bytes in element order.
// Returns the E8M0 code E + 127 (E = -127 for S = 0, every element then 0).
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t nv_group_to_fp8(const u32x4 q, uint32_t s01, uint32_t (&o)[8]) {
    const float s0 = e4m3_value(s01 & 0x7Fu), s1 = e4m3_value((s01 >> 8) & 0x7Fu);
    const float S = fmaxf(s0, s1);
    // E = smallest exponent with 448 * 2^E >= 6 S (6 S is exact in fp32)
    const int E = e8m0_exp<8, 0x600000u>(6.0f * S, true);
    const float sc = E > -127 ? pow2f(E) : 1.0f;  // S = 0: every product is 0
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float sb = w < 2 ? s0 : s1;
        const v2f p0 = fp4x2_to_f32<0>(q[w]), p1 = fp4x2_to_f32<1>(q[w]);
        const v2f p2 = fp4x2_to_f32<2>(q[w]), p3 = fp4x2_to_f32<3>(q[w]);
        uint32_t r0 = 0u, r1 = 0u;
        r0 = cvt_fp8x2<false>(r0, p0[0] * sb, p0[1] * sb, sc);
        r0 = cvt_fp8x2<true>(r0, p1[0] * sb, p1[1] * sb, sc);
        r1 = cvt_fp8x2<false>(r1, p2[0] * sb, p2[1] * sb, sc);
        r1 = cvt_fp8x2<true>(r1, p3[0] * sb, p3[1] * sb, sc);
        o[2 * w] = r0;
        o[2 * w + 1] = r1;
    }
    return (uint32_t)(E + 127);
}

// Tile coordinates of work item b (a workgroup index of the one-tile-per-workgroup launch): the
// workgroups of each of the 8 XCDs (which receive ids round-robin) own a contiguous run of tiles,
// walked in groups of 4 tile rows for L2 reuse.
__device__ __forceinline__ void big_tile_coords(int b, int ntm, int ntn, int& tm, int& tn) {
    const int T = ntm * ntn;
    if (T % 8 == 0) b = (b % 8) * (T / 8) + b / 8;
    const int GM = 4;
    const int grp = b / (GM * ntn), first = grp * GM;
    const int gs = (ntm - first) < GM ? (ntm - first) : GM;
    tm = first + (b % (GM * ntn)) % gs;
    tn = (b % (GM * ntn)) / gs;
}

// Epilogue of a TS x TS tile: the accumulators (lane layout of the 32x32x64 MFMA tiles of
// big_tile) to C, and to C_q when FQ; uses the first TS * 528 bytes of `smem`, which
// must be free (no copy into it still in flight). Every thread of the workgroup must call it.
template <bool FP8, int OUT, bool NVG, int FQ, int TS = 256>
__device__ __forceinline__ void big_epilogue(const GemmArgs& g, v16f (&acc)[Big<FP8, TS>::WTN][Big<FP8, TS>::WTM],
                                             int64_t m0, int64_t n0, uint8_t* smem) {
    using C = Big<FP8, TS>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int fr = lane & 31, fg = lane >> 5;
    // Epilogue, staged through LDS so that every global store writes whole 16-byte pieces of a
    // row and consecutive lanes cover consecutive bytes. Lane (fr, fg) holds, for 4-register group
    // q of tile (im, in), C[m][n .. n+3] with m = wm*128 + 32 im + fr and
    // n = wn*64 + 32 in + 8 q + 4 fg. A pass stages 256 rows x 512 bytes: bf16 output in one pass
    // (all 256 columns), fp32 output in two (pass p holds columns wn*64 + 32 p + [0, 32) of each
    // wave column wn, i.e. four 128-byte runs per row).
    constexpr int EP = 528;                       // staged row pitch (512 B + 16 B of padding)
    static_assert(TS == 128 || 256 * EP <= C::NST * C::STAGE, "staging buffer exceeds the stage buffers");
    constexpr int PASSES = OUT == DT_F32 ? 2 : 1;
    float gscale = 1.0f;
    if constexpr (NVG) gscale = (*g.ga) * (*g.gb);
    // an opaque zero keeps the compiler from computing the output addresses before the main
    // loop, where they would only add register pressure
    int opaque_zero;
    asm volatile("s_mov_b32 %0, 0" : "=s"(opaque_zero));
    const int64_t me0 = m0 + opaque_zero, ne0 = n0 + opaque_zero, ldc = g.ldc + opaque_zero;
    char* const cbase = reinterpret_cast<char*>(g.c) + opaque_zero;
    const int64_t Mx = g.M + opaque_zero, Nx = g.N + opaque_zero;
    if constexpr (TS == 128 && FQ == FQ_NONE) {
        // 128 x 128 tile, plain output: one pass stages all 128 rows (128 fp32 or bf16 values per
        // row), then each row goes out as 16 (bf16) or 32 (fp32) 16-byte pieces
        static_assert(128 * EP <= C::NST * C::STAGE, "staging buffer exceeds the stage buffers");
        constexpr int ESZ = OUT == DT_F32 ? 4 : 2;
        const bool vec_ok = ((reinterpret_cast<uintptr_t>(g.c) & 15) == 0) && ((ldc * ESZ) % 16 == 0);
        barrier_only();  // every wave is done reading the stage buffers
#pragma unroll
        for (int im = 0; im < C::WTM; ++im)
#pragma unroll
            for (int in = 0; in < C::WTN; ++in) {
                const int row = wm * 32 * C::WTM + 32 * im + fr;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = NVG ? acc[in][im][4 * q + i] * gscale : acc[in][im][4 * q + i];
                    const int col = wn * 32 * C::WTN + 32 * in + 8 * q + 4 * fg;
                    if constexpr (OUT == DT_F32) {
                        *reinterpret_cast<f32x4*>(smem + row * EP + 4 * col) = (f32x4){v[0], v[1], v[2], v[3]};
                    } else {
                        *reinterpret_cast<u32x2*>(smem + row * EP + 2 * col) =
                            (u32x2){pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
                    }
                }
            }
        wait_lgkm0();
        barrier_only();
        constexpr int EPC = 16 / ESZ;     // elements per 16-byte piece
        constexpr int PPR = C::TN / EPC;  // pieces per row
        const int c16 = tid % PPR;
        const int64_t n = ne0 + EPC * c16;
#pragma unroll 4
        for (int r = tid / PPR; r < C::TM; r += C::NTH / PPR) {
            const int64_t m = me0 + r;
            if (m >= Mx) break;
            const u32x4 val = *reinterpret_cast<const u32x4*>(smem + r * EP + 16 * c16);
            char* cp = cbase + (m * ldc + n) * ESZ;
            if (vec_ok && n + EPC <= Nx) {
                *reinterpret_cast<u32x4*>(cp) = val;
            } else {
#pragma unroll
                for (int i = 0; i < EPC; ++i) {
                    if (n + i < Nx) {
                        if constexpr (OUT == DT_F32)
                            reinterpret_cast<uint32_t*>(cp)[i] = val[i];
                        else
                            reinterpret_cast<uint16_t*>(cp)[i] = (uint16_t)(val[i >> 1] >> (16 * (i & 1)));
                    }
                }
            }
        }
        return;
    }
    if constexpr (FQ != FQ_NONE) {
        // fused output quantization, in passes of 128 columns (two for 256 x 256 tiles, one for
        // 128 x 128): the fp32 values (as an fp32 C would hold them) are staged in LDS, [TS rows][128]
        // per pass (pass p holds tile columns [128 p, 128 p + 128), written by the waves whose 64
        // columns lie there), then one thread per 32-column group reads its group back, rotates it
        // along N if asked (the four groups of a row are in consecutive lanes) and quantizes it with
        // the rules of the quantize kernels
        static_assert(C::WTN == 2, "64 columns per wave");
        static_assert(C::TM * EP <= C::NST * C::STAGE, "staging buffer exceeds the stage buffers");
        for (int p = 0; p < C::TN / 128; ++p) {
            barrier_only();  // every wave is done with the stage buffers / the last pass
            if ((wn >> 1) == p) {  // wave-uniform
#pragma unroll
                for (int in = 0; in < C::WTN; ++in)
#pragma unroll
                    for (int im = 0; im < C::WTM; ++im) {
                        const int row = wm * 32 * C::WTM + 32 * im + fr;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            f32x4 v;
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] = NVG ? acc[in][im][4 * q + i] * gscale : acc[in][im][4 * q + i];
                            *reinterpret_cast<f32x4*>(smem + row * EP + 4 * (64 * (wn & 1) + 32 * in + 8 * q + 4 * fg)) = v;
                        }
                    }
            }
            wait_lgkm0();
            barrier_only();
#pragma unroll 1
            for (int t = tid; t < C::TM * 4; t += C::NTH) {  // two sweeps, every lane in both
                const int r = t >> 2, j = t & 3;  // row, staged group
                const int64_t m = me0 + r, nb = ne0 + 128 * p + 32 * j;
                float v[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const f32x4 x = *reinterpret_cast<const f32x4*>(smem + r * EP + 4 * (32 * j + 4 * c));
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[4 * c + i] = x[i];
                }
                fwht_groups(v, g.q_hn);
                uint32_t out[8];
                const float amax = block_amax<32, 0>(v);
                uint32_t sbyte;
                const SrSource sr{g.q_seed, (uint64_t)(m * Nx + nb)};
                if constexpr (FQ == FQ_SR) {
                    sbyte = g.q_elem == ELEM_E2M1 ? e8m0_block<ELEM_E2M1, RND_SR, 32, 0>(v, amax, g.q_ceil != 0, sr, out)
                                                  : e8m0_block<ELEM_E4M3, RND_SR, 32, 0>(v, amax, g.q_ceil != 0, sr, out);
                } else {
                    sbyte = g.q_elem == ELEM_E2M1 ? e8m0_block<ELEM_E2M1, RND_RNE, 32, 0>(v, amax, g.q_ceil != 0, sr, out)
                                                  : e8m0_block<ELEM_E4M3, RND_RNE, 32, 0>(v, amax, g.q_ceil != 0, sr, out);
                }
                if (m < Mx && nb < Nx) {
                    if (g.q_elem == ELEM_E2M1) {
                        *reinterpret_cast<u32x4*>(g.qcodes + m * (Nx / 2) + nb / 2) = (u32x4){out[0], out[1], out[2], out[3]};
                    } else {
                        u32x4* d = reinterpret_cast<u32x4*>(g.qcodes + m * Nx + nb);
                        d[0] = (u32x4){out[0], out[1], out[2], out[3]};
                        d[1] = (u32x4){out[4], out[5], out[6], out[7]};
                    }
                    g.qscales[m * (Nx / 32) + nb / 32] = (uint8_t)sbyte;
                }
            }
            if (g.c) {
                // C from the same staged values: 16-byte output pieces, staged column c of a row
                // is tile column 128 p + c
                constexpr int ESZ = OUT == DT_F32 ? 4 : 2, EPC = 16 / ESZ, PPR = 128 / EPC;
                const bool vec_ok = ((reinterpret_cast<uintptr_t>(g.c) & 15) == 0) && ((ldc * ESZ) % 16 == 0);
#pragma unroll 1
                for (int t = tid; t < C::TM * PPR; t += C::NTH) {
                    const int r = t / PPR, c = (t % PPR) * EPC;
                    const int64_t m = me0 + r, n = ne0 + 128 * p + c;
                    if (m >= Mx) continue;
                    const float* src = reinterpret_cast<const float*>(smem + r * EP) + c;
                    u32x4 val;
                    if constexpr (OUT == DT_F32) {
                        val = *reinterpret_cast<const u32x4*>(src);
                    } else {
                        const f32x4 a = *reinterpret_cast<const f32x4*>(src), b = *reinterpret_cast<const f32x4*>(src + 4);
                        val = (u32x4){pack_bf16x2_rne(a[0], a[1]), pack_bf16x2_rne(a[2], a[3]),
                                      pack_bf16x2_rne(b[0], b[1]), pack_bf16x2_rne(b[2], b[3])};
                    }
                    char* cp = cbase + (m * ldc + n) * ESZ;
                    if (vec_ok && n + EPC <= Nx) {
                        *reinterpret_cast<u32x4*>(cp) = val;
                    } else {
                        for (int i = 0; i < EPC; ++i) {
                            if (n + i < Nx) {
                                if constexpr (OUT == DT_F32)
                                    reinterpret_cast<uint32_t*>(cp)[i] = val[i];
                                else
                                    reinterpret_cast<uint16_t*>(cp)[i] = (uint16_t)(val[i >> 1] >> (16 * (i & 1)));
                            }
                        }
                    }
                }
            }
        }
        return;
    }
    constexpr int ESZ = OUT == DT_F32 ? 4 : 2;
    // 16-byte stores need a 16-byte aligned row start
    const bool vec_ok = ((reinterpret_cast<uintptr_t>(g.c) & 15) == 0) && ((ldc * ESZ) % 16 == 0);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        barrier_only();  // every wave is done reading the stage buffers / the last pass
#pragma unroll
        for (int im = 0; im < C::WTM; ++im)
#pragma unroll
            for (int inn = 0; inn < (OUT == DT_F32 ? 1 : C::WTN); ++inn) {
                const int in = OUT == DT_F32 ? p : inn;
                const int row = wm * 128 + 32 * im + fr;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = NVG ? acc[in][im][4 * q + i] * gscale : acc[in][im][4 * q + i];
                    if constexpr (OUT == DT_F32) {
                        const int col = wn * 32 + 8 * q + 4 * fg;
                        *reinterpret_cast<f32x4*>(smem + row * EP + 4 * col) = (f32x4){v[0], v[1], v[2], v[3]};
                    } else {
                        const int col = wn * 64 + 32 * in + 8 * q + 4 * fg;
                        *reinterpret_cast<u32x2*>(smem + row * EP + 2 * col) =
                            (u32x2){pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
                    }
                }
            }
        wait_lgkm0();
        barrier_only();
        // 32 lanes per row, 16 rows per sweep of the workgroup
        const int c16 = tid & 31;
        const int64_t n = OUT == DT_F32 ? ne0 + (c16 >> 3) * 64 + 32 * p + 4 * (c16 & 7) : ne0 + 8 * c16;
        constexpr int EPC = 16 / ESZ;  // elements per 16-byte piece
#pragma unroll 4
        for (int r = tid >> 5; r < 256; r += C::NTH / 32) {
            const int64_t m = me0 + r;
            if (m >= Mx) break;
            const u32x4 val = *reinterpret_cast<const u32x4*>(smem + r * EP + 16 * c16);
            char* cp = cbase + (m * ldc + n) * ESZ;
            if (vec_ok && n + EPC <= Nx) {
                *reinterpret_cast<u32x4*>(cp) = val;
            } else {
#pragma unroll
                for (int i = 0; i < EPC; ++i) {
                    if (n + i < Nx) {
                        if constexpr (OUT == DT_F32)
                            reinterpret_cast<uint32_t*>(cp)[i] = val[i];
                        else
                            reinterpret_cast<uint16_t*>(cp)[i] = (uint16_t)(val[i >> 1] >> (16 * (i & 1)));
                    }
                }
            }
        }
    }
}

// Epilogue of the gated feed-forward's tile (gated.hip).
template <bool FP8, int OUT, int FQ, int TS, int NS>
__device__ __forceinline__ void gated_epilogue(const GemmArgs& g, v16f (&acc)[Big<FP8, TS>::WTN][Big<FP8, TS>::WTM],
                                               int64_t m0, int64_t n0, uint8_t* smem);

// One TS x TS tile of C (tile row tm, tile column tn) by the whole workgroup (512 threads for
// TS = 256, 256 for TS = 128), LDS `smem` of Big<FP8, TS>::NST stages; every thread must call it.
// Leaves the LDS free (every copy into it has landed) but does not end with a barrier.
// GATED: two products of TS x TS / 2 results with the operands b and b_up, N columns each. The rows of B's
// slab alternate between the two in groups of 32 (wave column wn: 32 rows of b, then the same 32 of b_up),
// so that a lane's accumulators of tile 0 and tile 1 are the two products' values of the same place.
// K is a multiple of a stage's depth; GATED also takes rows whose codes end within the last stage (K a multiple of
// 128). RAG (GATED, two stages): K any multiple of 32. Scale rows then begin at any byte, which the copies into LDS
// do not take: each thread reads its scale bytes of the next stage into registers and stores them when the present
// one has been multiplied.
template <bool FP8, bool B2D, int OUT, bool NVG, int FQ, int TS = 256, bool GATED = false, int NS = 2, bool RAG = false>
__device__ __forceinline__ void big_tile(const GemmArgs& g, int tm, int tn, uint8_t* smem) {
    using C = Big<FP8, TS, NS>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int64_t m0 = (int64_t)tm * C::TM, n0 = (int64_t)tn * (GATED ? C::TN / 2 : C::TN);
    const bool up = GATED && (wave & 1);  // this wave's copies of B are b_up's

    const int64_t rowbytes = FP8 ? g.K : g.K / 2;
    const int64_t kgroups = g.K / 32;
    static_assert(!RAG || (GATED && NS == 2), "scales through registers");
    const int KT = GATED ? (int)((g.K + C::KSTEP - 1) / C::KSTEP) : (int)(g.K / C::KSTEP);
    const bool ragged = GATED && g.K % C::KSTEP != 0;

    // Direct-to-LDS copies go through buffer resources: base + 32-bit byte offset. The row part of
    // every offset sits in the per-lane (vector) offset, which the range check covers, so rows
    // beyond M or N read as zero (they only feed outputs that are never stored); the scalar offset
    // only adds the K position within a row.
    const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc((void*)g.a, (short)0, (int)(g.M * rowbytes), 0x00020000);
    const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc((void*)(up ? g.b_up : g.b), (short)0, (int)(g.N * rowbytes), 0x00020000);
    const __amdgpu_buffer_rsrc_t rSA = __builtin_amdgcn_make_buffer_rsrc((void*)g.sa, (short)0, (int)(g.M * kgroups), 0x00020000);
    const __amdgpu_buffer_rsrc_t rSB = __builtin_amdgcn_make_buffer_rsrc(
        (void*)g.sb, (short)0, (int)((B2D ? (g.N + 31) / 32 : g.N) * kgroups), 0x00020000);
    const __amdgpu_buffer_rsrc_t rSU = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(GATED ? g.sb_up : g.sb), (short)0, (int)((B2D ? (g.N + 31) / 32 : g.N) * kgroups), 0x00020000);
    // extent 0: every read through it is out of range and returns zeros
    const __amdgpu_buffer_rsrc_t rZ = __builtin_amdgcn_make_buffer_rsrc((void*)g.a, (short)0, 0, 0x00020000);
    // copy i of this wave fills LDS rows r = (wave * IPW + i) * 8 + lane / 8, slot lane % 8, with
    // chunk slot ^ swz(r) = slot ^ (lane / 8) ^ (i & 1) of the row (IPW is even); wave * IPW * 8 is
    // a multiple of 16, so swz(r) = (lane / 8) ^ (i & 1)
    const int r0 = wave * C::IPW * 8 + (lane >> 3);
    const int rb0 = GATED ? (wave >> 1) * C::IPW * 8 + (lane >> 3) : r0;
    // (a literal bound: with the dependent C::IPW here the host pass silently drops the kernel stub)
    static_assert(C::IPW == 4, "four 1 KB copies per wave and operand");
    int voA[4], voB[4];
#pragma unroll
    for (int i = 0; i < C::IPW; ++i) {
        const int c = (lane & 7) ^ ((lane >> 3) & 7) ^ (i & 1);
        voA[i] = (int)((m0 + r0 + 8 * i) * rowbytes + 16 * c);
        voB[i] = (int)((n0 + rb0 + 8 * i) * rowbytes + 16 * c);
    }
    // scale dwords: the stage holds SPR bytes of each of A's and B's 256 rows, row-major, as
    // consecutive dwords; waves take them in order, A's first. GATED: b's TS / 2 rows, then b_up's, so that
    // a copy of 64 dwords never mixes the two
    int voS[C::SPW];
#pragma unroll
    for (int j = 0; j < C::SPW; ++j) {
        const int d = (wave * C::SPW + j) * 64 + lane;       // dword index over both operands
        const bool isb = (wave * C::SPW + j) * 64 >= C::SB / 4;
        const int dd = isb ? d - C::SB / 4 : d;
        const int r = dd / (C::SPR / 4), part = dd % (C::SPR / 4);
        if (!isb) {
            voS[j] = (int)((m0 + r) * kgroups + 4 * part);
        } else {
            const int64_t nr = n0 + (GATED ? r % (C::TN / 2) : r);
            const int64_t n = B2D ? (nr >> 5) : nr;
            voS[j] = (int)(n * kgroups + 4 * part);
        }
    }

    // The copies of a stage are issued in NKK parts, one per 64-deep MFMA step of the previous
    // stage, so that no wave stalls on a full address FIFO with all its copies at once (part p:
    // A and B copies i in [p IPW / NKK, (p + 1) IPW / NKK); the scales with part 0).
    static_assert(C::IPW % C::NKK == 0, "copies per step");
    // Stages from KT on are dummies: their copies go through the zero-extent resource, so they read
    // nothing and write zeros into a free stage buffer.
    auto issue_part = [&](int kt, int part) {
        uint8_t* st = smem + (kt % C::NST) * C::STAGE;
        const bool real = kt < KT;
        const int so = real ? kt * C::RB : 0, ss = real ? kt * C::SPR : 0;
        const __amdgpu_buffer_rsrc_t qA = real ? rA : rZ, qB = real ? rB : rZ;
        const __amdgpu_buffer_rsrc_t qSA = real ? rSA : rZ;
        const bool cut = ragged && kt == KT - 1;  // chunks past the row's end: offsets past the extent
        const int left = (int)rowbytes - kt * C::RB;
        constexpr int IPP = C::IPW / C::NKK;
#pragma unroll
        for (int ii = 0; ii < IPP; ++ii) {
            const int i = part * IPP + ii;
            const bool gone = cut && 16 * ((lane & 7) ^ ((lane >> 3) & 7) ^ (i & 1)) >= left;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(qA, (lds_ptr_t)(st + C::OFF_A + (wave * C::IPW + i) * 1024), 16,
                                                     gone ? -1 : voA[i], so, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(qB, (lds_ptr_t)(st + C::OFF_B + (wave * C::IPW + i) * 1024),
                                                     16, gone ? -1 : voB[i], so, 0, 0);
        }
        if (part != 0 || RAG) return;
#pragma unroll
        for (int j = 0; j < C::SPW; ++j) {
            const int d0 = (wave * C::SPW + j) * 64 - C::SB / 4;  // wave-uniform
            const bool su = GATED && d0 >= C::SB / 8;
            const int vo = cut && (lane % (C::SPR / 4)) ? -1 : voS[j];
            if (d0 >= 0)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(!real ? rZ : su ? rSU : rSB, (lds_ptr_t)(st + (wave * C::SPW + j) * 256),
                                                         4, vo, ss, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(qSA, (lds_ptr_t)(st + (wave * C::SPW + j) * 256),
                                                         4, vo, ss, 0, 0);
        }
    };
    // RAG: the scale dwords that the copies would place, a byte at a time (groups past the row's end: 0)
    uint32_t held[C::SPW];
    auto read_scales = [&](int kt) {
#pragma unroll
        for (int j = 0; j < C::SPW; ++j) {
            const int d0 = (wave * C::SPW + j) * 64 - C::SB / 4;  // wave-uniform
            const __amdgpu_buffer_rsrc_t r = kt >= KT ? rZ : d0 < 0 ? rSA : d0 >= C::SB / 8 ? rSU : rSB;
            const int first = kt * C::SPR + 4 * (lane % (C::SPR / 4));
            held[j] = 0u;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int vo = first + b < kgroups ? voS[j] + kt * C::SPR + b : -1;
                held[j] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, vo, 0, 0) << (8 * b);
            }
        }
    };
    auto place_scales = [&](int kt) {
        uint8_t* st = smem + (kt % C::NST) * C::STAGE;
#pragma unroll
        for (int j = 0; j < C::SPW; ++j)
            *reinterpret_cast<uint32_t*>(st + (wave * C::SPW + j) * 256 + 4 * lane) = held[j];
    };
    auto issue = [&](int kt) {
#pragma unroll
        for (int p = 0; p < C::NKK; ++p) issue_part(kt, p);
    };

    v16f acc[C::WTN][C::WTM];
#pragma unroll
    for (int i = 0; i < C::WTN; ++i)
#pragma unroll
        for (int j = 0; j < C::WTM; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    // Fragment addresses: rows of tile i of this wave are wm*128 + 32 i + l%32 (A) and
    // wn*64 + 32 i + l%32 (B); their low 4 bits, hence the chunk swizzle, depend on the lane only,
    // so a tile adds the constant 32 * 128 bytes and a K step only changes the chunk term.
    const int fr = lane & 31, fg = lane >> 5;
    const int sw = chunk_swz(fr);
    constexpr int NP = FP8 ? 2 : 1;
    int ch[C::NKK][NP];
#pragma unroll
    for (int kk = 0; kk < C::NKK; ++kk)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = FP8 ? (4 * kk + 2 * p + fg) : (2 * kk + fg);
            ch[kk][p] = 16 * (c ^ sw);
        }
    const int aRow = C::OFF_A + (wm * 32 * C::WTM + fr) * C::RB, bRow = C::OFF_B + (wn * 32 * C::WTN + fr) * C::RB;
    const int aScl = C::SPR * (wm * 32 * C::WTM + fr), bScl = C::OFF_SB + C::SPR * (wn * (GATED ? 32 : 32 * C::WTN) + fr);
    constexpr int BST = GATED ? C::TN / 2 : 32;  // rows from tile 0's scales to tile 1's
    const int sshift = 8 * fg;

#pragma unroll
    for (int s = 0; s < C::NST - 1; ++s) issue(s);
    if constexpr (RAG) {
        read_scales(0);
        place_scales(0);
    }

    auto frag = [&](const uint8_t* p0, const uint8_t* p1) -> v8i {
        const u32x4 x0 = *reinterpret_cast<const u32x4*>(p0);
        if constexpr (!FP8) {
            return (v8i){(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], 0, 0, 0, 0};
        } else {
            const u32x4 x1 = *reinterpret_cast<const u32x4*>(p1);
            return (v8i){(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3],
                         (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
        }
    };

    // One stage: NKK 64-deep steps. Fragments are double-buffered in registers: the reads for step
    // kk + 1 are issued while the MFMAs of step kk run, interleaved one read per MFMA.
    auto load_frags = [&](const uint8_t* st, int kk, v8i (&fa)[C::WTM], v8i (&fb)[C::WTN]) {
#pragma unroll
        for (int i = 0; i < C::WTM; ++i)
            fa[i] = frag(st + aRow + 32 * C::RB * i + ch[kk][0], st + aRow + 32 * C::RB * i + ch[kk][NP - 1]);
#pragma unroll
        for (int i = 0; i < C::WTN; ++i)
            fb[i] = frag(st + bRow + 32 * C::RB * i + ch[kk][0], st + bRow + 32 * C::RB * i + ch[kk][NP - 1]);
    };
    // one stage's MFMAs, with the copies of stage `next` issued along the way
    auto compute = [&](const uint8_t* st, int next) {
        int sa[C::WTM][C::SPR / 4], sb[C::WTN][C::SPR / 4];
#pragma unroll
        for (int i = 0; i < C::WTM; ++i)
#pragma unroll
            for (int d = 0; d < C::SPR / 4; ++d)
                sa[i][d] = (int)(*reinterpret_cast<const uint32_t*>(st + aScl + C::SPR * 32 * i + 4 * d) >> sshift);
#pragma unroll
        for (int i = 0; i < C::WTN; ++i)
#pragma unroll
            for (int d = 0; d < C::SPR / 4; ++d)
                sb[i][d] = (int)(*reinterpret_cast<const uint32_t*>(st + bScl + C::SPR * BST * i + 4 * d) >> sshift);
        v8i fa[2][C::WTM], fb[2][C::WTN];
        load_frags(st, 0, fa[0], fb[0]);
#pragma unroll
        for (int kk = 0; kk < C::NKK; ++kk) {
            const int cur = kk & 1, nxt = cur ^ 1;
            issue_part(next, kk);
            if (kk + 1 < C::NKK) load_frags(st, kk + 1, fa[nxt], fb[nxt]);
            // scale byte of group 2 kk + (l / 32): dword kk / 2 after the lane shift, byte 2 (kk % 2)
#pragma unroll
            for (int in = 0; in < C::WTN; ++in)
#pragma unroll
                for (int im = 0; im < C::WTM; ++im) {
                    if ((kk & 1) == 0)
                        acc[in][im] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            fb[cur][in], fa[cur][im], acc[in][im], FP8 ? 0 : 4, FP8 ? 0 : 4, 0,
                            sb[in][kk >> 1], 0, sa[im][kk >> 1]);
                    else
                        acc[in][im] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            fb[cur][in], fa[cur][im], acc[in][im], FP8 ? 0 : 4, FP8 ? 0 : 4, 2,
                            sb[in][kk >> 1], 2, sa[im][kk >> 1]);
                }
            // issue this step's part of the next stage's copies, the next step's reads, then this
            // step's MFMAs; nothing moves across step boundaries
            if (kk == 0) __builtin_amdgcn_sched_group_barrier(0x020, 2 * (C::IPW / C::NKK) + C::SPW, 0);
            else __builtin_amdgcn_sched_group_barrier(0x020, 2 * (C::IPW / C::NKK), 0);
            if (kk + 1 < C::NKK) __builtin_amdgcn_sched_group_barrier(0x100, (C::WTM + C::WTN) * NP, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, C::WTM * C::WTN, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // main loop, unrolled by the stage count so every stage base is a constant
    for (int k0 = 0; k0 < KT; k0 += C::NST) {
#pragma unroll
        for (int s = 0; s < C::NST; ++s) {
            const int kt = k0 + s;
            if (kt < KT) {
                wait_vm<(C::NST - 2) * C::LOADS>();  // this wave's copies of stage kt have landed
                if constexpr (RAG) wait_lgkm0();     // and its scales
                barrier_only();                      // ... and everyone's; stage kt-1 is no longer read
                if constexpr (RAG) read_scales(kt + 1);  // (past the last stage: nothing)
                compute(smem + s * C::STAGE, kt + C::NST - 1);
                // not past the last stage: no write may be under way when the epilogue takes the LDS
                if (RAG && kt + 1 < KT) place_scales(kt + 1);
            }
        }
    }
    wait_vm<0>();  // the dummy stages' zero-fill has landed before the LDS is reused

    if constexpr (GATED) gated_epilogue<FP8, OUT, FQ, TS, NS>(g, acc, m0, n0, smem);
    else big_epilogue<FP8, OUT, NVG, FQ, TS>(g, acc, m0, n0, smem);
}

}  // namespace bgf
