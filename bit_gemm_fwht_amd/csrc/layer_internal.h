// Kernel arguments and launchers of the operators between a layer's products (norm, rotary positions, gated
// feed-forward), behind the C ABI in layer_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp4.h"
#include "fp4_internal.h"
#include "kv_internal.h"

namespace bgf {

enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// A low-bit output of [rows, cols] fp32 results: MX groups of 32 along the rows.
struct QuantOut {
    uint8_t* codes;  // NULL: none
    uint8_t* scales;
    uint64_t seed;
    int elem, ceil_rule, hn;
};

enum { W_NONE = 0, W_BF16, W_F32 };  // how a norm's weight is stored; none: ones

struct NormArgs {
    const void* x;
    const void* r;
    const void* w;
    void* sum;
    void* y;
    int64_t rows, ldx, ldr, lds, ldy;
    int cols, w_kind;  // w_kind: W_*
    float eps;
    QuantOut q;
};
hipError_t launch_rmsnorm(const NormArgs& a, int dtype, int rnd, hipStream_t s);

struct NormGradArgs {
    const void* dy;
    const void* s;
    const void* dsum;
    const void* w;
    void* dx;
    float* dw;
    float* part;  // [slots, cols]: partial sums of dw
    int64_t rows, lddy, lds, lddsum, lddx;
    int cols, w_kind;  // w_kind: W_*
    float eps;
};
// How the rows are dealt: the same for the size query and the launch.
struct NormGradPlan {
    int lanes;    // lanes of a row
    int np;       // pieces of a lane
    int threads;  // of a workgroup
    int grid;
    int slots;    // partial sums of dw, 0: no dw
};
NormGradPlan plan_rmsnorm_grad(int64_t rows, int cols, bool dw);
hipError_t launch_rmsnorm_grad(const NormGradArgs& a, const NormGradPlan& p, int dtype, hipStream_t s);

struct RopeArgs {
    const void* x[2];
    void* out[2];
    int64_t ldx[2], ldx_head[2], ldo[2], ldo_head[2];
    int heads[2];
    int64_t tokens;
    const double* inv_freq;
    const int32_t* pos;  // NULL: from the batch
    KvView batch;        // cu, ctx, S, T
    float scale;
    int dim, rot, backward;
};
hipError_t launch_rope(const RopeArgs& a, int dtype, int layout, hipStream_t s);

// How a gated product is carried out: the same for the size query and the launch.
enum { GATED_ROWS = 1, GATED_STREAM, GATED_TILE128, GATED_TILE128_DEEP, GATED_TILE128_RAGGED, GATED_TILE256 };
struct GatedPlan {
    int kernel;     // GATED_*, the numbers of FP4_GATED_PLAN_*
    int quant_pass; // h goes to the workspace in fp32 and is quantized by a pass of its own
    int64_t ws;
};
hipError_t plan_gated(int64_t M, int64_t F, int64_t K, bool fp8, const fp4_qparams* q, GatedPlan* p);
hipError_t launch_gated(GemmArgs g, const GatedPlan& p, int kind, int dtype, int fused_q, void* ws, hipStream_t s);

struct GatedGradArgs {
    const void* dh;
    const void* gu;
    void* dgu;
    int64_t rows, lddh, ldgu, lddgu;
    int F, act;
    QuantOut q;
};
hipError_t launch_gated_grad(const GatedGradArgs& a, int dtype, int rnd, hipStream_t s);

}  // namespace bgf
