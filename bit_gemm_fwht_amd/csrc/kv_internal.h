// The paged 8-bit key / value cache as the kernels see it, and the launchers behind the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bgf {

// Tokens of a table at most, in attention: keys are counted in 32 bits, and pages are looked up a few
// steps past the last one.
constexpr int kMaxKeys = 0x7FFFF000;
// Tiles of 16 rows, and units of keys of them, in one call at most: their sums stay in 32 bits.
constexpr int64_t kMaxUnits = int64_t(1) << 30;
// Workgroups along one axis of a launch at most: its threads (512 each at most) have to stay below 2^32.
constexpr int64_t kMaxGrid = int64_t(1) << 22;

// Cache and batch of one call (layouts in include/fp4.h).
struct KvView {
    uint8_t* kc;
    uint8_t* vc;
    uint8_t* ks;
    uint8_t* vs;
    int64_t pages;
    int H, D, P, pshift;  // kv heads, head dim, tokens of a page and its log2
    const int32_t* cu;
    const int32_t* ctx;
    const int32_t* table;
    int64_t table_ld;
    int S, W;  // sequences, pages of a table row
    int T;     // rows of the batch
};

// Rows to or from the cache: k and v [T, H, D], strides in elements.
struct KvRowsArgs {
    KvView c;
    const void* k;
    const void* v;
    int64_t ldk, ldk_head, ldv, ldv_head;
    int ceil_rule;
};

struct KvAttnArgs {
    KvView c;
    const void* q;
    void* out;
    float* lse;
    int64_t ldq, ldq_head, ldo, ldo_head;
    int Hq, G;
    float scale_log2;  // |scale| * log2(e)
    int flip;          // scale < 0: q is negated
    int causal, window;
    int slots;         // row tiles of the kernel for many rows (at least those that have rows)
    int grid;          // workgroups of the kernel for few rows
    uint32_t unit;     // keys that work is counted in, a multiple of 64 (16 rows), 2^31: whole tiles
    int share_min;     // units of a workgroup, at least
    bool near;         // shares that follow one another go to the same XCD
    float* part_o;     // [grid][2][16][D] unnormalised outputs of tiles that workgroups share
    float* part_ml;    // [grid][2][16][2] maximum (log2 units) and sum
};

hipError_t launch_kv_append(const KvRowsArgs& a, int dtype, hipStream_t s);
hipError_t launch_kv_read(const KvRowsArgs& a, int dtype, hipStream_t s);

// How an attention call is cut into workgroups; the same for the size query and the launch.
struct KvAttnPlan {
    int tile_slots;  // row tiles of the kernel for many rows, 0: the kernel for few
    int grid, share_min, nw;
    uint32_t unit;
    bool near;
    int join_rows;  // workgroups of the join for each share, 0: no tile is split
    int64_t ws;     // bytes of workspace
};
KvAttnPlan plan_kv_attention(const KvView& c, int Hq, int window, int dtype, int max_tokens, int max_context);
hipError_t launch_kv_attention(KvAttnArgs a, const KvAttnPlan& p, int dtype, void* ws, hipStream_t s);

}  // namespace bgf
