// C ABI of the key / value cache (declared in include/fp4.h): host-side validation and dispatch.
// Nothing is queued unless every argument has been accepted.
#include "../../include/fp4.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "fp4_internal.h"
#include "kv_internal.h"

namespace {

using namespace bgf;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

constexpr int64_t kMaxRows = int64_t(1) << 30;  // rows and row tiles are counted in 32 bits

int check_batch(const fp4_kv_cache* c, const fp4_kv_batch* b, KvView* v) {
    if (!c || !b) return FP4_ERR_INVALID_ARG;
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return FP4_ERR_INVALID_ARG;
    if (c->pages <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 || c->page_tokens <= 0) return FP4_ERR_INVALID_ARG;
    if (c->k_codes == c->v_codes || c->k_scales == c->v_scales) return FP4_ERR_INVALID_ARG;
    int shift = -1;
    for (int i = 4; i <= 7; ++i)
        if (c->page_tokens == 1 << i) shift = i;
    if (shift < 0 || c->head_dim % 16 || c->head_dim > 256 || c->kv_heads > 65535) return FP4_ERR_UNSUPPORTED;
    if (!b->cu_tokens || !b->context || !b->table) return FP4_ERR_INVALID_ARG;
    if (b->seqs <= 0 || b->table_pages <= 0 || b->table_ld < b->table_pages || b->tokens < 0) return FP4_ERR_INVALID_ARG;
    if (b->max_tokens < 0 || b->max_context < 0) return FP4_ERR_INVALID_ARG;
    if (c->pages > (int64_t(1) << 31) / c->kv_heads - 1) return FP4_ERR_UNSUPPORTED;  // blocks: 32 bits
    if (b->tokens > kMaxRows || b->seqs > kMaxRows / 4) return FP4_ERR_UNSUPPORTED;
    if (!aligned16(c->k_codes) || !aligned16(c->v_codes)) return FP4_ERR_ALIGNMENT;
    v->kc = reinterpret_cast<uint8_t*>(c->k_codes);
    v->vc = reinterpret_cast<uint8_t*>(c->v_codes);
    v->ks = reinterpret_cast<uint8_t*>(c->k_scales);
    v->vs = reinterpret_cast<uint8_t*>(c->v_scales);
    v->pages = c->pages;
    v->H = c->kv_heads;
    v->D = c->head_dim;
    v->P = c->page_tokens;
    v->pshift = shift;
    v->cu = b->cu_tokens;
    v->ctx = b->context;
    v->table = b->table;
    v->table_ld = b->table_ld;
    v->S = b->seqs;
    v->W = b->table_pages;
    v->T = (int)b->tokens;
    return FP4_OK;
}

// rows [tokens, heads, dim] at p: 16-byte aligned, strides of whole 16-byte pieces
int check_rows(const void* p, int64_t ld, int64_t ld_head, int dtype) {
    if (!p || ld < 0 || ld_head < 0) return FP4_ERR_INVALID_ARG;
    const int64_t per = dtype == FP4_DT_BF16 ? 8 : 4;
    if (!aligned16(p) || ld % per || ld_head % per) return FP4_ERR_ALIGNMENT;
    return FP4_OK;
}

// written rows must not share memory with one another
bool disjoint(int64_t tokens, int64_t heads, int64_t dim, int64_t ld, int64_t ld_head) {
    if (tokens > 1 && ld < dim) return false;
    if (heads > 1 && ld_head < dim) return false;
    return tokens <= 1 || heads <= 1 || ld >= (heads - 1) * ld_head + dim || ld_head >= (tokens - 1) * ld + dim;
}

int rows_args(const fp4_kv_cache* cache, const fp4_kv_batch* batch, const void* k, int64_t ldk, int64_t ldk_head,
              const void* v, int64_t ldv, int64_t ldv_head, int32_t dtype, KvRowsArgs* a) {
    int rc = check_batch(cache, batch, &a->c);
    if (rc != FP4_OK) return rc;
    if (dtype != FP4_DT_F32 && dtype != FP4_DT_BF16) return FP4_ERR_INVALID_ARG;
    if (batch->tokens == 0) return FP4_OK;  // no rows: k and v may be NULL
    if ((rc = check_rows(k, ldk, ldk_head, dtype)) != FP4_OK) return rc;
    if ((rc = check_rows(v, ldv, ldv_head, dtype)) != FP4_OK) return rc;
    const void* ins[2] = {k, v};
    for (const void* p : ins)
        if (p == cache->k_codes || p == cache->v_codes || p == cache->k_scales || p == cache->v_scales)
            return FP4_ERR_INVALID_ARG;
    a->k = k;
    a->v = v;
    a->ldk = ldk;
    a->ldk_head = ldk_head;
    a->ldv = ldv;
    a->ldv_head = ldv_head;
    return FP4_OK;
}

int attn_args(const fp4_kv_cache* cache, const fp4_kv_batch* batch, const fp4_kv_attn* t, KvAttnArgs* a, KvAttnPlan* p) {
    const int rc = check_batch(cache, batch, &a->c);
    if (rc != FP4_OK) return rc;
    if (!t) return FP4_ERR_INVALID_ARG;
    if ((int64_t)batch->table_pages * cache->page_tokens > kMaxKeys) return FP4_ERR_UNSUPPORTED;
    if (t->dtype != FP4_DT_F32 && t->dtype != FP4_DT_BF16) return FP4_ERR_INVALID_ARG;
    if (t->q_heads <= 0 || t->q_heads % cache->kv_heads || t->window < 0 || !std::isfinite(t->scale))
        return FP4_ERR_INVALID_ARG;
    const int64_t rows = batch->tokens * (t->q_heads / cache->kv_heads);
    if (rows > kMaxRows || (rows / 16 + batch->seqs) * cache->kv_heads > kMaxUnits) return FP4_ERR_UNSUPPORTED;
    a->q = t->q;
    a->out = t->out;
    a->lse = t->lse;
    a->ldq = t->ldq;
    a->ldq_head = t->ldq_head;
    a->ldo = t->ldo;
    a->ldo_head = t->ldo_head;
    a->Hq = t->q_heads;
    a->G = t->q_heads / cache->kv_heads;
    a->scale_log2 = (float)(std::fabs((double)t->scale) * 1.4426950408889634);
    a->flip = t->scale < 0.0f;
    a->causal = t->causal != 0;
    a->window = t->window;
    *p = plan_kv_attention(a->c, t->q_heads, t->window, t->dtype, batch->max_tokens, batch->max_context);
    return FP4_OK;
}

int hip_status(hipError_t e) { return e == hipSuccess ? FP4_OK : FP4_ERR_HIP; }

}  // namespace

extern "C" {

int fp4_kv_append(const fp4_kv_cache* cache, const fp4_kv_batch* batch, const void* k, int64_t ldk, int64_t ldk_head,
                  const void* v, int64_t ldv, int64_t ldv_head, int32_t dtype, int32_t scale_mode, void* stream) {
    try {
        KvRowsArgs a{};
        const int rc = rows_args(cache, batch, k, ldk, ldk_head, v, ldv, ldv_head, dtype, &a);
        if (rc != FP4_OK) return rc;
        if (scale_mode != FP4_SCALE_E8M0_FLOOR && scale_mode != FP4_SCALE_E8M0_CEIL) return FP4_ERR_UNSUPPORTED;
        if (batch->tokens == 0) return FP4_OK;
        a.ceil_rule = scale_mode == FP4_SCALE_E8M0_CEIL;
        return hip_status(launch_kv_append(a, dtype, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int fp4_kv_read(const fp4_kv_cache* cache, const fp4_kv_batch* batch, void* k, int64_t ldk, int64_t ldk_head, void* v,
                int64_t ldv, int64_t ldv_head, int32_t dtype, void* stream) {
    try {
        KvRowsArgs a{};
        const int rc = rows_args(cache, batch, k, ldk, ldk_head, v, ldv, ldv_head, dtype, &a);
        if (rc != FP4_OK) return rc;
        if (batch->tokens == 0) return FP4_OK;
        if (k == v || !disjoint(batch->tokens, cache->kv_heads, cache->head_dim, ldk, ldk_head) ||
            !disjoint(batch->tokens, cache->kv_heads, cache->head_dim, ldv, ldv_head))
            return FP4_ERR_INVALID_ARG;
        return hip_status(launch_kv_read(a, dtype, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int fp4_kv_attention_plan(const fp4_kv_cache* cache, const fp4_kv_batch* batch, const fp4_kv_attn* t, fp4_kv_plan* out) {
    try {
        KvAttnArgs a{};
        KvAttnPlan p{};
        if (!out) return FP4_ERR_INVALID_ARG;
        const int rc = attn_args(cache, batch, t, &a, &p);
        if (rc != FP4_OK) return rc;
        *out = fp4_kv_plan{};
        if (batch->tokens == 0) return FP4_OK;
        out->waves = p.nw;
        if (p.tile_slots) {
            out->kernel = FP4_KV_PLAN_TILES;
            out->tile_rows = 32 * p.nw;
            out->workgroups = (int64_t)p.tile_slots * cache->kv_heads;
        } else {
            out->kernel = !p.join_rows ? FP4_KV_PLAN_ROWS : p.near ? FP4_KV_PLAN_ROWS_NEAR : FP4_KV_PLAN_ROWS_SPLIT;
            out->tile_rows = 16;
            out->workgroups = p.grid;
        }
        return FP4_OK;
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int64_t fp4_kv_attention_workspace_bytes(const fp4_kv_cache* cache, const fp4_kv_batch* batch, const fp4_kv_attn* t) {
    try {
        KvAttnArgs a{};
        KvAttnPlan p{};
        if (attn_args(cache, batch, t, &a, &p) != FP4_OK) return -1;
        return batch->tokens == 0 ? 0 : p.ws;
    } catch (...) {
        return -1;
    }
}

int fp4_kv_attention(const fp4_kv_cache* cache, const fp4_kv_batch* batch, const fp4_kv_attn* t, void* workspace,
                     int64_t ws_bytes, void* stream) {
    try {
        KvAttnArgs a{};
        KvAttnPlan p{};
        int rc = attn_args(cache, batch, t, &a, &p);
        if (rc != FP4_OK) return rc;
        if (batch->tokens == 0) return FP4_OK;
        if ((rc = check_rows(t->q, t->ldq, t->ldq_head, t->dtype)) != FP4_OK) return rc;
        if ((rc = check_rows(t->out, t->ldo, t->ldo_head, t->dtype)) != FP4_OK) return rc;
        if (!disjoint(batch->tokens, t->q_heads, cache->head_dim, t->ldo, t->ldo_head)) return FP4_ERR_INVALID_ARG;
        const void* held[4] = {cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales};
        for (const void* q : held)
            if (q == t->out || q == t->lse) return FP4_ERR_INVALID_ARG;
        if (t->out == t->q || (t->lse && (t->lse == t->out || t->lse == t->q))) return FP4_ERR_INVALID_ARG;
        if (p.ws > 0) {
            if (!workspace || ws_bytes < p.ws) return FP4_ERR_WORKSPACE;
            if (!aligned16(workspace)) return FP4_ERR_ALIGNMENT;
        }
        return hip_status(launch_kv_attention(a, p, t->dtype, workspace, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

}  // extern "C"
