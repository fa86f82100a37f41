// C ABI of the operators between a layer's products (declared in include/fp4.h): host-side validation and
// dispatch. Nothing is queued unless every argument has been accepted.
#include "../../include/fp4.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "layer_internal.h"

namespace {

using namespace bgf;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxPlaces = int64_t(1) << 58;  // of h: bytes of gu and of the workspace stay in 64 bits
constexpr int kMaxCols = 32768;  // of a norm: a row's pieces stay in registers

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(int d) { return d == FP4_DT_F32 || d == FP4_DT_BF16; }
int per16(int dtype) { return dtype == FP4_DT_BF16 ? 8 : 4; }
int hip_status(hipError_t e) { return e == hipSuccess ? FP4_OK : FP4_ERR_HIP; }

// a [rows, cols] tensor of 16-byte aligned rows
int check_matrix(const void* p, int64_t ld, int64_t cols, int dtype) {
    if (!p || ld < cols) return FP4_ERR_INVALID_ARG;
    if (!aligned(p, 16) || ld % per16(dtype)) return FP4_ERR_ALIGNMENT;
    return FP4_OK;
}

// in place: the same pointer needs the same pitch
bool in_place_ok(const void* out, int64_t ldo, const void* in, int64_t ldi) { return out != in || ldo == ldi; }

// out_q and q of a [rows, cols] result; fills o (codes NULL: none)
int check_quant(const fp4_qparams* p, const fp4_qtensor* q, int64_t rows, int64_t cols, int max_hn, QuantOut* o) {
    *o = QuantOut{};
    if ((p != nullptr) != (q != nullptr)) return FP4_ERR_INVALID_ARG;
    if (!p) return FP4_OK;
    if (p->elem != FP4_ELEM_E2M1 && p->elem != FP4_ELEM_E4M3) return FP4_ERR_INVALID_ARG;
    if (p->round_mode != FP4_ROUND_RNE && p->round_mode != FP4_ROUND_SR) return FP4_ERR_INVALID_ARG;
    const int n = p->hadamard_n;
    if (n != 0 && n != 16 && n != 32 && n != 64 && n != 128 && n != 256) return FP4_ERR_INVALID_ARG;
    if (p->block_rows != 1 || p->block_cols != 32 || n > max_hn) return FP4_ERR_UNSUPPORTED;
    if (p->scale_mode != FP4_SCALE_E8M0_FLOOR && p->scale_mode != FP4_SCALE_E8M0_CEIL) return FP4_ERR_UNSUPPORTED;
    if (cols % 32 || (n && cols % n)) return FP4_ERR_INVALID_ARG;
    if (rows == 0) return FP4_OK;  // nothing is written
    if (!q->codes || !q->scales || q->codes == q->scales) return FP4_ERR_INVALID_ARG;
    if (!aligned(q->codes, 16)) return FP4_ERR_ALIGNMENT;
    o->codes = reinterpret_cast<uint8_t*>(q->codes);
    o->scales = reinterpret_cast<uint8_t*>(q->scales);
    o->seed = p->seed;
    o->elem = p->elem == FP4_ELEM_E2M1 ? ELEM_E2M1 : ELEM_E4M3;
    o->ceil_rule = p->scale_mode == FP4_SCALE_E8M0_CEIL;
    o->hn = n;
    return FP4_OK;
}

// describe what is written
void set_quant(fp4_qtensor* q, const fp4_qparams* p, int64_t rows, int64_t cols) {
    if (!p) return;
    q->rows = rows;
    q->cols = cols;
    q->tensor_scale = nullptr;
    q->p = *p;
}

int rnd_of(const fp4_qparams* p) { return p && p->round_mode == FP4_ROUND_SR ? RND_SR : RND_RNE; }

template <typename... T>
bool writes(const QuantOut& q, T... in) {  // whether a low-bit output is one of the other tensors
    bool hit = false;
    const void* a[] = {in...};
    for (const void* p : a) hit = hit || (p && (p == q.codes || p == q.scales));
    return hit;
}

int check_norm_grad(const fp4_norm_grad* n) {
    if (!n || n->rows < 0 || n->cols <= 0 || !dtype_ok(n->dtype)) return FP4_ERR_INVALID_ARG;
    if (n->weight && !dtype_ok(n->w_dtype)) return FP4_ERR_INVALID_ARG;
    if (!(n->eps >= 0.0f) || !std::isfinite(n->eps)) return FP4_ERR_INVALID_ARG;
    if (n->cols % 8 || n->cols > kMaxCols || n->rows > kMaxRows) return FP4_ERR_UNSUPPORTED;
    return FP4_OK;
}

bool groups32(const fp4_qparams& p) {
    return p.block_rows == 1 && p.block_cols == 32 && (p.scale_mode == FP4_SCALE_E8M0_FLOOR || p.scale_mode == FP4_SCALE_E8M0_CEIL);
}
bool tiles32(const fp4_qparams& p) {
    return p.block_rows == 32 && p.block_cols == 32 && (p.scale_mode == FP4_SCALE_E8M0_FLOOR || p.scale_mode == FP4_SCALE_E8M0_CEIL);
}

// Shapes and parameters of a gated call, without its buffers; rows of A may be none.
int check_gated(const fp4_qtensor* A, const fp4_qtensor* G, const fp4_qtensor* U, const fp4_gated* o, const fp4_qparams* out_q,
                int* kind, int* b2d, GatedPlan* plan) {
    if (!A || !G || !U || !o || !dtype_ok(o->dtype)) return FP4_ERR_INVALID_ARG;
    if (o->act < FP4_ACT_SILU || o->act > FP4_ACT_GELU_TANH) return FP4_ERR_INVALID_ARG;
    if (A->rows < 0 || G->rows <= 0 || A->cols <= 0 || G->rows != U->rows || A->cols != G->cols || A->cols != U->cols)
        return FP4_ERR_INVALID_ARG;
    const int64_t M = A->rows, F = G->rows, K = A->cols;
    const fp4_qparams &pa = A->p, &pg = G->p, &pu = U->p;
    if (K % 32 || pa.hadamard_n != pg.hadamard_n) return FP4_ERR_INVALID_ARG;
    if (pg.elem != pu.elem || pg.block_rows != pu.block_rows || pg.block_cols != pu.block_cols || pg.hadamard_n != pu.hadamard_n)
        return FP4_ERR_INVALID_ARG;
    if (pa.elem != pg.elem || !groups32(pa) || !((groups32(pg) && groups32(pu)) || (tiles32(pg) && tiles32(pu)))) return FP4_ERR_UNSUPPORTED;
    *b2d = tiles32(pg);
    *kind = pa.elem == FP4_ELEM_E4M3 ? 1 : 0;
    if (pa.elem != FP4_ELEM_E2M1 && pa.elem != FP4_ELEM_E4M3) return FP4_ERR_INVALID_ARG;
    if (*kind == 1 && *b2d) return FP4_ERR_UNSUPPORTED;
    if (*b2d && F % 32) return FP4_ERR_INVALID_ARG;
    if (M > kMaxRows || F > kMaxRows || K > kMaxRows) return FP4_ERR_UNSUPPORTED;
    if (M > 0 && F > kMaxPlaces / M) return FP4_ERR_UNSUPPORTED;
    if (out_q) {
        fp4_qtensor none{};
        QuantOut unused;
        const int rc = check_quant(out_q, &none, 0, F, 128, &unused);
        if (rc != FP4_OK) return rc;
    }
    *plan = GatedPlan{};
    if (M == 0) return FP4_OK;
    return hip_status(plan_gated(M, F, K, *kind == 1, out_q, plan));
}

// scales of K a multiple of 128 are read four at a time, others one at a time (a fused weight's lower half may then
// begin anywhere)
int check_codes(const fp4_qtensor* t) {
    if (!t->codes || !t->scales) return FP4_ERR_INVALID_ARG;
    if (!aligned(t->codes, 16) || (t->cols % 128 == 0 && !aligned(t->scales, 4))) return FP4_ERR_ALIGNMENT;
    return FP4_OK;
}

}  // namespace

extern "C" {

int fp4_rmsnorm(const fp4_norm* n, const fp4_qparams* out_q, fp4_qtensor* y_q, void* stream) {
    try {
        if (!n || n->rows < 0 || n->cols <= 0 || !dtype_ok(n->dtype)) return FP4_ERR_INVALID_ARG;
        if (n->weight && !dtype_ok(n->w_dtype)) return FP4_ERR_INVALID_ARG;
        if (!(n->eps >= 0.0f) || !std::isfinite(n->eps)) return FP4_ERR_INVALID_ARG;
        if (!out_q && !n->y && n->rows > 0) return FP4_ERR_INVALID_ARG;
        if ((n->residual != nullptr) != (n->sum != nullptr)) return FP4_ERR_INVALID_ARG;
        if (n->cols % 8 || n->cols > kMaxCols || n->rows > kMaxRows) return FP4_ERR_UNSUPPORTED;
        NormArgs a{};
        int rc = check_quant(out_q, y_q, n->rows, n->cols, 256, &a.q);
        if (rc != FP4_OK) return rc;
        if (n->rows == 0) {
            set_quant(y_q, out_q, 0, n->cols);
            return FP4_OK;
        }
        if ((rc = check_matrix(n->x, n->ldx, n->cols, n->dtype)) != FP4_OK) return rc;
        if (n->residual) {
            if ((rc = check_matrix(n->residual, n->ldr, n->cols, n->dtype)) != FP4_OK) return rc;
            if ((rc = check_matrix(n->sum, n->lds, n->cols, n->dtype)) != FP4_OK) return rc;
            if (!in_place_ok(n->sum, n->lds, n->x, n->ldx) || !in_place_ok(n->sum, n->lds, n->residual, n->ldr)) return FP4_ERR_INVALID_ARG;
        }
        if (n->y) {
            if ((rc = check_matrix(n->y, n->ldy, n->cols, n->dtype)) != FP4_OK) return rc;
            if (!in_place_ok(n->y, n->ldy, n->x, n->ldx) || n->y == n->sum || (n->residual && n->y == n->residual)) return FP4_ERR_INVALID_ARG;
        }
        if (n->weight) {
            if (!aligned(n->weight, 16)) return FP4_ERR_ALIGNMENT;
            if (n->weight == n->sum || n->weight == n->y) return FP4_ERR_INVALID_ARG;
        }
        if (writes(a.q, n->x, n->residual, n->weight, (const void*)n->sum, (const void*)n->y)) return FP4_ERR_INVALID_ARG;
        a.x = n->x;
        a.r = n->residual;
        a.w = n->weight;
        a.sum = n->sum;
        a.y = n->y;
        a.rows = n->rows;
        a.ldx = n->ldx;
        a.ldr = n->ldr;
        a.lds = n->lds;
        a.ldy = n->ldy;
        a.cols = (int)n->cols;
        a.w_kind = !n->weight ? W_NONE : n->w_dtype == FP4_DT_BF16 ? W_BF16 : W_F32;
        a.eps = n->eps;
        set_quant(y_q, out_q, n->rows, n->cols);
        return hip_status(launch_rmsnorm(a, n->dtype, rnd_of(out_q), reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int64_t fp4_rmsnorm_backward_workspace_bytes(const fp4_norm_grad* n) {
    try {
        if (check_norm_grad(n) != FP4_OK) return -1;
        return (int64_t)plan_rmsnorm_grad(n->rows, (int)n->cols, n->dweight != nullptr).slots * n->cols * 4;
    } catch (...) {
        return -1;
    }
}

int fp4_rmsnorm_backward(const fp4_norm_grad* n, void* workspace, int64_t ws_bytes, void* stream) {
    try {
        int rc = check_norm_grad(n);
        if (rc != FP4_OK) return rc;
        if (n->dweight && !aligned(n->dweight, 16)) return FP4_ERR_ALIGNMENT;
        if (n->rows > 0) {
            if ((rc = check_matrix(n->dy, n->lddy, n->cols, n->dtype)) != FP4_OK) return rc;
            if ((rc = check_matrix(n->s, n->lds, n->cols, n->dtype)) != FP4_OK) return rc;
            if ((rc = check_matrix(n->dx, n->lddx, n->cols, n->dtype)) != FP4_OK) return rc;
            if (n->dsum && (rc = check_matrix(n->dsum, n->lddsum, n->cols, n->dtype)) != FP4_OK) return rc;
            if (!in_place_ok(n->dx, n->lddx, n->dy, n->lddy) || (n->dsum && !in_place_ok(n->dx, n->lddx, n->dsum, n->lddsum)))
                return FP4_ERR_INVALID_ARG;
            if (n->dx == n->s) return FP4_ERR_INVALID_ARG;
            if (n->weight && !aligned(n->weight, 16)) return FP4_ERR_ALIGNMENT;
            const void* in[] = {n->dy, n->s, n->dsum, n->dx, n->weight};
            for (const void* p : in)
                if (n->dweight && p == n->dweight) return FP4_ERR_INVALID_ARG;
            if (n->weight && n->weight == n->dx) return FP4_ERR_INVALID_ARG;
        }
        const NormGradPlan p = plan_rmsnorm_grad(n->rows, (int)n->cols, n->dweight != nullptr);
        const int64_t need = (int64_t)p.slots * n->cols * 4;
        if (need > 0) {
            if (!workspace || ws_bytes < need) return FP4_ERR_WORKSPACE;
            if (!aligned(workspace, 16)) return FP4_ERR_ALIGNMENT;
        }
        if (n->rows == 0 && !n->dweight) return FP4_OK;
        NormGradArgs a{};
        a.dy = n->dy;
        a.s = n->s;
        a.dsum = n->dsum;
        a.w = n->weight;
        a.dx = n->dx;
        a.dw = n->dweight;
        a.part = need > 0 ? reinterpret_cast<float*>(workspace) : nullptr;
        a.rows = n->rows;
        a.lddy = n->lddy;
        a.lds = n->lds;
        a.lddsum = n->lddsum;
        a.lddx = n->lddx;
        a.cols = (int)n->cols;
        a.w_kind = !n->weight ? W_NONE : n->w_dtype == FP4_DT_BF16 ? W_BF16 : W_F32;
        a.eps = n->eps;
        return hip_status(launch_rmsnorm_grad(a, p, n->dtype, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int fp4_rope(const fp4_rope_args* r, void* stream) {
    try {
        if (!r || r->tokens < 0 || !dtype_ok(r->dtype)) return FP4_ERR_INVALID_ARG;
        if (r->layout != FP4_ROPE_HALF && r->layout != FP4_ROPE_INTERLEAVED) return FP4_ERR_INVALID_ARG;
        if (r->heads[0] <= 0 || r->heads[1] < 0 || r->head_dim <= 0) return FP4_ERR_INVALID_ARG;
        if (r->rotary_dim <= 0 || r->rotary_dim % 2 || r->rotary_dim > r->head_dim) return FP4_ERR_INVALID_ARG;
        if (!std::isfinite(r->scale) || !r->inv_freq || (r->positions && r->batch)) return FP4_ERR_INVALID_ARG;
        if (!r->positions && !r->batch && r->tokens > 0) return FP4_ERR_INVALID_ARG;
        const int64_t heads = (int64_t)r->heads[0] + r->heads[1];
        if (r->head_dim > 1024 || r->head_dim % 2 || heads > 65536 || r->tokens > kMaxRows || r->tokens * heads > kMaxRows) return FP4_ERR_UNSUPPORTED;
        if (!aligned(r->inv_freq, 8) || !aligned(r->positions, 4)) return FP4_ERR_ALIGNMENT;
        RopeArgs a{};
        if (r->batch) {
            const fp4_kv_batch* b = r->batch;
            if (!b->cu_tokens || !b->context || b->seqs <= 0 || b->tokens != r->tokens) return FP4_ERR_INVALID_ARG;
            if (b->seqs > (1 << 28) || r->tokens > (1 << 30)) return FP4_ERR_UNSUPPORTED;
            a.batch.cu = b->cu_tokens;
            a.batch.ctx = b->context;
            a.batch.S = b->seqs;
            a.batch.T = (int)b->tokens;
        }
        if (r->tokens == 0) return FP4_OK;
        const int per = per16(r->dtype);
        for (int i = 0; i < 2; ++i) {
            if (!r->heads[i]) continue;
            if (!r->x[i] || !r->out[i] || r->ldx[i] < 0 || r->ldx_head[i] < 0 || r->ldo[i] < 0 || r->ldo_head[i] < 0)
                return FP4_ERR_INVALID_ARG;
            if (!aligned(r->x[i], 16) || !aligned(r->out[i], 16) || r->ldx[i] % per || r->ldx_head[i] % per || r->ldo[i] % per ||
                r->ldo_head[i] % per)
                return FP4_ERR_ALIGNMENT;
            if (r->out[i] == r->x[i] && (r->ldo[i] != r->ldx[i] || r->ldo_head[i] != r->ldx_head[i])) return FP4_ERR_INVALID_ARG;
            // written rows must not share memory with one another
            const int64_t T = r->tokens, H = r->heads[i], D = r->head_dim, ld = r->ldo[i], lh = r->ldo_head[i];
            if ((T > 1 && ld < D) || (H > 1 && lh < D)) return FP4_ERR_INVALID_ARG;
            if (T > 1 && H > 1 && ld < (H - 1) * lh + D && lh < (T - 1) * ld + D) return FP4_ERR_INVALID_ARG;
        }
        if (r->heads[1] && (r->out[0] == r->out[1] || r->out[0] == r->x[1] || r->out[1] == r->x[0])) return FP4_ERR_INVALID_ARG;
        for (int i = 0; i < 2; ++i) {
            a.x[i] = r->x[i];
            a.out[i] = r->out[i];
            a.ldx[i] = r->ldx[i];
            a.ldx_head[i] = r->ldx_head[i];
            a.ldo[i] = r->ldo[i];
            a.ldo_head[i] = r->ldo_head[i];
            a.heads[i] = r->heads[i];
        }
        a.tokens = r->tokens;
        a.inv_freq = r->inv_freq;
        a.pos = r->positions;
        a.scale = r->scale;
        a.dim = r->head_dim;
        a.rot = r->rotary_dim;
        a.backward = r->backward != 0;
        return hip_status(launch_rope(a, r->dtype, r->layout, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int64_t fp4_gemm_gated_workspace_bytes(const fp4_qtensor* A, const fp4_qtensor* gate, const fp4_qtensor* up,
                                       const fp4_gated* o, const fp4_qparams* out_q) {
    try {
        int kind, b2d;
        GatedPlan p{};
        if (check_gated(A, gate, up, o, out_q, &kind, &b2d, &p) != FP4_OK) return -1;
        return p.ws;
    } catch (...) {
        return -1;
    }
}

int fp4_gemm_gated_plan(const fp4_qtensor* A, const fp4_qtensor* gate, const fp4_qtensor* up, const fp4_gated* o,
                        const fp4_qparams* out_q, fp4_gated_plan* plan) {
    try {
        int kind, b2d;
        GatedPlan p{};
        if (!plan) return FP4_ERR_INVALID_ARG;
        const int rc = check_gated(A, gate, up, o, out_q, &kind, &b2d, &p);
        if (rc != FP4_OK) return rc;
        plan->kernel = p.kernel;
        plan->quantize_pass = p.quant_pass;
        return FP4_OK;
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int fp4_gemm_gated(const fp4_qtensor* A, const fp4_qtensor* gate, const fp4_qtensor* up, const fp4_gated* o,
                   const fp4_qparams* out_q, fp4_qtensor* h_q, void* workspace, int64_t ws_bytes, void* stream) {
    try {
        int kind, b2d;
        GatedPlan p{};
        int rc = check_gated(A, gate, up, o, out_q, &kind, &b2d, &p);
        if (rc != FP4_OK) return rc;
        const int64_t M = A->rows, F = gate->rows, K = A->cols;
        QuantOut q;
        if ((rc = check_quant(out_q, h_q, M, F, 128, &q)) != FP4_OK) return rc;
        if (M == 0) {
            set_quant(h_q, out_q, 0, F);
            return FP4_OK;
        }
        if (!o->h && !o->gu && !out_q) return FP4_ERR_INVALID_ARG;
        const fp4_qtensor* ops[] = {A, gate, up};
        for (const fp4_qtensor* t : ops)
            if ((rc = check_codes(t)) != FP4_OK) return rc;
        if (o->h) {
            if (o->ldh < F) return FP4_ERR_INVALID_ARG;
            if (!aligned(o->h, 16)) return FP4_ERR_ALIGNMENT;
        }
        if (o->gu) {
            if (o->ldgu < 2 * F || o->gu == o->h) return FP4_ERR_INVALID_ARG;
            if (!aligned(o->gu, 16)) return FP4_ERR_ALIGNMENT;
        }
        const void* in[] = {A->codes, A->scales, gate->codes, gate->scales, up->codes, up->scales};
        for (const void* x : in)
            if (x == o->h || x == o->gu || (q.codes && (x == q.codes || x == q.scales))) return FP4_ERR_INVALID_ARG;
        if (writes(q, (const void*)o->h, (const void*)o->gu)) return FP4_ERR_INVALID_ARG;
        if (p.ws > 0) {
            if (!workspace || ws_bytes < p.ws) return FP4_ERR_WORKSPACE;
            if (!aligned(workspace, 16)) return FP4_ERR_ALIGNMENT;
        }
        GemmArgs g{};
        g.a = reinterpret_cast<const uint8_t*>(A->codes);
        g.sa = reinterpret_cast<const uint8_t*>(A->scales);
        g.b = reinterpret_cast<const uint8_t*>(gate->codes);
        g.sb = reinterpret_cast<const uint8_t*>(gate->scales);
        g.b_up = reinterpret_cast<const uint8_t*>(up->codes);
        g.sb_up = reinterpret_cast<const uint8_t*>(up->scales);
        g.M = M;
        g.N = F;
        g.K = K;
        g.c = o->h;
        g.ldc = o->ldh;
        g.gu = o->gu;
        g.ldgu = o->ldgu;
        g.act = o->act == FP4_ACT_SILU ? ACT_SILU : o->act == FP4_ACT_GELU ? ACT_GELU : ACT_GELU_TANH;
        g.b_2d = b2d;
        g.qcodes = q.codes;
        g.qscales = q.scales;
        g.q_elem = q.elem;
        g.q_ceil = q.ceil_rule;
        g.q_hn = q.hn;
        g.q_seed = q.seed;
        g.q_round = rnd_of(out_q);
        set_quant(h_q, out_q, M, F);
        return hip_status(launch_gated(g, p, kind, o->dtype, out_q != nullptr, workspace, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

int fp4_gated_backward(const fp4_gated_grad* n, const fp4_qparams* out_q, fp4_qtensor* dgu_q, void* stream) {
    try {
        if (!n || n->rows < 0 || n->cols <= 0 || !dtype_ok(n->dtype)) return FP4_ERR_INVALID_ARG;
        if (n->act < FP4_ACT_SILU || n->act > FP4_ACT_GELU_TANH) return FP4_ERR_INVALID_ARG;
        if (!out_q && !n->dgu && n->rows > 0) return FP4_ERR_INVALID_ARG;
        if (n->cols % 8 || n->cols > (1 << 28) || n->rows > kMaxRows) return FP4_ERR_UNSUPPORTED;
        GatedGradArgs a{};
        // groups and chunks of the 2 F columns have to lie within one of the two halves
        int rc = check_quant(out_q, dgu_q, n->rows, n->cols, 256, &a.q);
        if (rc != FP4_OK) return rc;
        if (n->rows == 0) {
            set_quant(dgu_q, out_q, 0, 2 * n->cols);
            return FP4_OK;
        }
        if ((rc = check_matrix(n->dh, n->lddh, n->cols, n->dtype)) != FP4_OK) return rc;
        if ((rc = check_matrix(n->gu, n->ldgu, 2 * n->cols, n->dtype)) != FP4_OK) return rc;
        if (n->dgu) {
            if ((rc = check_matrix(n->dgu, n->lddgu, 2 * n->cols, n->dtype)) != FP4_OK) return rc;
            if (!in_place_ok(n->dgu, n->lddgu, n->gu, n->ldgu) || n->dgu == n->dh) return FP4_ERR_INVALID_ARG;
        }
        if (writes(a.q, n->dh, n->gu, (const void*)n->dgu)) return FP4_ERR_INVALID_ARG;
        a.dh = n->dh;
        a.gu = n->gu;
        a.dgu = n->dgu;
        a.rows = n->rows;
        a.lddh = n->lddh;
        a.ldgu = n->ldgu;
        a.lddgu = n->lddgu;
        a.F = (int)n->cols;
        a.act = n->act == FP4_ACT_SILU ? ACT_SILU : n->act == FP4_ACT_GELU ? ACT_GELU : ACT_GELU_TANH;
        set_quant(dgu_q, out_q, n->rows, 2 * n->cols);
        return hip_status(launch_gated_grad(a, n->dtype, rnd_of(out_q), reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return FP4_ERR_INTERNAL;
    }
}

}  // extern "C"
