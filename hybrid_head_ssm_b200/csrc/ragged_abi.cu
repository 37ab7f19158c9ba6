// The C entry points of ragged batches: argument checks, then one launcher each.
#include <math.h>

#include "kernels.h"

using namespace hymba;

namespace {

constexpr int kMostRows = 1 << 30;

int esz_of(int dtype) { return dtype == HYMBA_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == HYMBA_F32 || d == HYMBA_BF16 || d == HYMBA_F16; }
bool dim_ok(int d) { return d == 64 || d == 128; }
bool scale_ok(float s) { return s >= 0.f && s <= 3.0e38f; }

int check_attn(const hymba_attn_shape* s) {
    if (!s || s->n_q_heads <= 0 || s->n_kv_heads <= 0 || s->n_meta < 0 || !dtype_ok(s->dtype) || !scale_ok(s->scale))
        return HYMBA_ERR_INVALID_ARG;
    if (!dim_ok(s->head_dim) || !dim_ok(s->v_head_dim) || s->n_q_heads % s->n_kv_heads || s->n_q_heads > 1024)
        return HYMBA_ERR_UNSUPPORTED;
    return HYMBA_OK;
}
float attn_scale(const hymba_attn_shape* s) { return s->scale > 0.f ? s->scale : 1.f / sqrtf((float)s->head_dim); }

int check_linattn(const hymba_linattn_shape* s) {
    if (!s || s->n_qk_heads <= 0 || s->n_heads <= 0 || s->v_head_dim <= 0 || !dtype_ok(s->dtype) ||
        !scale_ok(s->scale))
        return HYMBA_ERR_INVALID_ARG;
    if ((s->key_dim != 16 && s->key_dim != 64 && s->key_dim != 128) || s->v_head_dim % 64 || s->v_head_dim > 512 ||
        s->n_heads % s->n_qk_heads || s->n_heads > 1024)
        return HYMBA_ERR_UNSUPPORTED;
    return HYMBA_OK;
}
float linattn_scale(const hymba_linattn_shape* s) { return s->scale > 0.f ? s->scale : 1.f / sqrtf((float)s->key_dim); }

// rows of `width` elements with stride ld: present, 16-byte aligned, no row inside another
bool rows_ok(const void* p, int64_t ld, int width, int esz) {
    return p && ((uintptr_t)p & 15) == 0 && ld >= width && ld <= ((int64_t)1 << 40) && (ld * esz) % 16 == 0;
}

int check_paged(const hymba_paged_kv* kv) {
    if (!kv || !kv->k_pages || !kv->v_pages || !kv->page_table || !kv->len || kv->n_pages <= 0 || kv->page_size <= 0 ||
        kv->max_pages <= 0 || kv->batch <= 0 || kv->n_kv_heads <= 0 || !dtype_ok(kv->dtype) ||
        (((uintptr_t)kv->k_pages | (uintptr_t)kv->v_pages) & 15) ||
        (((uintptr_t)kv->page_table | (uintptr_t)kv->len) & 3))
        return HYMBA_ERR_INVALID_ARG;
    if (!dim_ok(kv->head_dim) || !dim_ok(kv->v_head_dim) || kv->n_kv_heads > 1024 ||
        (int64_t)kv->max_pages * kv->page_size > kMostRows || kv->batch > 65535 ||
        (int64_t)kv->n_pages * kv->page_size > 0x7fffffffLL / kv->n_kv_heads)
        return HYMBA_ERR_UNSUPPORTED;
    return HYMBA_OK;
}

bool workspace_ok(const void* ws) { return ws && ((uintptr_t)ws & 255) == 0; }

}  // namespace

extern "C" {

int hymba_attn_prefill_packed(const hymba_attn_shape* shape, const void* q, int64_t ldq, const void* k, int64_t ldk,
                              const void* v, int64_t ldv, const int32_t* cu_seqlens, int n_seqs, int total_rows,
                              void* o, int64_t ldo, void* stream) {
    int rc = check_attn(shape);
    if (rc) return rc;
    if (n_seqs < 0 || n_seqs > kMostRows || total_rows < 0 || total_rows > kMostRows) return HYMBA_ERR_INVALID_ARG;
    if (n_seqs == 0 || total_rows == 0) return HYMBA_OK;
    const hymba_attn_shape& s = *shape;
    const int e = esz_of(s.dtype);
    if (!rows_ok(q, ldq, s.n_q_heads * s.head_dim, e) || !rows_ok(k, ldk, s.n_kv_heads * s.head_dim, e) ||
        !rows_ok(v, ldv, s.n_kv_heads * s.v_head_dim, e) || !rows_ok(o, ldo, s.n_q_heads * s.v_head_dim, e) ||
        !cu_seqlens || ((uintptr_t)cu_seqlens & 3))
        return HYMBA_ERR_INVALID_ARG;
    Ctx ctx;
    if ((rc = launch_context(static_cast<cudaStream_t>(stream), &ctx))) return rc;
    PackedAttn a;
    a.q = q; a.k = k; a.v = v; a.o = o;
    a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldo = ldo;
    a.cu = cu_seqlens; a.n_seqs = n_seqs; a.total = total_rows;
    a.H = s.n_q_heads; a.G = s.n_kv_heads; a.dh = s.head_dim; a.dv = s.v_head_dim;
    a.n_meta = s.n_meta; a.window = s.window;
    a.scale = attn_scale(shape);
    if (s.dtype == HYMBA_F32) return launch_attn_packed_simt<float>(ctx, a);
    if (s.dtype == HYMBA_F16) return launch_attn_packed_tc<f16>(ctx, a);
    return launch_attn_packed_tc<bf16>(ctx, a);
}

int hymba_kv_append_paged(const hymba_paged_kv* kv, const void* k, int64_t ldk, const void* v, int64_t ldv,
                          const int32_t* cu_seqlens, int total_rows, void* stream) {
    int rc = check_paged(kv);
    if (rc) return rc;
    if (total_rows < 0 || total_rows > kMostRows || (!cu_seqlens && total_rows != kv->batch))
        return HYMBA_ERR_INVALID_ARG;
    if (total_rows == 0) return HYMBA_OK;
    const int e = esz_of(kv->dtype);
    if (!rows_ok(k, ldk, kv->n_kv_heads * kv->head_dim, e) || !rows_ok(v, ldv, kv->n_kv_heads * kv->v_head_dim, e) ||
        ((uintptr_t)cu_seqlens & 3))
        return HYMBA_ERR_INVALID_ARG;
    Ctx ctx;
    if ((rc = launch_context(static_cast<cudaStream_t>(stream), &ctx))) return rc;
    return launch_kv_append(ctx, *kv, e, k, ldk, v, ldv, cu_seqlens, total_rows);
}

size_t hymba_attn_decode_paged_workspace(const hymba_attn_shape* shape, int batch, int max_len) {
    if (check_attn(shape) || batch <= 0 || batch > 65535 || max_len <= 0 || max_len > kMostRows) return 0;
    return decode_paged_bytes(*shape, batch, max_len);
}

int hymba_attn_decode_paged(const hymba_attn_shape* shape, const void* q, int64_t ldq, const hymba_paged_kv* kv,
                            int max_len, void* o, int64_t ldo, void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_attn(shape);
    if (rc) return rc;
    if ((rc = check_paged(kv))) return rc;
    const hymba_attn_shape& s = *shape;
    if (s.n_kv_heads != kv->n_kv_heads || s.head_dim != kv->head_dim || s.v_head_dim != kv->v_head_dim ||
        s.dtype != kv->dtype)
        return HYMBA_ERR_KV_INCOMPATIBLE;
    const int cap = kv->max_pages * kv->page_size;
    if (max_len < 0 || max_len > cap) return HYMBA_ERR_INVALID_ARG;
    if (max_len == 0) max_len = cap;
    const int e = esz_of(s.dtype);
    if (!rows_ok(q, ldq, s.n_q_heads * s.head_dim, e) || !rows_ok(o, ldo, s.n_q_heads * s.v_head_dim, e) ||
        !workspace_ok(workspace))
        return HYMBA_ERR_INVALID_ARG;
    if (ws_bytes < decode_paged_bytes(s, kv->batch, max_len)) return HYMBA_ERR_WORKSPACE_TOO_SMALL;
    Ctx ctx;
    if ((rc = launch_context(static_cast<cudaStream_t>(stream), &ctx))) return rc;
    return launch_decode_paged(ctx, s, attn_scale(shape), q, ldq, *kv, max_len, o, ldo, workspace);
}

static void fill(LinAttn* a, const hymba_linattn_shape& s, const void* q, int64_t ldq, const void* k, int64_t ldk,
                 const void* v, int64_t ldv, const float* g, int64_t ldg, void* o, int64_t ldo) {
    a->q = q; a->k = k; a->v = v; a->o = o; a->g = g;
    a->ldq = ldq; a->ldk = ldk; a->ldv = ldv; a->ldo = ldo; a->ldg = ldg;
    a->Hk = s.n_qk_heads; a->H = s.n_heads; a->dk = s.key_dim; a->dv = s.v_head_dim;
    a->scale = linattn_scale(&s);
}

static bool linattn_rows_ok(const hymba_linattn_shape& s, const void* q, int64_t ldq, const void* k, int64_t ldk,
                            const void* v, int64_t ldv, const float* g, int64_t ldg, const void* o, int64_t ldo) {
    const int e = esz_of(s.dtype);
    return rows_ok(q, ldq, s.n_qk_heads * s.key_dim, e) && rows_ok(k, ldk, s.n_qk_heads * s.key_dim, e) &&
           rows_ok(v, ldv, s.n_heads * s.v_head_dim, e) && rows_ok(o, ldo, s.n_heads * s.v_head_dim, e) && g &&
           ((uintptr_t)g & 3) == 0 && (ldg == 0 || ldg >= s.n_heads) && ldg <= ((int64_t)1 << 40);
}

size_t hymba_linattn_workspace(const hymba_linattn_shape* shape, int n_seqs, int total_rows) {
    if (check_linattn(shape) || n_seqs <= 0 || n_seqs > kMostRows || total_rows < 0 || total_rows > kMostRows) return 0;
    if (shape->dtype != HYMBA_F32 && total_rows > 0 && linattn_tc_applies(shape->key_dim))
        return linattn_tc_bytes(n_seqs, total_rows, shape->n_heads, shape->v_head_dim);
    return 256;
}

int hymba_linattn_prefill(const hymba_linattn_shape* shape, const void* q, int64_t ldq, const void* k, int64_t ldk,
                          const void* v, int64_t ldv, const float* g, int64_t ldg, const int32_t* cu_seqlens,
                          int n_seqs, int total_rows, const float* state_in, float* state_out, void* o, int64_t ldo,
                          void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_linattn(shape);
    if (rc) return rc;
    if (n_seqs < 0 || n_seqs > kMostRows || total_rows < 0 || total_rows > kMostRows) return HYMBA_ERR_INVALID_ARG;
    if (n_seqs == 0) return HYMBA_OK;
    if (!cu_seqlens || ((uintptr_t)cu_seqlens & 3) || (((uintptr_t)state_in | (uintptr_t)state_out) & 15) ||
        !workspace_ok(workspace))
        return HYMBA_ERR_INVALID_ARG;
    if (total_rows > 0 && !linattn_rows_ok(*shape, q, ldq, k, ldk, v, ldv, g, ldg, o, ldo)) return HYMBA_ERR_INVALID_ARG;
    if (state_in && state_out && state_in != state_out) {
        const uintptr_t n = (uintptr_t)n_seqs * shape->n_heads * shape->v_head_dim * shape->key_dim * 4;
        const uintptr_t x = (uintptr_t)state_in, y = (uintptr_t)state_out;
        if (x < y + n && y < x + n) return HYMBA_ERR_INVALID_ARG;
    }
    if (ws_bytes < hymba_linattn_workspace(shape, n_seqs, total_rows)) return HYMBA_ERR_WORKSPACE_TOO_SMALL;
    Ctx ctx;
    if ((rc = launch_context(static_cast<cudaStream_t>(stream), &ctx))) return rc;
    LinAttn a;
    fill(&a, *shape, q, ldq, k, ldk, v, ldv, g, ldg, o, ldo);
    a.state_in = state_in;
    a.state_out = state_out;
    a.ws = workspace;
    a.cu = cu_seqlens;
    a.n_seqs = n_seqs;
    a.total = total_rows;
    // (without rows only states are copied)
    if (shape->dtype == HYMBA_F32 || total_rows == 0) return launch_linattn_recurrent<float>(ctx, a);
    if (linattn_tc_applies(a.dk))
        return shape->dtype == HYMBA_F16 ? launch_linattn_tc<f16>(ctx, a) : launch_linattn_tc<bf16>(ctx, a);
    if (shape->dtype == HYMBA_F16) return launch_linattn_chunk<f16>(ctx, a);
    return launch_linattn_chunk<bf16>(ctx, a);
}

int hymba_linattn_step(const hymba_linattn_shape* shape, const void* q, int64_t ldq, const void* k, int64_t ldk,
                       const void* v, int64_t ldv, const float* g, int64_t ldg, float* state, int batch, void* o,
                       int64_t ldo, void* stream) {
    int rc = check_linattn(shape);
    if (rc) return rc;
    if (batch <= 0 || batch > kMostRows || !state || ((uintptr_t)state & 15) ||
        !linattn_rows_ok(*shape, q, ldq, k, ldk, v, ldv, g, ldg, o, ldo))
        return HYMBA_ERR_INVALID_ARG;
    Ctx ctx;
    if ((rc = launch_context(static_cast<cudaStream_t>(stream), &ctx))) return rc;
    LinAttn a;
    fill(&a, *shape, q, ldq, k, ldk, v, ldv, g, ldg, o, ldo);
    a.state_in = state;
    a.state_out = state;
    a.ws = nullptr;
    a.cu = nullptr;
    a.n_seqs = batch;
    a.total = batch;
    if (shape->dtype == HYMBA_F32) return launch_linattn_recurrent<float>(ctx, a);
    if (shape->dtype == HYMBA_F16) return launch_linattn_recurrent<f16>(ctx, a);
    return launch_linattn_recurrent<bf16>(ctx, a);
}

}  // extern "C"
