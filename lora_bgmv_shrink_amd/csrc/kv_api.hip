// C entry points of the paged key/value cache: argument checks, workspace
// layout and dispatch.  Semantics: include/lora_mi355x.h.
#include <cmath>
#include <cstring>

#include "kv_internal.hpp"

using namespace lora;

namespace {

// enum arguments may hold any int: compared as ints, taken by reference
bool dtype_ok(const lora_dtype_t& d) {
    int v = 0;
    std::memcpy(&v, &d, sizeof v);
    return v == LORA_F32 || v == LORA_BF16;
}
int elem_bytes(lora_dtype_t d) { return d == LORA_BF16 ? 2 : 4; }
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool ld16(int64_t ld, int eb) { return ld % (16 / eb) == 0; }
lora_status_t dev_status(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_E_DEVICE; }

constexpr int64_t kMost = (int64_t)1 << 30;   // rows, lengths, columns and table widths

lora_status_t check_cache(const lora_kv_cache_t* c, KvDev& C) {
    if (!c || !dtype_ok(c->dtype) || !c->k || !c->v) return LORA_E_INVALID;
    if (c->n_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0) return LORA_E_INVALID;
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return LORA_E_INVALID;
    const bool dim_ok = c->head_dim == 64 || c->head_dim == 128 || (c->head_dim == 256 && c->dtype == LORA_BF16);
    if (!dim_ok || (c->page_size & (c->page_size - 1)) != 0 || c->page_size > (1 << 20)) return LORA_E_UNSUPPORTED;
    const int eb = elem_bytes(c->dtype);
    if (!al16(c->k) || !al16(c->v) || !ld16(c->page_stride, eb) || !ld16(c->token_stride, eb) ||
        !ld16(c->head_stride, eb))
        return LORA_E_UNSUPPORTED;
    if (c->token_stride >= kMost / c->page_size) return LORA_E_UNSUPPORTED;   // offsets in a page are 32-bit
    C.k = c->k;
    C.v = c->v;
    C.page_stride = c->page_stride;
    C.token_stride = c->token_stride;
    C.head_stride = c->head_stride;
    C.n_pages = c->n_pages;
    C.page_shift = __builtin_ctz((unsigned)c->page_size);
    C.n_kv_heads = c->n_kv_heads;
    return LORA_OK;
}

lora_status_t check_batch(const lora_kv_batch_t* b, KvBatchDev& B) {
    if (!b || b->n_seqs < 0 || b->n_rows < 0 || b->n_groups < 0) return LORA_E_INVALID;
    if (b->n_seqs == 0 && b->n_rows > 0) return LORA_E_INVALID;
    if (b->max_rows < 0 || b->max_kv_len < 0 || b->ldp < 0 || b->max_group_rows < 0 || b->max_prefix_len < 0 ||
        b->ldpp < 0)
        return LORA_E_INVALID;
    // a table of no columns is never read, and may have no address
    if (b->n_seqs > 0 && (!b->row_off || !b->kv_len || (!b->pages && b->ldp > 0) || !al4(b->row_off) ||
                          !al4(b->kv_len) || !al4(b->pages)))
        return LORA_E_INVALID;
    if (b->n_groups > 0 && (!b->group_off || !b->prefix_len || (!b->prefix_pages && b->ldpp > 0) ||
                            !al4(b->group_off) || !al4(b->prefix_len) || !al4(b->prefix_pages)))
        return LORA_E_INVALID;
    if (b->n_rows > kMost || b->n_seqs > kMost || b->max_kv_len > kMost || b->max_prefix_len > kMost || b->ldp > kMost ||
        b->ldpp > kMost)
        return LORA_E_UNSUPPORTED;
    B.row_off = b->row_off;
    B.kv_len = b->kv_len;
    B.pages = b->pages;
    B.ldp = b->ldp;
    B.n_seqs = b->n_seqs;
    B.n_rows = b->n_rows;
    B.group_off = b->group_off;
    B.prefix_len = b->prefix_len;
    B.prefix_pages = b->prefix_pages;
    B.ldpp = b->ldpp;
    B.n_groups = b->n_groups;
    return LORA_OK;
}

// The attention's plan: everything but the tensors and the workspace's address.
lora_status_t make_plan(const lora_kv_cache_t* cache, const lora_kv_batch_t* batch, int32_t n_q_heads, int32_t window,
                        int32_t n_sink, bool groups, AttnPlan& P) {
    std::memset(&P, 0, sizeof P);
    lora_status_t st = check_cache(cache, P.a.C);
    if (st != LORA_OK) return st;
    st = check_batch(batch, P.a.B);
    if (st != LORA_OK) return st;
    if (n_q_heads <= 0 || n_q_heads % cache->n_kv_heads != 0 || window < 0 || n_sink < 0) return LORA_E_INVALID;
    if (groups != (batch->n_groups > 0)) return LORA_E_INVALID;
    if ((int64_t)batch->n_rows * n_q_heads > kMost || (int64_t)batch->n_seqs * cache->n_kv_heads > kMost ||
        (int64_t)batch->n_groups * cache->n_kv_heads > kMost)
        return LORA_E_UNSUPPORTED;
    P.a.n_q_heads = n_q_heads;
    P.a.share = n_q_heads / cache->n_kv_heads;
    P.a.window = window < kMost ? window : 0;   // no length reaches it
    P.a.n_sink = n_sink < kMost ? n_sink : (int32_t)kMost;
    const int32_t n_prob[2] = {batch->n_seqs, batch->n_groups};
    const int32_t rows[2] = {std::min(batch->max_rows, batch->n_rows), std::min(batch->max_group_rows, batch->n_rows)};
    const int32_t len[2] = {batch->max_kv_len, batch->max_prefix_len};
    plan_attn(P, cache->head_dim, elem_bytes(cache->dtype), n_prob, rows, len);
    return LORA_OK;
}

lora_status_t run_attn(const lora_kv_cache_t* cache, const lora_kv_batch_t* batch, const void* q, int64_t ldq,
                       int32_t n_q_heads, float scale, int32_t window, int32_t n_sink, bool groups, void* o,
                       const lora_dtype_t& o_dtype, int64_t ldo, float* lse, int32_t* status, void* ws, size_t ws_bytes,
                       hipStream_t stream) {
    AttnPlan P;
    const lora_status_t st = make_plan(cache, batch, n_q_heads, window, n_sink, groups, P);
    if (st != LORA_OK) return st;
    if (!dtype_ok(o_dtype) || !(scale > 0.f) || !std::isfinite(scale)) return LORA_E_INVALID;
    if (batch->n_rows == 0) return LORA_OK;
    const int64_t width = (int64_t)n_q_heads * cache->head_dim;
    if (!q || !o || ldq < width || ldo < width) return LORA_E_INVALID;
    if (!al16(q) || !al16(o) || !ld16(ldq, elem_bytes(cache->dtype)) || !ld16(ldo, elem_bytes(o_dtype)) || !al4(lse) ||
        !al4(status))
        return LORA_E_UNSUPPORTED;
    if (P.bytes > 0 && (!ws || !al16(ws) || ws_bytes < P.bytes)) return LORA_E_WORKSPACE;
    AttnArgs& a = P.a;
    a.q = q;
    a.ldq = ldq;
    a.scale = scale;
    a.o = o;
    a.ldo = ldo;
    a.o_bf16 = o_dtype == LORA_BF16 ? 1 : 0;
    a.lse = lse;
    a.status = status;
    uint8_t* w = (uint8_t*)ws;
    for (int k = 0; k < 2; ++k) {
        AttnPart& W = a.part[k];
        W.rec = (int2*)(w + P.off[k][0]);
        W.few_o = (float*)(w + P.off[k][1]);
        W.few_ml = (float2*)(w + P.off[k][2]);
        W.item = (int4*)(w + P.off[k][3]);
        W.tile_o = (float*)(w + P.off[k][4]);
        W.tile_ml = (float2*)(w + P.off[k][5]);
        W.row_o = (float*)(w + P.off[k][6]);
        W.row_ml = (float2*)(W.row_o + (size_t)batch->n_rows * width);
    }
    return dev_status(launch_attn(a, cache->dtype, cache->head_dim, stream));
}

}  // namespace

extern "C" {

lora_status_t lora_kv_append(const lora_kv_cache_t* cache, const lora_kv_batch_t* batch, const lora_rope_t* rope,
                             lora_dtype_t dtype, const void* q, int64_t ldq, int32_t n_q_heads, const void* k,
                             int64_t ldk, const void* v, int64_t ldv, void* q_out, int64_t ldqo, int32_t* status,
                             hipStream_t stream) {
    AppendArgs a;
    std::memset(&a, 0, sizeof a);
    lora_status_t st = check_cache(cache, a.C);
    if (st != LORA_OK) return st;
    st = check_batch(batch, a.B);
    if (st != LORA_OK) return st;
    if (!dtype_ok(dtype) || n_q_heads < 0) return LORA_E_INVALID;
    const int ei = elem_bytes(dtype), eo = elem_bytes(cache->dtype), d = cache->head_dim;
    if (rope) {
        if (!rope->cos || !rope->sin || rope->n_pos <= 0 || rope->rot_dim <= 0 || rope->rot_dim > d ||
            rope->ld < rope->rot_dim / 2)
            return LORA_E_INVALID;
        if (rope->rot_dim % 16 != 0 || !al16(rope->cos) || !al16(rope->sin) || rope->ld % 4 != 0)
            return LORA_E_UNSUPPORTED;
        a.cos = rope->cos;
        a.sin = rope->sin;
        a.ldr = rope->ld;
        a.n_pos = rope->n_pos;
        a.half = rope->rot_dim / 2;
        a.interleaved = rope->interleaved ? 1 : 0;
    }
    if (batch->n_rows == 0) return LORA_OK;
    const int64_t wq = (int64_t)n_q_heads * d, wk = (int64_t)cache->n_kv_heads * d;
    if (!k || !v || ldk < wk || ldv < wk) return LORA_E_INVALID;
    if (n_q_heads > 0 && (!q || !q_out || ldq < wq || ldqo < wq)) return LORA_E_INVALID;
    if (!al16(k) || !al16(v) || !ld16(ldk, ei) || !ld16(ldv, ei) || !al4(status)) return LORA_E_UNSUPPORTED;
    if (n_q_heads > 0 && (!al16(q) || !al16(q_out) || !ld16(ldq, ei) || !ld16(ldqo, eo))) return LORA_E_UNSUPPORTED;
    if (wq + 2 * wk > kMost) return LORA_E_UNSUPPORTED;
    a.q = q;
    a.ldq = ldq;
    a.k = k;
    a.ldk = ldk;
    a.v = v;
    a.ldv = ldv;
    a.n_q_heads = n_q_heads;
    a.q_out = q_out;
    a.ldqo = ldqo;
    a.status = status;
    return dev_status(launch_kv_append(a, dtype, cache->dtype, d, stream));
}

lora_status_t lora_attn_workspace(const lora_kv_cache_t* cache, const lora_kv_batch_t* batch, int32_t n_q_heads,
                                  size_t* bytes) {
    if (!bytes) return LORA_E_INVALID;
    AttnPlan P;
    const lora_status_t st = make_plan(cache, batch, n_q_heads, 0, 0, batch && batch->n_groups > 0, P);
    if (st == LORA_OK) *bytes = P.bytes;
    return st;
}

lora_status_t lora_attn_paged(const lora_kv_cache_t* cache, const lora_kv_batch_t* batch, const void* q, int64_t ldq,
                              int32_t n_q_heads, float scale, int32_t window, int32_t n_sink, void* o,
                              lora_dtype_t o_dtype, int64_t ldo, float* lse, int32_t* status, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
    return run_attn(cache, batch, q, ldq, n_q_heads, scale, window, n_sink, false, o, o_dtype, ldo, lse, status, ws,
                    ws_bytes, stream);
}

lora_status_t lora_attn_prefix(const lora_kv_cache_t* cache, const lora_kv_batch_t* batch, const void* q, int64_t ldq,
                               int32_t n_q_heads, float scale, int32_t window, int32_t n_sink, void* o,
                               lora_dtype_t o_dtype, int64_t ldo, float* lse, int32_t* status, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
    return run_attn(cache, batch, q, ldq, n_q_heads, scale, window, n_sink, true, o, o_dtype, ldo, lse, status, ws,
                    ws_bytes, stream);
}

}  // extern "C"
