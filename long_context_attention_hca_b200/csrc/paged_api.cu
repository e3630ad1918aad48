// paged_api.cu -- extern "C" entry points of the paged calls: argument
// validation on the host, then the launch.  See include/hca.h.
#include <cmath>

#include "paged_attention.cuh"

namespace hca {

int page_plan_launch(const int32_t* ctx, const int32_t* nnew, int B, int m, int P, int32_t* table, int width,
                     const int32_t* free_pages, const int32_t* free_count, int free_cap, int64_t max_rows,
                     int32_t* row_start, int32_t* row_req, int32_t* row_pos, int64_t* slot, int32_t* missing,
                     int32_t* free_left, cudaStream_t st);
int page_store_launch(const uint16_t* x, int64_t n_rows, const int32_t* n_live, const int32_t* pos,
                      const int64_t* slot, const hca_kv_layout& L, const hca_entry_extras* ex, uint16_t* pages,
                      int64_t n_slots, cudaStream_t st);
int page_compress_launch(int m, const uint16_t* x, const uint16_t* gate, int64_t n_tok, const int32_t* tok_start,
                         const int32_t* ctx, int B, const float* bias, const int32_t* ent_start, const int32_t* ent_req,
                         const int32_t* ent_pos, const int64_t* ent_slot, int64_t max_ent, uint16_t* tail_x,
                         uint16_t* tail_gate, const hca_kv_layout& L, const hca_kv_cache& pool, int64_t n_slots,
                         const hca_entry_extras* ex, cudaStream_t st);
size_t paged_attn_ws_bytes(int64_t n_rows, int B, int H, int D, int64_t max_new, int64_t max_entries, int W, int n_first);
int paged_attn_launch(paged::Params p, int D, int64_t max_new, int64_t max_entries, void* ws, size_t ws_bytes,
                      cudaStream_t st);

namespace {

#define REQUIRE(cond) do { if (!(cond)) return HCA_ERR_INVALID_ARG; } while (0)
#define REQ_PTR(p) REQUIRE((p) != nullptr && aligned16(p))
// integer arrays (lengths, tables, slots) are read one element at a time: their own alignment
#define REQ_INT(p) REQUIRE((p) != nullptr && (reinterpret_cast<uintptr_t>(p) & (sizeof(*(p)) - 1)) == 0)

bool layout_ok(const hca_kv_layout& L) {
    return (L.d == 512 && L.d_rope == 64 && L.scale_group == 64) ||
           (L.d == 128 && L.d_rope == 32 && L.scale_group == 32);
}

bool opt_ok(const void* p) { return p == nullptr || aligned16(p); }

bool entry_extras_ok(const hca_entry_extras* ex) {
    return !ex || (opt_ok(ex->norm_w) && opt_ok(ex->inv_freq) && ex->norm_eps >= 0.0f);
}

bool map_ok(const hca_page_map& m) {
    return m.page_size >= 1 && m.width >= 0 && m.pages >= 0 && (m.width == 0 || (m.table && (reinterpret_cast<uintptr_t>(m.table) & 3u) == 0));
}

int attn_common(const uint16_t* q, int64_t n_rows, int32_t H, int32_t B, const int32_t* row_start,
                const int32_t* ctx_len, int64_t max_new, int32_t m, const hca_kv_layout& L, const hca_kv_cache* pool,
                const hca_page_map* emap, const uint16_t* pages, const hca_page_map& tmap, int32_t W, int32_t n_first,
                float scale, const hca_attn_extras* ex, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
    REQUIRE(n_rows >= 0 && B >= 0 && max_new >= 0);
    if (!layout_ok(L)) return HCA_ERR_UNSUPPORTED;
    if (H < 1 || H > 128 || W < 1 || W > 4096 || n_first < 0 || n_first > 4096) return HCA_ERR_UNSUPPORTED;
    if (n_rows * H > 0x7FFFFFFFLL - 0x10000) return HCA_ERR_UNSUPPORTED;
    REQUIRE(std::isfinite(scale) && scale > 0.0f);
    if (n_rows == 0 || B == 0) return HCA_OK;
    REQ_PTR(q); REQ_PTR(out); REQ_INT(row_start); REQ_INT(ctx_len);
    REQUIRE(map_ok(tmap));
    if (tmap.pages > 0) REQ_PTR(pages);
    paged::Params p = {};
    if (pool) {
        REQUIRE(m >= 1 && map_ok(*emap));
        if (emap->pages > 0) { REQ_PTR(pool->codes); REQ_PTR(pool->scales); REQ_PTR(pool->rope); }
        REQUIRE(static_cast<int64_t>(emap->width) * emap->page_size <= 0x7FFFFFFFLL - 0x10000);
        p.m = m;
        p.codes = pool->codes; p.scales = pool->scales; p.rope = pool->rope;
        p.e_pages = emap->pages; p.e_size = emap->page_size; p.e_table = emap->table; p.e_width = emap->width;
    }
    if (ex) {
        REQUIRE(opt_ok(ex->q_norm_w) && opt_ok(ex->sink) && opt_ok(ex->inv_freq) && ex->norm_eps >= 0.0f);
        REQUIRE(ex->q_pos == nullptr && ex->win_len == nullptr);
        p.q_norm_w = ex->q_norm_w; p.norm_eps = ex->norm_eps; p.sink = ex->sink; p.inv_freq = ex->inv_freq;
    }
    if (ws) REQUIRE(aligned16(ws));
    p.q = q; p.n_rows = n_rows; p.H = H; p.B = B; p.row_start = row_start; p.ctx = ctx_len;
    p.tok = pages; p.t_pages = tmap.pages; p.t_size = tmap.page_size; p.t_table = tmap.table; p.t_width = tmap.width;
    p.W = W; p.n_first = n_first;
    p.scale_log2 = scale * paged::LOG2E;
    p.out = out;
    const int64_t max_entries = pool ? static_cast<int64_t>(emap->width) * emap->page_size : 0;
    return paged_attn_launch(p, L.d, max_new > 0 && max_new < n_rows ? max_new : n_rows, max_entries, ws, ws_bytes,
                             as_stream(stream));
}

}  // namespace
}  // namespace hca

using namespace hca;

extern "C" {

int kv_page_plan(const int32_t* ctx_len, const int32_t* new_len, int32_t B, int32_t m, int32_t page_size,
                 int32_t* table, int32_t width, const int32_t* free_pages, const int32_t* free_count,
                 int32_t free_cap, int64_t max_rows, int32_t* row_start, int32_t* row_req, int32_t* row_pos,
                 int64_t* slot, int32_t* missing, int32_t* free_left, void* stream) {
    REQUIRE(B >= 0 && m >= 1 && page_size >= 1 && width >= 0 && free_cap >= 0 && max_rows >= 0);
    if (B > 16384) return HCA_ERR_UNSUPPORTED;
    REQ_INT(row_start); REQ_INT(free_count); REQ_INT(missing); REQ_INT(free_left);
    REQUIRE(free_count != free_left);
    if (B > 0) { REQ_INT(ctx_len); REQ_INT(new_len); if (width > 0) REQ_INT(table); }
    if (free_cap > 0) REQ_INT(free_pages);
    if (max_rows > 0) { REQ_INT(row_req); REQ_INT(row_pos); REQ_INT(slot); }
    return page_plan_launch(ctx_len, new_len, B, m, page_size, table, width, free_pages, free_count, free_cap, max_rows,
                            row_start, row_req, row_pos, slot, missing, free_left, as_stream(stream));
}

int kv_page_store(const uint16_t* x, int64_t n_rows, const int32_t* n_live, const int32_t* row_pos,
                  const int64_t* slot, hca_kv_layout layout, const hca_entry_extras* ex, uint16_t* pages,
                  int64_t n_slots, void* stream) {
    REQUIRE(n_rows >= 0 && n_slots >= 0);
    if (!layout_ok(layout)) return HCA_ERR_UNSUPPORTED;
    if (n_rows > 0x7FFFFFFFLL) return HCA_ERR_UNSUPPORTED;
    if (n_rows == 0 || n_slots == 0) return HCA_OK;
    REQ_PTR(x); REQ_INT(row_pos); REQ_INT(slot); REQ_PTR(pages);
    REQ_INT(n_live);
    REQUIRE(entry_extras_ok(ex));
    return page_store_launch(x, n_rows, n_live, row_pos, slot, layout, ex, pages, n_slots, as_stream(stream));
}

int kv_page_compress(int32_t m, const uint16_t* x, const uint16_t* gate, int64_t n_tokens,
                     const int32_t* tok_start, const int32_t* ctx_len, int32_t B, const float* pos_bias,
                     const int32_t* ent_start, const int32_t* ent_req, const int32_t* ent_pos,
                     const int64_t* ent_slot, int64_t max_entries, uint16_t* tail_x, uint16_t* tail_gate,
                     hca_kv_layout layout, hca_kv_cache pool, int64_t n_slots, const hca_entry_extras* ex,
                     void* stream) {
    REQUIRE(n_tokens >= 0 && B >= 0 && max_entries >= 0 && n_slots >= 0);
    if (!layout_ok(layout) || (m != 4 && m != 128)) return HCA_ERR_UNSUPPORTED;
    if (n_tokens > 0x7FFFFFFFLL || max_entries + B > 0x7FFFFFFFLL / 8) return HCA_ERR_UNSUPPORTED;
    if (n_tokens == 0 || B == 0) return HCA_OK;
    REQ_PTR(x); REQ_PTR(gate); REQ_INT(tok_start); REQ_INT(ctx_len); REQ_PTR(pos_bias); REQ_INT(ent_start);
    REQ_PTR(tail_x); REQ_PTR(tail_gate);
    if (max_entries > 0) { REQ_INT(ent_req); REQ_INT(ent_pos); REQ_INT(ent_slot); }
    if (n_slots > 0) { REQ_PTR(pool.codes); REQ_PTR(pool.scales); REQ_PTR(pool.rope); }
    REQUIRE(entry_extras_ok(ex));
    return page_compress_launch(m, x, gate, n_tokens, tok_start, ctx_len, B, pos_bias, ent_start, ent_req, ent_pos,
                                ent_slot, max_entries, tail_x, tail_gate, layout, pool, n_slots, ex, as_stream(stream));
}

size_t paged_attn_workspace_size(int64_t n_rows, int32_t B, int32_t H, hca_kv_layout layout, int64_t max_new,
                                 int64_t max_entries, int32_t W, int32_t n_first) {
    if (n_rows <= 0 || B <= 0 || !layout_ok(layout) || H < 1 || H > 128 || max_new < 0 || max_entries < 0 || W < 1 ||
        W > 4096 || n_first < 0 || n_first > 4096 || n_rows * H > 0x7FFFFFFFLL - 0x10000)
        return 0;
    return paged_attn_ws_bytes(n_rows, B, H, layout.d, max_new > 0 && max_new < n_rows ? max_new : n_rows, max_entries, W,
                               n_first);
}

int paged_attn_chunk(const uint16_t* q, int64_t n_rows, int32_t H, int32_t B, const int32_t* row_start,
                     const int32_t* ctx_len, int64_t max_new, int32_t m, hca_kv_layout layout, hca_kv_cache pool,
                     hca_page_map entry_map, const uint16_t* pages, hca_page_map token_map, int32_t W,
                     float softmax_scale, const hca_attn_extras* ex, uint16_t* out, void* ws, size_t ws_bytes,
                     void* stream) {
    return attn_common(q, n_rows, H, B, row_start, ctx_len, max_new, m, layout, &pool, &entry_map, pages, token_map, W, 0,
                       softmax_scale, ex, out, ws, ws_bytes, stream);
}

int paged_attn_window(const uint16_t* q, int64_t n_rows, int32_t H, int32_t B, const int32_t* row_start,
                      const int32_t* ctx_len, int64_t max_new, hca_kv_layout layout, const uint16_t* pages,
                      hca_page_map token_map, int32_t W, int32_t n_first, float softmax_scale,
                      const hca_attn_extras* ex, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
    return attn_common(q, n_rows, H, B, row_start, ctx_len, max_new, 0, layout, nullptr, nullptr, pages, token_map, W,
                       n_first, softmax_scale, ex, out, ws, ws_bytes, stream);
}

}  // extern "C"
