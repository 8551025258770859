// jano_api.cu -- the exported C ABI of libjano: argument validation on the
// host, then one or more asynchronous launches on the caller's stream.  See
// include/jano.h for the contract of each entry point.
#include <cmath>
#include <cstdint>
#include <climits>

#include "jano_common.cuh"

namespace jano {

__device__ int g_device_error = JANO_OK;

int* device_error_word() {
    // cached per device; several host threads may fill a slot, all with the
    // same address
    static std::atomic<int*> addr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    int* a = addr[dev].load(std::memory_order_acquire);
    if (!a) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
        a = static_cast<int*>(p);
        addr[dev].store(a, std::memory_order_release);
    }
    return a;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

jano_status from_cuda(cudaError_t e) { return e == cudaSuccess ? JANO_OK : JANO_ECUDA; }

jano_status check_geom(const jano_geom* g, bool need_patch) {
    if (!g) return JANO_EINVAL;
    if (g->F < 1 || g->H < 1 || g->W < 1 || g->bf < 1 || g->bh < 1 || g->bw < 1)
        return JANO_EINVAL;
    if (need_patch) {
        if (g->pf < 1 || g->ph < 1 || g->pw < 1) return JANO_EINVAL;
        if (g->F % g->pf || g->H % g->ph || g->W % g->pw) return JANO_ESHAPE;
        const long long nt = (long long)(g->F / g->pf) * (g->H / g->ph) * (g->W / g->pw);
        if (nt > INT_MAX) return JANO_EUNSUPPORTED;
    }
    const long long nb = (long long)((g->F + g->bf - 1) / g->bf) * ((g->H + g->bh - 1) / g->bh) *
                         ((g->W + g->bw - 1) / g->bw);
    if (nb > INT_MAX) return JANO_EUNSUPPORTED;
    return JANO_OK;
}

}  // namespace
}  // namespace jano

using namespace jano;

extern "C" {

namespace {
jano_status block_scores_impl(const float* lat, int K, int C, const jano_geom* g, float w_temporal,
                              float w_spatial, bool literal, float* scores, void* stream) {
    if (!lat || !scores) return JANO_EINVAL;
    if (K < 2 || C < 1) return JANO_EINVAL;
    if (!std::isfinite(w_temporal) || !std::isfinite(w_spatial)) return JANO_EINVAL;
    const jano_status gs = check_geom(g, false);
    if (gs != JANO_OK) return gs;
    if (g->W % 4) return JANO_EUNSUPPORTED;
    if (!aligned16(lat)) return JANO_EALIGN;
    if (!analyzer_supported(*g, K, C, literal)) return JANO_EUNSUPPORTED;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_block_scores(lat, K, C, *g, w_temporal, w_spatial, literal, scores, err,
                                         static_cast<cudaStream_t>(stream)));
}
}  // namespace

jano_status jano_block_scores(const float* lat, int K, int C, const jano_geom* g,
                              float w_temporal, float w_spatial, float* scores,
                              void* stream) {
    return block_scores_impl(lat, K, C, g, w_temporal, w_spatial, false, scores, stream);
}

jano_status jano_block_scores_literal(const float* lat, int K, int C, const jano_geom* g,
                                      float w_temporal, float w_spatial, float* scores,
                                      void* stream) {
    return block_scores_impl(lat, K, C, g, w_temporal, w_spatial, true, scores, stream);
}

jano_status jano_classify(const float* scores, int n_blocks, float frac_active,
                          float frac_static, uint8_t* levels, void* stream) {
    if (!scores || !levels || n_blocks < 1) return JANO_EINVAL;
    if (!(frac_active >= 0.0f && frac_active <= 1.0f) || !(frac_static >= 0.0f && frac_static <= 1.0f))
        return JANO_EINVAL;
    const long long bpA = std::llround((double)frac_active * 10000.0);
    const long long bpS = std::llround((double)frac_static * 10000.0);
    if (bpA + bpS > 10000) return JANO_EINVAL;
    const long long nA = bpA * n_blocks / 10000;
    const long long nS = bpS * n_blocks / 10000;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_classify(scores, n_blocks, nS, (long long)n_blocks - nA, levels, err,
                                     static_cast<cudaStream_t>(stream)));
}

size_t jano_build_schedule_workspace_bytes(const jano_geom* g) {
    if (check_geom(g, true) != JANO_OK) return 0;
    return schedule_workspace_bytes(*g);
}

jano_status jano_build_schedule(const uint8_t* block_levels, const jano_geom* g,
                                const jano_sched_cfg* c, int32_t* offsets, int32_t* idx,
                                size_t idx_capacity, uint8_t* token_levels, void* workspace,
                                size_t ws_bytes, void* stream) {
    if (!block_levels || !c || !offsets || !idx || !workspace) return JANO_EINVAL;
    const jano_status gs = check_geom(g, true);
    if (gs != JANO_OK) return gs;
    if (c->T < 1 || c->warmup < 0 || c->cooldown < 0 || c->warmup + c->cooldown > c->T ||
        c->period_moderate < 1 || c->period_static < 1)
        return JANO_EINVAL;
    if (c->T > 65535) return JANO_EUNSUPPORTED;
    const long long nt = (long long)(g->F / g->pf) * (g->H / g->ph) * (g->W / g->pw);
    if (nt * c->T > INT_MAX) return JANO_EUNSUPPORTED;
    if (idx_capacity < (size_t)(nt * c->T)) return JANO_EINVAL;
    if (ws_bytes < schedule_workspace_bytes(*g)) return JANO_EINVAL;
    if (!aligned16(workspace)) return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_build_schedule(block_levels, *g, *c, offsets, idx, token_levels,
                                           workspace, err, static_cast<cudaStream_t>(stream)));
}

jano_status jano_kv_scatter(const void* k_act, const void* v_act, const int32_t* idx, int n_act,
                            int heads, int d, void* k_cache, void* v_cache, int n_tokens,
                            void* stream) {
    if (n_act < 0 || heads < 1 || d < 1 || n_tokens < 1) return JANO_EINVAL;
    if (n_act == 0) return JANO_OK;
    if (!k_act || !v_act || !idx || !k_cache || !v_cache) return JANO_EINVAL;
    const long long row_bytes = (long long)heads * d * 2;
    if (row_bytes % 16) return JANO_EUNSUPPORTED;
    if (row_bytes > INT_MAX) return JANO_EUNSUPPORTED;
    if (!aligned16(k_act) || !aligned16(v_act) || !aligned16(k_cache) || !aligned16(v_cache))
        return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_kv_scatter(k_act, v_act, idx, n_act, (int)row_bytes, k_cache, v_cache,
                                       n_tokens, err, static_cast<cudaStream_t>(stream)));
}

jano_status jano_active_attention(const void* q_act, const void* k_cache, const void* v_cache,
                                  const int32_t* idx, int n_act, int n_tokens, int heads, int d,
                                  float scale, void* out, void* stream) {
    if (n_act < 0 || n_tokens < 1 || heads < 1) return JANO_EINVAL;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return JANO_EINVAL;
    if (d != 64 && d != 128) return JANO_EUNSUPPORTED;
    if (heads > 65535) return JANO_EUNSUPPORTED;
    if (n_act == 0) return JANO_OK;
    if (!q_act || !k_cache || !v_cache || !idx || !out) return JANO_EINVAL;
    if (!aligned16(q_act) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_active_attention(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads,
                                             d, scale, out, err, static_cast<cudaStream_t>(stream)));
}

jano_status jano_active_attention_split(const void* q_act, const void* k_cache, const void* v_cache,
                                        const int32_t* idx, int n_act, int n_tokens, int heads, int d,
                                        float scale, int n_split, void* workspace, size_t ws_bytes,
                                        void* out, void* stream) {
    if (n_act < 0 || n_tokens < 1 || heads < 1) return JANO_EINVAL;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return JANO_EINVAL;
    if (d != 64 && d != 128) return JANO_EUNSUPPORTED;
    if (heads > 65535) return JANO_EUNSUPPORTED;
    if (n_split < 1 || n_split > attention_key_tiles(n_tokens) || n_split > 65535) return JANO_EINVAL;
    if (n_split == 1)
        return jano_active_attention(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads, d, scale,
                                     out, stream);
    if (n_act == 0) return JANO_OK;
    if (!workspace || ws_bytes < attention_workspace_bytes(n_act, heads, d, n_split)) return JANO_EINVAL;
    if (!aligned16(workspace)) return JANO_EALIGN;
    if (!q_act || !k_cache || !v_cache || !idx || !out) return JANO_EINVAL;
    if (!aligned16(q_act) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_active_attention(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads, d,
                                             scale, out, err, static_cast<cudaStream_t>(stream),
                                             n_split, workspace));
}

size_t jano_active_attention_workspace_bytes(int n_act, int heads, int d, int n_split) {
    if (n_act <= 0 || heads <= 0 || d <= 0 || n_split <= 1) return 0;
    return attention_workspace_bytes(n_act, heads, d, n_split);
}

int jano_active_attention_splits_on(int n_act, int n_tokens, int heads, int d, int sm_count) {
    if (n_act <= 0 || n_tokens < 1 || heads < 1 || (d != 64 && d != 128) || sm_count < 1) return 1;
    return attention_split_count(n_act, n_tokens, heads, sm_count);
}

int jano_active_attention_splits(int n_act, int n_tokens, int heads, int d) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return jano_active_attention_splits_on(n_act, n_tokens, heads, d, sms);
}

jano_status jano_gather_gemm(const void* x, int n_x, const int32_t* gather, int m, const void* w,
                             int n, int k, const int32_t* scatter, void* out, int n_out,
                             void* stream) {
    if (n_x < 1 || m < 0 || n < 1 || k < 1 || n_out < 1) return JANO_EINVAL;
    if (m == 0) return JANO_OK;
    if (!x || !w || !out) return JANO_EINVAL;
    if (!gather && m > n_x) return JANO_ESHAPE;
    if (!scatter && m > n_out) return JANO_ESHAPE;
    if (k % 8 || n % 8) return JANO_EUNSUPPORTED;
    if (!aligned16(x) || !aligned16(w) || !aligned16(out)) return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    ProjSeg seg{out, scatter, n, n_out};
    return from_cuda(launch_projection(x, n_x, gather, m, w, n, k, 1, &seg, err,
                                       static_cast<cudaStream_t>(stream)));
}

jano_status jano_qkv_project(const void* x, int n_tokens, const int32_t* idx, int n_act,
                             const void* w_qkv, int hd, int k, void* q_act, void* k_cache,
                             void* v_cache, void* stream) {
    if (n_tokens < 1 || n_act < 0 || hd < 1 || k < 1) return JANO_EINVAL;
    if (n_act == 0) return JANO_OK;
    if (!x || !idx || !w_qkv || !q_act || !k_cache || !v_cache) return JANO_EINVAL;
    if (k % 8 || projection_tile_n(3 * hd, hd, 3) == 0) return JANO_EUNSUPPORTED;
    if (3ll * hd > INT_MAX) return JANO_EUNSUPPORTED;
    if (!aligned16(x) || !aligned16(w_qkv) || !aligned16(q_act) || !aligned16(k_cache) ||
        !aligned16(v_cache))
        return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    const ProjSeg segs[3] = {{q_act, nullptr, hd, n_act}, {k_cache, idx, hd, n_tokens},
                             {v_cache, idx, hd, n_tokens}};
    return from_cuda(launch_projection(x, n_tokens, idx, n_act, w_qkv, 3 * hd, k, 3, segs, err,
                                       static_cast<cudaStream_t>(stream)));
}

jano_status jano_random_scores(int n_blocks, uint64_t seed, float* scores, void* stream) {
    if (n_blocks < 1 || !scores) return JANO_EINVAL;
    return from_cuda(launch_random_scores(n_blocks, seed, scores, static_cast<cudaStream_t>(stream)));
}

jano_status jano_fft_scores(const float* x, int C, const jano_geom* g, int cutoff, float* scores,
                            void* stream) {
    if (!x || !scores || C < 1 || cutoff < 0) return JANO_EINVAL;
    const jano_status gs = check_geom(g, false);
    if (gs != JANO_OK) return gs;
    if ((long long)C * g->F * g->H * g->W > (1ll << 40)) return JANO_EUNSUPPORTED;
    if (!fft_scores_supported(*g)) return JANO_EUNSUPPORTED;
    return from_cuda(launch_fft_scores(x, C, *g, cutoff, scores, static_cast<cudaStream_t>(stream)));
}

jano_status jano_stream_sum(const float* x, long long n, float* partial, int n_partial, void* stream) {
    if (n < 0 || n % 4 || n_partial < 1 || n_partial > 65535 || !partial) return JANO_EINVAL;
    if (n > 0 && !x) return JANO_EINVAL;
    if (!aligned16(x) || !aligned16(partial)) return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_stream_sum(x, n, partial, n_partial, err, static_cast<cudaStream_t>(stream)));
}

namespace {
jano_status check_rope(const jano_rope_cfg* c, int d, bool have_coords) {
    if (!c) return JANO_EINVAL;
    long long rot = 0, entries = 0;
    for (int x = 0; x < 3; ++x) {
        if (c->axes[x] < 0 || c->axes[x] % 2 || c->n_pos[x] < 1) return JANO_EINVAL;
        rot += c->axes[x];
        entries += (long long)c->n_pos[x] * (c->axes[x] / 2);
    }
    if (rot < 1 || rot > d) return JANO_EINVAL;
    if (!have_coords && (c->grid_h < 1 || c->grid_w < 1)) return JANO_EINVAL;
    if (entries > INT_MAX / 2 || (c->halves && rot % 16)) return JANO_EUNSUPPORTED;
    return JANO_OK;
}

// A row buffer: rows of `width` elements, ld apart.
jano_status check_rows(const void* p, long long ld, long long width) {
    if (!p) return JANO_EINVAL;
    if (ld < width) return JANO_ESHAPE;
    if (ld % 8) return JANO_EUNSUPPORTED;
    return aligned16(p) ? JANO_OK : JANO_EALIGN;
}

bool head_dim_ok(int d) { return d % 8 == 0 && d <= 1024; }

jano_status check_pool(const jano_page_pool* p, const jano_page_seqs* s) {
    if (!p || !s || !p->k || !p->v || !s->page_table || !s->seq_lens || !s->cu_rows) return JANO_EINVAL;
    if (p->n_pages < 1 || p->kv_heads < 1 || p->d < 1 || s->n_seqs < 1 || s->max_pages < 1) return JANO_EINVAL;
    const int z = p->page_size;
    if (z != 16 && z != 32 && z != 64 && z != 128 && z != 256) return JANO_EUNSUPPORTED;
    const long long most = 1ll << 38;          // a stride in bytes stays below 2^40
    for (const long long st : {p->page_stride, p->token_stride, p->head_stride}) {
        if (st < p->d) return JANO_ESHAPE;
        if (st % 8 || st >= most) return JANO_EUNSUPPORTED;
    }
    if ((long long)s->max_pages * z > INT_MAX) return JANO_EUNSUPPORTED;
    if (!aligned16(p->k) || !aligned16(p->v)) return JANO_EALIGN;
    return JANO_OK;
}

// The queries, keys and values of an append or scatter.
jano_status check_qkv(const RopeCacheCall& r) {
    if (r.n_rows < 0 || r.heads < 1 || r.kv_heads < 1 || r.d < 1) return JANO_EINVAL;
    if (!head_dim_ok(r.d)) return JANO_EUNSUPPORTED;
    const long long q_w = (long long)r.heads * r.d, k_w = (long long)r.kv_heads * r.d;
    if (q_w > INT_MAX || k_w > INT_MAX) return JANO_EUNSUPPORTED;
    if (!r.ids || (r.q != nullptr) != (r.q_out != nullptr)) return JANO_EINVAL;
    jano_status st;
    if (r.q) {
        if ((st = check_rows(r.q, r.q_ld, q_w)) != JANO_OK) return st;
        if ((st = check_rows(r.q_out, r.q_out_ld, q_w)) != JANO_OK) return st;
    }
    if ((st = check_rows(r.k, r.k_ld, k_w)) != JANO_OK) return st;
    return check_rows(r.v, r.v_ld, k_w);
}

int current_sms() {
    int dev = 0, sms = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
                   cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? sms : 0;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
}  // namespace

size_t jano_rope_table_floats(const jano_rope_cfg* c) {
    if (check_rope(c, INT_MAX, true) != JANO_OK) return 0;
    size_t n = 0;
    for (int x = 0; x < 3; ++x) n += (size_t)c->n_pos[x] * c->axes[x];
    return n;
}

jano_status jano_rope_table(const jano_rope_cfg* c, double theta, int shared_freq, float* table, void* stream) {
    const jano_status s = check_rope(c, INT_MAX, true);
    if (s != JANO_OK) return s;
    if (!table || !(theta > 0.0) || !std::isfinite(theta)) return JANO_EINVAL;
    if (!aligned8(table)) return JANO_EALIGN;
    return from_cuda(launch_rope_table(*c, theta, shared_freq, table, static_cast<cudaStream_t>(stream)));
}

jano_status jano_axis_rope(const void* x, long long x_ld, const int32_t* ids, const int32_t* coords, int n_rows,
                           int heads, int d, const jano_rope_cfg* c, const float* table, void* out,
                           long long out_ld, void* stream) {
    if (n_rows < 0 || heads < 1 || d < 1) return JANO_EINVAL;
    const jano_status cs = check_rope(c, d, coords != nullptr);
    if (cs != JANO_OK) return cs;
    if (!head_dim_ok(d) || (long long)heads * d > INT_MAX) return JANO_EUNSUPPORTED;
    if (n_rows == 0) return JANO_OK;
    if (!table) return JANO_EINVAL;
    jano_status s = check_rows(x, x_ld, (long long)heads * d);
    if (s == JANO_OK) s = check_rows(out, out_ld, (long long)heads * d);
    if (s != JANO_OK) return s;
    if (!aligned8(table)) return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_axis_rope(x, x_ld, coords ? nullptr : ids, coords, n_rows, heads, d, *c, table, out,
                                      out_ld, err, static_cast<cudaStream_t>(stream)));
}

jano_status jano_rope_scatter(const void* q, long long q_ld, const void* k, long long k_ld, const void* v,
                              long long v_ld, const int32_t* idx, const int32_t* coords, int n_act, int heads,
                              int kv_heads, int d, const jano_rope_cfg* c, const float* table, void* q_out,
                              long long q_out_ld, void* k_cache, void* v_cache, int n_tokens, void* stream) {
    if (n_act < 0 || n_tokens < 1 || heads < 1 || kv_heads < 1 || d < 1) return JANO_EINVAL;
    const jano_status cs = check_rope(c, d, coords != nullptr);
    if (cs != JANO_OK) return cs;
    if (n_act == 0) return JANO_OK;
    RopeCacheCall r{q, k, v, q_ld, k_ld, v_ld, idx, coords, nullptr, n_act, heads, kv_heads, d, c, table,
                    q_out, q_out_ld, k_cache, v_cache, 0, (long long)kv_heads * d, d, n_tokens, 0, 0, nullptr};
    const jano_status s = check_qkv(r);
    if (s != JANO_OK) return s;
    if (!table || !k_cache || !v_cache) return JANO_EINVAL;
    if (!aligned8(table) || !aligned16(k_cache) || !aligned16(v_cache)) return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_rope_cache(r, err, static_cast<cudaStream_t>(stream)));
}

jano_status jano_paged_append(const jano_page_pool* pool, const jano_page_seqs* seqs, const void* q, long long q_ld,
                              const void* k, long long k_ld, const void* v, long long v_ld, const int32_t* pos,
                              const int32_t* coords, const int32_t* grids, int n_rows, int heads,
                              const jano_rope_cfg* c, const float* table, void* q_out, long long q_out_ld,
                              void* stream) {
    if (n_rows < 0) return JANO_EINVAL;
    if (n_rows == 0) return JANO_OK;
    jano_status s = check_pool(pool, seqs);
    if (s != JANO_OK) return s;
    if ((c != nullptr) != (table != nullptr)) return JANO_EINVAL;
    if (c && (s = check_rope(c, pool->d, coords || grids)) != JANO_OK) return s;
    if (c && !aligned8(table)) return JANO_EALIGN;
    RopeCacheCall r{q, k, v, q_ld, k_ld, v_ld, pos, coords, grids, n_rows, heads, pool->kv_heads, pool->d, c, table,
                    q_out, q_out_ld, pool->k, pool->v, pool->page_stride, pool->token_stride, pool->head_stride, 0,
                    pool->n_pages, pool->page_size, seqs};
    if ((s = check_qkv(r)) != JANO_OK) return s;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    return from_cuda(launch_rope_cache(r, err, static_cast<cudaStream_t>(stream)));
}

jano_status jano_paged_attention(const jano_page_pool* pool, const jano_page_seqs* seqs, const void* q, long long q_ld,
                                 const int32_t* limits, int n_rows, int max_rows, int max_len, int heads,
                                 float scale, int n_split, void* workspace, size_t ws_bytes, void* out,
                                 long long out_ld, void* stream) {
    if (n_rows < 0 || max_rows < 0 || max_len < 0 || heads < 1) return JANO_EINVAL;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return JANO_EINVAL;
    if (n_split < 0 || n_split > 8 || (n_split & (n_split - 1))) return JANO_EINVAL;
    if (n_rows == 0) return JANO_OK;
    jano_status s = check_pool(pool, seqs);
    if (s != JANO_OK) return s;
    if (pool->d != 64 && pool->d != 128) return JANO_EUNSUPPORTED;
    if (heads % pool->kv_heads) return JANO_ESHAPE;
    if (heads / pool->kv_heads > 128 || pool->kv_heads > 65535 || max_len > (1 << 26)) return JANO_EUNSUPPORTED;
    if (q_ld >= (1ll << 38) || (long long)heads * pool->d > INT_MAX) return JANO_EUNSUPPORTED;
    if ((s = check_rows(q, q_ld, (long long)heads * pool->d)) != JANO_OK) return s;
    if ((s = check_rows(out, out_ld, (long long)heads * pool->d)) != JANO_OK) return s;
    if (!aligned16(workspace)) return JANO_EALIGN;
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    const PagedAttentionCall c{pool, seqs, q, q_ld, limits, n_rows, max_rows < 1 ? 1 : max_rows, max_len, heads,
                               scale, n_split, workspace, out, out_ld};
    if (n_split == 0 && workspace) {
        const int sms = current_sms();
        if (sms < 1) return JANO_ECUDA;
        const size_t need = paged_decode_workspace_bytes(c.max_rows, heads, pool->kv_heads, pool->d, sms);
        if (ws_bytes < need) return JANO_EINVAL;
        if (need > 0 && paged_decode_fits(c))
            return from_cuda(launch_paged_decode(c, sms, err, static_cast<cudaStream_t>(stream)));
    }
    return from_cuda(launch_paged_attention(c, err, static_cast<cudaStream_t>(stream)));
}

size_t jano_paged_attention_workspace_bytes(int max_rows, int heads, int kv_heads, int d) {
    if (max_rows < 1 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || (d != 64 && d != 128)) return 0;
    const int sms = current_sms();
    return sms < 1 ? 0 : paged_decode_workspace_bytes(max_rows, heads, kv_heads, d, sms);
}

int jano_paged_attention_splits_on(int n_rows, int max_rows, int max_len, int n_seqs, int heads, int kv_heads,
                                   int sm_count) {
    if (n_rows < 1 || max_rows < 1 || max_len < 1 || n_seqs < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads ||
        heads / kv_heads > 128 || sm_count < 1)
        return 1;
    return paged_split_count(n_rows, max_rows, max_len, n_seqs, heads, kv_heads, sm_count);
}

jano_status jano_get_device_error(void* stream) {
    int* err = device_error_word();
    if (!err) return JANO_ECUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(st) != cudaSuccess) return JANO_ECUDA;
    int v = JANO_OK;
    if (cudaMemcpy(&v, err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return JANO_ECUDA;
    if (v != JANO_OK) {
        const int zero = JANO_OK;
        if (cudaMemcpy(err, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
            return JANO_ECUDA;
    }
    return static_cast<jano_status>(v);
}

const char* jano_status_str(jano_status s) {
    switch (s) {
        case JANO_OK: return "ok";
        case JANO_EINVAL: return "invalid argument";
        case JANO_ESHAPE: return "inconsistent shape";
        case JANO_EALIGN: return "pointer not 16-byte aligned";
        case JANO_EUNSUPPORTED: return "unsupported configuration";
        case JANO_ENONFINITE: return "non-finite score";
        case JANO_EINDEX: return "index or level out of range, or indices not strictly ascending";
        case JANO_ETIMEOUT: return "device wait timed out";
        case JANO_ECUDA: return "CUDA error";
    }
    return "unknown status";
}

int jano_version(void) { return 100; }

}  // extern "C"
