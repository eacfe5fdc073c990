// C ABI of the paged KV cache and of beam search (nanochat_b200.h): argument
// checks, then the launches of paged.cu and beam.cu.
#include "model.h"
#include "paged.h"

#include <initializer_list>

using namespace nc;

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

bool all4(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p || !al4(p)) return false;
    return true;
}

int check_paging(int page_size, int max_blocks, int n_pages) {
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) || max_blocks < 1 || n_pages < 1)
        return NC_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_size > (1ll << 30) || (long long)n_pages * page_size > (1ll << 30))
        return NC_ERR_UNSUPPORTED_SHAPE;
    return NC_OK;
}

int check_requests(int n_req, int rows, int max_blocks) {
    if (n_req < 1 || rows < 1) return NC_ERR_INVALID_ARG;
    if (n_req > kMaxRequests || rows > (1 << 24) || (long long)n_req * max_blocks > 0x7fffffffll)
        return NC_ERR_UNSUPPORTED_SHAPE;
    return NC_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? NC_OK : NC_ERR_CUDA; }

}  // namespace

namespace nc {
int check_paged_step(const nc_model* m, int n_req, int rows, int max_new, int max_blocks, int page_size, int n_pages) {
    if (max_new < 0) return NC_ERR_INVALID_ARG;
    const int r = check_paging(page_size, max_blocks, n_pages);
    if (r != NC_OK) return r;
    // the attention counts 64-key tiles of all requests and K/V heads in 31 bits
    if ((long long)n_req * max_blocks * page_size / 64 > 0x7fffffffll / m->nkv - n_req) return NC_ERR_UNSUPPORTED_SHAPE;
    return check_requests(n_req, rows, max_blocks);
}
}  // namespace nc

extern "C" {

size_t nc_paged_kv_bytes(const nc_model* m, int n_pages, int page_size) {
    if (!m || check_paging(page_size, 1, n_pages) != NC_OK) return 0;
    return (size_t)m->L * 2 * n_pages * page_size * m->nkv * m->hd * dt_size(m->at);
}

int nc_page_plan(nc_model* m, int n_req, int page_size, int max_blocks, int n_pages, int rows,
                 const int32_t* cached_len, const int32_t* new_len, const int32_t* release, int32_t* block_table,
                 int32_t* free_pages, int32_t* free_count, int32_t* cu_rows, int32_t* kv_len, int32_t* positions,
                 int32_t* slots, void* stream) {
    if (!m || !on_model_device(m)) return NC_ERR_INVALID_ARG;
    if (!all4({cached_len, new_len, block_table, free_pages, free_count, cu_rows, kv_len, positions, slots}) ||
        !al4(release))
        return NC_ERR_INVALID_ARG;
    const int r = check_paged_step(m, n_req, rows, 0, max_blocks, page_size, n_pages);
    if (r != NC_OK) return r;
    return done(launch_page_plan(n_req, page_size, max_blocks, n_pages, rows, cached_len, new_len, release,
                                 block_table, free_pages, free_count, cu_rows, kv_len, positions, slots, m->status,
                                 (cudaStream_t)stream));
}

size_t nc_paged_attention_workspace_bytes(const nc_model* m, int n_req, int rows) {
    if (!m || check_requests(n_req, rows, 1) != NC_OK) return 0;
    return paged_attention_workspace(m->at, m->H, m->nkv, m->hd);
}

int nc_paged_attention(nc_model* m, const void* qkv, int rows, int n_req, int max_new, const int32_t* cu_rows,
                       const int32_t* kv_len, const int32_t* slots, const int32_t* block_table, int max_blocks,
                       int page_size, int n_pages, void* k_pages, void* v_pages, void* o, void* workspace,
                       size_t ws_bytes, void* stream) {
    if (!m || !on_model_device(m)) return NC_ERR_INVALID_ARG;
    if (!all4({cu_rows, kv_len, slots, block_table})) return NC_ERR_INVALID_ARG;
    if (!qkv || !k_pages || !v_pages || !o || !workspace || !al16(qkv) || !al16(k_pages) || !al16(v_pages) ||
        !al16(o) || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return NC_ERR_INVALID_ARG;
    const int r = check_paged_step(m, n_req, rows, max_new, max_blocks, page_size, n_pages);
    if (r != NC_OK) return r;
    if (ws_bytes < nc_paged_attention_workspace_bytes(m, n_req, rows)) return NC_ERR_WORKSPACE_TOO_SMALL;
    const PagedKv kv{k_pages, v_pages, block_table, cu_rows, kv_len, n_req, max_blocks, page_size, n_pages};
    return done(paged_attention(m->at, qkv, m->H, m->nkv, m->hd, rows, max_new, slots, kv, o, workspace, m->status,
                                (cudaStream_t)stream));
}

int nc_beam_select(nc_model* m, const void* logits, int batch, int beams, const float* scores,
                   const int32_t* finished, int eos, float* scores_out, int32_t* tokens, int32_t* parents,
                   int32_t* finished_out, void* stream) {
    if (!m || !on_model_device(m) || batch < 1 || beams < 1) return NC_ERR_INVALID_ARG;
    if (!logits || !al16(logits) || !all4({scores, scores_out, tokens, parents})) return NC_ERR_INVALID_ARG;
    if (!finished != !finished_out || !al4(finished) || !al4(finished_out)) return NC_ERR_INVALID_ARG;
    if (finished ? eos < 0 || eos >= m->V : eos != -1) return NC_ERR_INVALID_ARG;
    if (beams > NC_MAX_BEAMS || batch > (1 << 20)) return NC_ERR_UNSUPPORTED_SHAPE;
    return done(launch_beam_select(m->at, logits, batch, beams, m->V, scores, finished, eos, scores_out, tokens,
                                   parents, finished_out, m->status, (cudaStream_t)stream));
}

int nc_beam_reorder(nc_model* m, void* kv_cache, int batch, int beams, int T_max, const int32_t* parents, int start,
                    int end, void* stream) {
    if (!m || !on_model_device(m) || batch < 1 || beams < 1 || T_max < 1) return NC_ERR_INVALID_ARG;
    if (!kv_cache || !al16(kv_cache) || !all4({parents}) || start < 0 || end < start || end > T_max)
        return NC_ERR_INVALID_ARG;
    if (beams > NC_MAX_BEAMS || batch > (1 << 20) || 2ll * m->L * batch > (1 << 30)) return NC_ERR_UNSUPPORTED_SHAPE;
    ReorderArgs a{};
    a.base = (char*)kv_cache;
    a.planes = 2 * m->L; a.batch = batch; a.beams = beams;
    a.width = (int)(m->nkv * m->hd * dt_size(m->at));
    a.plane_stride = (size_t)batch * beams * T_max * a.width;
    a.parents = parents;
    a.t_max = T_max; a.start = start; a.end = end;
    a.status = m->status;
    return done(launch_beam_reorder(a, (cudaStream_t)stream));
}

int nc_beam_reorder_paged(nc_model* m, void* kv_pages, int batch, int beams, int n_pages, int page_size,
                          const int32_t* parents, const int32_t* block_table, int max_blocks, const int32_t* starts,
                          const int32_t* ends, void* stream) {
    if (!m || !on_model_device(m) || batch < 1 || beams < 1) return NC_ERR_INVALID_ARG;
    if (!kv_pages || !al16(kv_pages) || !all4({parents, block_table, starts, ends})) return NC_ERR_INVALID_ARG;
    const int r = check_paging(page_size, max_blocks, n_pages);
    if (r != NC_OK) return r;
    if (beams > NC_MAX_BEAMS || batch > (1 << 20) || 2ll * m->L * batch > (1 << 30)) return NC_ERR_UNSUPPORTED_SHAPE;
    ReorderArgs a{};
    a.base = (char*)kv_pages;
    a.planes = 2 * m->L; a.batch = batch; a.beams = beams;
    a.width = (int)(m->nkv * m->hd * dt_size(m->at));
    a.plane_stride = (size_t)n_pages * page_size * a.width;
    a.parents = parents;
    a.table = block_table; a.starts = starts; a.ends = ends;
    a.max_blocks = max_blocks; a.page = page_size; a.n_pages = n_pages;
    a.status = m->status;
    return done(launch_beam_reorder(a, (cudaStream_t)stream));
}

}  // extern "C"
