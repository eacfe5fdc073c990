// Paged KV cache: step planning, cache writes, attention and reordering
// (internal to the library).
#pragma once
#include "kernels.h"

#include <cuda_bf16.h>

struct nc_model;

namespace nc {

// Requests that one plan or attention call takes: their prefix sums live in
// one block's shared memory.
constexpr int kMaxRequests = 4096;

// A paged cache of one layer and the requests' tables over it.
//   k, v: [n_pages, page, nkv, hd] in the activation type; page is a power of two
//   table: [n_req, max_blocks] page of every block of a request, -1 where none
//   cu_rows: [n_req + 1] first packed row of every request's new tokens
//   kv_len: [n_req] positions of every request, the new ones among them
struct PagedKv {
    void* k;
    void* v;
    const int32_t* table;
    const int32_t* cu_rows;
    const int32_t* kv_len;
    int n_req, max_blocks, page, n_pages;
};

// New rows and length of request r; false (nothing to do, or reported) where the
// step's arrays do not fit each other.
__device__ __forceinline__ bool request(const PagedKv& kv, int rows, int r, int& lo, int& n, int& len) {
    lo = kv.cu_rows[r];
    const int hi = kv.cu_rows[r + 1];
    len = kv.kv_len[r];
    n = hi - lo;
    const long long cap = (long long)kv.max_blocks * kv.page;
    return lo >= 0 && hi <= rows && n >= 0 && len >= n && len <= cap;
}

// Block tables, row offsets, positions and slots of a step (see nc_page_plan).
cudaError_t launch_page_plan(int n_req, int page, int max_blocks, int n_pages, int rows, const int32_t* cached,
                             const int32_t* new_len, const int32_t* release, int32_t* table, int32_t* free_pages,
                             int32_t* free_count, int32_t* cu_rows, int32_t* kv_len, int32_t* positions,
                             int32_t* slots, int* status, cudaStream_t s);

// The k, v heads of the packed qkv rows to their cache slots (slot < 0: the row has none).
cudaError_t launch_paged_append(const __nv_bfloat16* qkv, int H, int nkv, int hd, int rows, const int32_t* slots,
                                const PagedKv& kv, int* status, cudaStream_t s);

// The rows' k, v to their slots and o[row, h] = softmax over the keys at positions 0..pos(row) of the
// row's request, plain FMA kernel.
cudaError_t launch_paged_attention_simt(DType at, const void* qkv, int H, int nkv, int hd, int rows, const int32_t* slots,
                                        const PagedKv& kv, void* o, int* status, cudaStream_t s);

// The last new row of every request: out[r] = x[cu_rows[r + 1] - 1] (rows of d elements), zeros for a
// request without new rows.
cudaError_t launch_last_rows(DType at, const void* x, int d, int rows, const int32_t* cu_rows, int n_req, void* out,
                             cudaStream_t s);

// One layer's step: the rows' k, v to their slots, then their attention (see nc_paged_attention).
cudaError_t paged_attention(DType at, const void* qkv, int H, int nkv, int hd, int rows, int max_new,
                            const int32_t* slots, const PagedKv& kv, void* o, void* workspace, int* status,
                            cudaStream_t s);
// Sizes of a paged step that the kernels take (NC_OK or the error code).
int check_paged_step(const nc_model* m, int n_req, int rows, int max_new, int max_blocks, int page_size, int n_pages);
size_t paged_attention_workspace(DType at, int H, int nkv, int hd);

// Rows (b, i) of a cache, i < beams, take the entries of row (b, parents[b, i]) at positions start..end-1, in place.
// planes: K and V of every layer, plane_stride bytes apart; width: bytes of one position in a plane.
struct ReorderArgs {
    char* base;
    size_t plane_stride;
    int planes, batch, beams, width;
    const int32_t* parents;
    // dense: [batch * beams, t_max] positions per plane, one span for all rows
    int t_max, start, end;
    // paged (table != null): spans per row, positions through the block table
    const int32_t* table;
    const int32_t* starts;
    const int32_t* ends;
    int max_blocks, page, n_pages;
    int* status;
};
cudaError_t launch_beam_reorder(const ReorderArgs& a, cudaStream_t s);

// Beam search's selection (see nc_beam_select).
constexpr int kMaxBeams = 32;
cudaError_t launch_beam_select(DType at, const void* logits, int batch, int beams, int V, const float* scores,
                               const int32_t* finished, int eos, float* scores_out, int32_t* tokens, int32_t* parents,
                               int32_t* finished_out, int* status, cudaStream_t s);

}  // namespace nc
