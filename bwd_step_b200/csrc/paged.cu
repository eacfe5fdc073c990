// Paged KV cache: planning of a step from the requests' lengths, writes of new
// K and V to their slots, plain-FMA attention over the pages, and the beams'
// reordering of dense or paged caches.
//
// A page holds `page` consecutive positions of one request (a power of two); a
// request's block table names the page of each of its blocks, so position p
// lives in slot table[p / page] * page + p % page.
#include "paged.h"
#include "common.cuh"

#include <algorithm>

namespace nc {
namespace {

// ---------------------------------------------------------------- plan
// A step with this many packed rows or fewer is planned by one block alone;
// above it a second launch over many blocks writes the rows' positions and
// slots.
constexpr int kPlanThreads = 1024;
constexpr int kPlanFusedRows = 4096;
// Blocks of a request checked by its own thread; longer runs take a warp.
constexpr int kPlanOwn = 4;

struct PlanArgs {
    int n_req, page, max_blocks, n_pages, rows;
    const int32_t* cached;
    const int32_t* new_len;
    const int32_t* release;
    int32_t* table;
    int32_t* free_pages;
    int32_t* free_count;
    int32_t* cu_rows;
    int32_t* kv_len;
    int32_t* positions;
    int32_t* slots;
    int* status;
};

// Exclusive prefix sums, in place, of three arrays of n ints in shared memory
// (n <= kMaxRequests) by kPlanThreads threads; tot[i] gets the sums.
__device__ __forceinline__ void plan_scan3(int* a, int* b, int* c, int n, int* tot) {
    constexpr int PER = kMaxRequests / kPlanThreads;
    __shared__ int ws[3][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int lo = threadIdx.x * PER;
    int va[PER], vb[PER], vc[PER], sa = 0, sb = 0, sc = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = lo + i < n;
        va[i] = in ? a[lo + i] : 0; vb[i] = in ? b[lo + i] : 0; vc[i] = in ? c[lo + i] : 0;
        sa += va[i]; sb += vb[i]; sc += vc[i];
    }
    int ia = sa, ib = sb, ic = sc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ib, o),
                  z = __shfl_up_sync(0xffffffffu, ic, o);
        if (lane >= o) { ia += x; ib += y; ic += z; }
    }
    if (lane == 31) { ws[0][w] = ia; ws[1][w] = ib; ws[2][w] = ic; }
    __syncthreads();
    if (w < 3) {
        int t = ws[w][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += x;
        }
        ws[w][lane] = t;
    }
    __syncthreads();
    ia += (w ? ws[0][w - 1] : 0) - sa; ib += (w ? ws[1][w - 1] : 0) - sb; ic += (w ? ws[2][w - 1] : 0) - sc;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (lo + i < n) {
            a[lo + i] = ia; b[lo + i] = ib; c[lo + i] = ic;
            ia += va[i]; ib += vb[i]; ic += vc[i];
        }
    tot[0] = ws[0][31]; tot[1] = ws[1][31]; tot[2] = ws[2][31];
    __syncthreads();
}

// Request of packed row i: the last r with cu[r] <= i (requests without rows are passed over).
__device__ __forceinline__ int row_request(const int* cu, int n_req, int i) {
    int lo = 0, hi = n_req;  // cu[lo] <= i < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void plan_row(const PlanArgs& p, const int* cu, int shift, int i) {
    int pos = 0, slot = -1;
    if (i < cu[p.n_req]) {
        const int r = row_request(cu, p.n_req, i);
        pos = p.kv_len[r] - (cu[r + 1] - i);
        const int page = p.table[(size_t)r * p.max_blocks + (pos >> shift)];
        if ((unsigned)page < (unsigned)p.n_pages) slot = (page << shift) + (pos & (p.page - 1));
        else set_status(p.status, ST_BAD_PAGE);  // the stack of free pages held something else
    }
    p.positions[i] = pos;
    p.slots[i] = slot;
}

// One block.  Lengths to shared memory; per request the blocks that need a page
// and the pages that it gives back; their prefix sums; then pages go back onto
// the stack and are taken from its top, each at the place that its prefix names,
// so that the result does not depend on timing.  Bound by latency: the chain
// lengths -> table -> stack -> table -> rows of dependent global accesses.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs p, bool fill_rows) {
    extern __shared__ int sm[];
    __shared__ int s_bad;
    __shared__ unsigned long long s_rows;
    int* s_cached = sm;                  // positions kept of every request (0 when released)
    int* s_new = s_cached + p.n_req;     // its new positions
    int* s_need = s_new + p.n_req;       // its blocks without a page, then their prefix
    int* s_back = s_need + p.n_req;      // pages it gives back, then their prefix
    int* s_cu = s_back + p.n_req;        // [n_req + 1]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = kPlanThreads / 32;
    const int shift = 31 - __clz(p.page);
    const long long cap = (long long)p.max_blocks << shift;
    auto held = [&](int e) { return (unsigned)e < (unsigned)p.n_pages; };
    auto released = [&](int r) { return p.release && p.release[r] != 0; };
    if (tid == 0) { s_bad = 0; s_rows = 0; }
    const int count0 = *p.free_count;
    const int count = min(max(count0, 0), p.n_pages);
    __syncthreads();
    for (int r = tid; r < p.n_req; r += kPlanThreads) {
        const int cached = p.cached[r], nw = p.new_len[r];
        const bool rel = released(r);
        const long long total = (long long)(rel ? 0 : cached) + nw;
        const bool bad = cached < 0 || nw < 0 || total > cap || nw > p.rows;
        if (bad) s_bad = ST_BAD_LENGTH;
        s_cached[r] = bad || rel ? 0 : cached;
        s_new[r] = s_cu[r] = bad ? 0 : nw;
        if (!bad && nw) atomicAdd(&s_rows, (unsigned long long)nw);
        // a short run of blocks is checked here, all loads in flight together
        const int lo = s_cached[r] >> shift, hi = bad ? lo : (int)((total + p.page - 1) >> shift);
        int need = 0;
        if (rel || hi - lo > kPlanOwn) need = -1;
        else
#pragma unroll
            for (int j = 0; j < kPlanOwn; ++j)
                need += lo + j < hi && !held(p.table[(size_t)r * p.max_blocks + lo + j]);
        s_need[r] = need;
        s_back[r] = 0;
    }
    __syncthreads();
    for (int r = warp; r < p.n_req; r += nwarp) {
        if (s_need[r] >= 0) continue;
        const int32_t* row = p.table + (size_t)r * p.max_blocks;
        const int lo = s_cached[r] >> shift, hi = (int)(((long long)s_cached[r] + s_new[r] + p.page - 1) >> shift);
        int n = 0;
        if (released(r)) {
            for (int j = lane; j < p.max_blocks; j += 32) n += held(row[j]);
        } else {
            for (int j = lo + lane; j < hi; j += 32) n += !held(row[j]);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) {
            if (released(r)) { s_back[r] = n; s_need[r] = hi; }
            else s_need[r] = n;
        }
    }
    __syncthreads();
    int tot[3];
    plan_scan3(s_need, s_back, s_cu, p.n_req, tot);
    const int need_all = tot[0], back_all = tot[1];
    const int grown = min(count + back_all, p.n_pages);
    int refused = s_bad;
    if (s_rows > (unsigned long long)p.rows) refused |= ST_BAD_LENGTH;
    if (!refused && need_all > grown) refused |= ST_OUT_OF_PAGES;
    if (refused) {  // nothing changes, and the step has no rows
        if (tid == 0) set_status(p.status, refused);
        for (int r = tid; r <= p.n_req; r += kPlanThreads) {
            p.cu_rows[r] = 0;
            if (r < p.n_req) p.kv_len[r] = p.cached[r];
        }
        if (fill_rows)
            for (int i = tid; i < p.rows; i += kPlanThreads) { p.positions[i] = 0; p.slots[i] = -1; }
        return;
    }
    if (tid == 0) {
        s_cu[p.n_req] = (int)s_rows;
        if (count != count0 || count + back_all > p.n_pages) set_status(p.status, ST_BAD_PAGE);
    }
    if (back_all) {
        for (int r = warp; r < p.n_req; r += nwarp) {
            if (!released(r)) continue;
            int32_t* row = p.table + (size_t)r * p.max_blocks;
            int at = count + s_back[r];
            for (int j0 = 0; j0 < p.max_blocks; j0 += 32) {
                const int e = j0 + lane < p.max_blocks ? row[j0 + lane] : -1;
                const unsigned m = __ballot_sync(0xffffffffu, held(e));
                if (held(e)) {
                    const int to = at + __popc(m & ((1u << lane) - 1));
                    if (to < p.n_pages) p.free_pages[to] = e;
                    row[j0 + lane] = -1;
                }
                at += __popc(m);
            }
        }
    }
    __syncthreads();
    if (need_all) {
        for (int r = tid; r < p.n_req; r += kPlanThreads) {
            const int lo = s_cached[r] >> shift, hi = (s_cached[r] + s_new[r] + p.page - 1) >> shift;
            if (hi - lo > kPlanOwn) continue;
            int32_t* row = p.table + (size_t)r * p.max_blocks;
            int from = grown - 1 - s_need[r];
#pragma unroll
            for (int j = 0; j < kPlanOwn; ++j)
                if (lo + j < hi && !held(row[lo + j])) row[lo + j] = p.free_pages[from--];
        }
        for (int r = warp; r < p.n_req; r += nwarp) {
            const int lo = s_cached[r] >> shift, hi = (s_cached[r] + s_new[r] + p.page - 1) >> shift;
            if (hi - lo <= kPlanOwn) continue;
            int32_t* row = p.table + (size_t)r * p.max_blocks;
            int from = grown - 1 - s_need[r];
            for (int j0 = lo; j0 < hi; j0 += 32) {
                const bool want = j0 + lane < hi && !held(row[j0 + lane]);
                const unsigned m = __ballot_sync(0xffffffffu, want);
                if (want) row[j0 + lane] = p.free_pages[from - __popc(m & ((1u << lane) - 1))];
                from -= __popc(m);
            }
        }
    }
    for (int r = tid; r <= p.n_req; r += kPlanThreads) {
        p.cu_rows[r] = s_cu[r];
        if (r < p.n_req) p.kv_len[r] = s_cached[r] + s_new[r];
    }
    __syncthreads();
    if (tid == 0) *p.free_count = grown - need_all;
    if (fill_rows)
        for (int i = tid; i < p.rows; i += kPlanThreads) plan_row(p, s_cu, shift, i);
}

// Positions and slots of the rows, over many blocks.
__global__ void __launch_bounds__(256) page_rows_kernel(const PlanArgs p) {
    extern __shared__ int s_cu[];
    for (int r = threadIdx.x; r <= p.n_req; r += blockDim.x) s_cu[r] = p.cu_rows[r];
    __syncthreads();
    const int shift = 31 - __clz(p.page);
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.rows; i += gridDim.x * blockDim.x)
        plan_row(p, s_cu, shift, i);
}

// ---------------------------------------------------------------- cache writes
template <typename A>
__global__ void __launch_bounds__(256) paged_append_kernel(const A* __restrict__ qkv, int H, int nkv, int hd, int rows,
                                                           const int32_t* __restrict__ slots, A* __restrict__ kc,
                                                           A* __restrict__ vc, int n_slots, int* status) {
    constexpr int VEC = Vec<A>::N;
    const int kvn = nkv * hd, per_row = 2 * kvn / VEC;  // vectors of k then v
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)rows * per_row) return;
    const int r = (int)(i / per_row), e = (int)(i % per_row) * VEC;
    const int slot = slots[r];
    if ((unsigned)slot >= (unsigned)n_slots) {
        if (slot >= 0) set_status(status, ST_BAD_PAGE);
        return;
    }
    const A* src = qkv + (size_t)r * ((H + 2 * nkv) * hd) + (size_t)H * hd + e;
    A* dst = (e < kvn ? kc : vc) + (size_t)slot * kvn + (e < kvn ? e : e - kvn);
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
}

template <typename A>
__global__ void __launch_bounds__(128) last_rows_kernel(const A* __restrict__ x, int d, int rows,
                                                        const int32_t* __restrict__ cu, A* __restrict__ out) {
    constexpr int VEC = Vec<A>::N;
    const int r = blockIdx.x, row = cu[r + 1] - 1;
    const bool live = row >= cu[r] && row < rows;
    for (int c = threadIdx.x * VEC; c < d; c += blockDim.x * VEC)
        *reinterpret_cast<uint4*>(out + (size_t)r * d + c) =
            live ? *reinterpret_cast<const uint4*>(x + (size_t)row * d + c) : make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- plain attention
// One block per (packed row, query head), four warps over the keys, 32 keys of a
// warp at a time: each lane forms one key's whole score, the warp keeps a running
// maximum and sum, and the lanes then own HD/32 output dims each while the 32
// weights and slots pass by shuffles.  The four warps are joined at the end.
template <typename A, int HD>
__global__ void __launch_bounds__(128) paged_attention_kernel(const A* __restrict__ qkv, int H, int nkv,
                                                              const A* __restrict__ kc, const A* __restrict__ vc,
                                                              const PagedKv kv, float scale_log2, A* __restrict__ o,
                                                              int* status) {
    constexpr int VEC = Vec<A>::N;
    constexpr int EPL = HD >= 32 ? HD / 32 : 1;
    __shared__ float sq[HD], sm[4], sl[4], so[4][HD];
    __shared__ int s_r;
    const int row = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) s_r = row < kv.cu_rows[kv.n_req] && row >= kv.cu_rows[0] ? row_request(kv.cu_rows, kv.n_req, row) : -1;
    const int Nqkv = (H + 2 * nkv) * HD;
    for (int c = threadIdx.x; c < HD; c += blockDim.x) sq[c] = tof(qkv[(size_t)row * Nqkv + (size_t)h * HD + c]) * scale_log2;
    __syncthreads();
    const int r = s_r;
    if (r < 0) return;  // a row behind the last sequence stays as it was
    const int len = kv.kv_len[r] - (kv.cu_rows[r + 1] - row) + 1;  // keys that the row sees
    if (kv.kv_len[r] > (long long)kv.max_blocks * kv.page || len <= 0) {
        if (threadIdx.x == 0 && h == 0) set_status(status, ST_BAD_LENGTH);
        return;
    }
    const int32_t* table = kv.table + (size_t)r * kv.max_blocks;
    const int shift = 31 - __clz(kv.page);
    const int g = h / (H / nkv);
    const size_t ld = (size_t)nkv * HD;
    float acc[EPL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
    for (int j0 = warp * 32; j0 < len; j0 += 128) {
        const int j = j0 + lane;
        int slot = -1;
        if (j < len) {
            const int page = table[j >> shift];
            if ((unsigned)page < (unsigned)kv.n_pages) slot = (page << shift) + (j & (kv.page - 1));
            else set_status(status, ST_BAD_PAGE);
        }
        float sc = j < len ? 0.f : -INFINITY;  // a position without a page reads as zeros
        if (slot >= 0) {
            const A* kr = kc + (size_t)slot * ld + (size_t)g * HD;
#pragma unroll
            for (int c = 0; c < HD; c += VEC) {
                float x[VEC];
                load_vec(kr + c, x);
#pragma unroll
                for (int e = 0; e < VEC; ++e) sc = fmaf(sq[c + e], x[e], sc);
            }
        }
        const float mn = fmaxf(m, warp_max(sc));
        if (mn == -INFINITY) continue;  // the warp has seen no key yet
        const float alpha = exp2f(m - mn), pj = exp2f(sc - mn);
        l = l * alpha + pj;
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] *= alpha;
        m = mn;
        const int n = min(32, len - j0);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float pk = __shfl_sync(0xffffffffu, pj, k);
            const int sk = __shfl_sync(0xffffffffu, slot, k);
            if (sk < 0) continue;
            const A* vr = vc + (size_t)sk * ld + (size_t)g * HD;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (lane + 32 * i < HD) acc[i] = fmaf(pk, tof(vr[lane + 32 * i]), acc[i]);
        }
    }
    l = warp_sum(l);
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < HD) so[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float w4[4], L = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        w4[w] = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M);
        L += sl[w] * w4[w];
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;  // a row without a key gives zeros
    for (int c = threadIdx.x; c < HD; c += blockDim.x) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) x += so[w][c] * w4[w];
        o[(size_t)row * H * HD + (size_t)h * HD + c] = fromf<A>(x * inv);
    }
}

// ---------------------------------------------------------------- beams' reordering
// One thread owns 16 bytes of one position in every beam of a batch row: it
// loads the parents' vectors of all beams that change, then stores them, so the
// exchange is in place without a buffer or a barrier (a parent wanted twice is
// read again from L1).  Bound by HBM: each wanted parent is read once from
// memory, each changed beam written once.
template <int NB, bool PAGED>
__global__ void __launch_bounds__(256) beam_reorder_kernel(const ReorderArgs a) {
    __shared__ int s_par[NB];
    const int vecs = a.width >> 4;
    for (int pb = blockIdx.y; pb < a.planes * a.batch; pb += gridDim.y) {
        const int plane = pb / a.batch, b = pb % a.batch;
        __syncthreads();
        if (threadIdx.x < NB) {
            const int i = threadIdx.x;
            int par = i < a.beams ? a.parents[b * a.beams + i] : i;
            if ((unsigned)par >= (unsigned)a.beams && i < a.beams) {
                set_status(a.status, ST_BAD_LENGTH);
                par = i;
            }
            s_par[i] = par;
        }
        __syncthreads();
        int lo = a.start, hi = a.end;
        if (PAGED) {
            lo = 0x7fffffff; hi = 0;
            const int cap = (int)min((long long)a.max_blocks * a.page, 0x7fffffffll);
            for (int i = 0; i < a.beams; ++i) {
                if (s_par[i] == i) continue;
                lo = min(lo, max(a.starts[b * a.beams + i], 0));
                hi = max(hi, min(a.ends[b * a.beams + i], cap));
            }
        }
        char* base = a.base + (size_t)plane * a.plane_stride;
        const int shift = PAGED ? 31 - __clz(a.page) : 0;
        const long long n = hi > lo ? (long long)(hi - lo) * vecs : 0;
        for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (long long)gridDim.x * blockDim.x) {
            const int pos = lo + (int)(x / vecs);
            const size_t e = (size_t)(x % vecs) << 4;
            auto addr = [&](int i) -> char* {  // null: the position has no page
                const int row = b * a.beams + i;
                if (!PAGED) return base + ((size_t)row * a.t_max + pos) * a.width + e;
                const int page = a.table[(size_t)row * a.max_blocks + (pos >> shift)];
                if ((unsigned)page >= (unsigned)a.n_pages) {
                    set_status(a.status, ST_BAD_PAGE);
                    return nullptr;
                }
                return base + (((size_t)page << shift) + (pos & (a.page - 1))) * a.width + e;
            };
            uint4 v[NB];
            char* to[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                to[i] = nullptr;
                const int par = s_par[i];
                if (par == i) continue;
                if (PAGED && (pos < a.starts[b * a.beams + i] || pos >= a.ends[b * a.beams + i])) continue;
                const char* from = addr(par);
                char* t = addr(i);
                if (!from || !t || from == t) continue;
                v[i] = *reinterpret_cast<const uint4*>(from);
                to[i] = t;
            }
#pragma unroll
            for (int i = 0; i < NB; ++i)
                if (to[i]) *reinterpret_cast<uint4*>(to[i]) = v[i];
        }
    }
}

template <bool PAGED>
void reorder_launch(const ReorderArgs& a, dim3 grid, cudaStream_t s) {
    if (a.beams <= 4) beam_reorder_kernel<4, PAGED><<<grid, 256, 0, s>>>(a);
    else if (a.beams <= 8) beam_reorder_kernel<8, PAGED><<<grid, 256, 0, s>>>(a);
    else if (a.beams <= 16) beam_reorder_kernel<16, PAGED><<<grid, 256, 0, s>>>(a);
    else beam_reorder_kernel<32, PAGED><<<grid, 256, 0, s>>>(a);
}

template <typename A>
cudaError_t attention_simt_t(const void* qkv, int H, int nkv, int hd, int rows, const PagedKv& kv, void* o,
                             int* status, cudaStream_t s) {
    const float sl = 1.44269504088896340736f / sqrtf((float)hd);
    const dim3 grid(rows, H);
    const A* q = reinterpret_cast<const A*>(qkv);
    const A* k = reinterpret_cast<const A*>(kv.k);
    const A* v = reinterpret_cast<const A*>(kv.v);
    A* out = reinterpret_cast<A*>(o);
    switch (hd) {
        case 16: paged_attention_kernel<A, 16><<<grid, 128, 0, s>>>(q, H, nkv, k, v, kv, sl, out, status); break;
        case 32: paged_attention_kernel<A, 32><<<grid, 128, 0, s>>>(q, H, nkv, k, v, kv, sl, out, status); break;
        case 64: paged_attention_kernel<A, 64><<<grid, 128, 0, s>>>(q, H, nkv, k, v, kv, sl, out, status); break;
        case 128: paged_attention_kernel<A, 128><<<grid, 128, 0, s>>>(q, H, nkv, k, v, kv, sl, out, status); break;
        default: return cudaErrorInvalidValue;
    }
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_plan(int n_req, int page, int max_blocks, int n_pages, int rows, const int32_t* cached,
                             const int32_t* new_len, const int32_t* release, int32_t* table, int32_t* free_pages,
                             int32_t* free_count, int32_t* cu_rows, int32_t* kv_len, int32_t* positions,
                             int32_t* slots, int* status, cudaStream_t s) {
    const PlanArgs p{n_req, page, max_blocks, n_pages, rows, cached, new_len, release, table, free_pages, free_count,
                     cu_rows, kv_len, positions, slots, status};
    cudaError_t e = ensure_smem_limit((const void*)page_plan_kernel, (5 * kMaxRequests + 1) * 4);
    if (e != cudaSuccess) return e;
    const bool fused = rows <= kPlanFusedRows;
    page_plan_kernel<<<1, kPlanThreads, (5 * n_req + 1) * 4, s>>>(p, fused);
    count_launch();
    if (!fused) {
        const int blocks = std::min((rows + 255) / 256, 4 * device_sm_count());
        page_rows_kernel<<<blocks, 256, (n_req + 1) * 4, s>>>(p);
        count_launch();
    }
    return cudaGetLastError();
}

cudaError_t launch_paged_append(DType at, const void* qkv, int H, int nkv, int hd, int rows, const int32_t* slots,
                                const PagedKv& kv, int* status, cudaStream_t s) {
    const long long n = (long long)rows * (2ll * nkv * hd * (long long)dt_size(at) / 16);
    const unsigned blocks = (unsigned)((n + 255) / 256);
    const int n_slots = kv.n_pages * kv.page;
    if (at == DT_BF16)
        paged_append_kernel<bf16><<<blocks, 256, 0, s>>>(reinterpret_cast<const bf16*>(qkv), H, nkv, hd, rows, slots,
                                                         reinterpret_cast<bf16*>(kv.k), reinterpret_cast<bf16*>(kv.v),
                                                         n_slots, status);
    else
        paged_append_kernel<float><<<blocks, 256, 0, s>>>(reinterpret_cast<const float*>(qkv), H, nkv, hd, rows, slots,
                                                          reinterpret_cast<float*>(kv.k),
                                                          reinterpret_cast<float*>(kv.v), n_slots, status);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_paged_attention_simt(DType at, const void* qkv, int H, int nkv, int hd, int rows, const PagedKv& kv,
                                        void* o, int* status, cudaStream_t s) {
    return at == DT_BF16 ? attention_simt_t<bf16>(qkv, H, nkv, hd, rows, kv, o, status, s)
                         : attention_simt_t<float>(qkv, H, nkv, hd, rows, kv, o, status, s);
}

cudaError_t launch_last_rows(DType at, const void* x, int d, int rows, const int32_t* cu_rows, int n_req, void* out,
                             cudaStream_t s) {
    if (at == DT_BF16)
        last_rows_kernel<bf16><<<n_req, 128, 0, s>>>(reinterpret_cast<const bf16*>(x), d, rows, cu_rows,
                                                     reinterpret_cast<bf16*>(out));
    else
        last_rows_kernel<float><<<n_req, 128, 0, s>>>(reinterpret_cast<const float*>(x), d, rows, cu_rows,
                                                      reinterpret_cast<float*>(out));
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const ReorderArgs& a, cudaStream_t s) {
    const long long span = a.table ? (long long)a.max_blocks * a.page : a.end - a.start;
    const long long n = span * (a.width / 16);
    if (n <= 0) return cudaSuccess;
    const unsigned gy = (unsigned)std::min(65535ll, (long long)a.planes * a.batch);
    const long long want = std::max(1ll, 16ll * device_sm_count() / gy);  // blocks along a span, enough to fill the GPU
    const dim3 grid((unsigned)std::min((n + 255) / 256, want), gy);
    if (a.table) reorder_launch<true>(a, grid, s);
    else reorder_launch<false>(a, grid, s);
    count_launch();
    return cudaGetLastError();
}

}  // namespace nc
