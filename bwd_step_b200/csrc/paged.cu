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
#include <climits>

namespace nc {
namespace {

// ---------------------------------------------------------------- plan
// A step with this many packed rows or fewer is planned by one block alone;
// above it a second launch over many blocks writes the rows' positions and
// slots.
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

// Exclusive prefix sums, in place, of three arrays of n <= NT * PER ints in shared
// memory by the block's NT threads; tot[i] gets the sums.
template <int NT, int PER>
__device__ __forceinline__ void plan_scan3(int* a, int* b, int* c, int n, int* tot) {
    __shared__ int ws[3][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int lo = threadIdx.x * PER, used = (n + 32 * PER - 1) / (32 * PER);  // warps with a value
    int va[PER], vb[PER], vc[PER], ia = 0, ib = 0, ic = 0;
    if (w < used) {
        int sa = 0, sb = 0, sc = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool in = lo + i < n;
            va[i] = in ? a[lo + i] : 0; vb[i] = in ? b[lo + i] : 0; vc[i] = in ? c[lo + i] : 0;
            sa += va[i]; sb += vb[i]; sc += vc[i];
        }
        ia = sa; ib = sb; ic = sc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ib, o),
                      z = __shfl_up_sync(0xffffffffu, ic, o);
            if (lane >= o) { ia += x; ib += y; ic += z; }
        }
        if (lane == 31) { ws[0][w] = ia; ws[1][w] = ib; ws[2][w] = ic; }
        ia -= sa; ib -= sb; ic -= sc;
    }
    __syncthreads();
    int ta = 0, tb = 0, tc = 0;
    for (int k = 0; k < used; ++k) {
        const int xa = ws[0][k], xb = ws[1][k], xc = ws[2][k];
        if (k < w) { ia += xa; ib += xb; ic += xc; }
        ta += xa; tb += xb; tc += xc;
    }
    if (w < used) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lo + i < n) {
                a[lo + i] = ia; b[lo + i] = ib; c[lo + i] = ic;
                ia += va[i]; ib += vb[i]; ic += vc[i];
            }
    }
    tot[0] = ta; tot[1] = tb; tot[2] = tc;
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

// (kept: the requests' kept positions, or null: read what the plan wrote)
__device__ __forceinline__ void plan_row(const PlanArgs& p, const int* cu, const int* kept, int shift, int i) {
    int pos = 0, slot = -1;
    if (i < cu[p.n_req]) {
        const int r = row_request(cu, p.n_req, i);
        pos = kept ? kept[r] + (i - cu[r]) : p.kv_len[r] - (cu[r + 1] - i);
        const int page = p.table[(size_t)r * p.max_blocks + (pos >> shift)];
        if ((unsigned)page < (unsigned)p.n_pages) slot = (page << shift) + (pos & (p.page - 1));
        else set_status(p.status, ST_BAD_PAGE);  // the stack of free pages held something else
    }
    p.positions[i] = pos;
    p.slots[i] = slot;
}

// One block.  Per request, the blocks that need a page and the pages that it gives
// back; their prefix sums; then pages go back onto the stack and are taken from its
// top, each at the place that its prefix names, so that the result does not depend on
// timing.  Bound by latency: the chain lengths -> table -> stack -> table -> rows of
// dependent global accesses, and the first run of every stage's code.  So every stage
// has its loads on their way together: a thread's requests with up to kPlanOwn blocks
// each, and for the others (long chunks, released requests) a warp with kPlanWide
// blocks of kPlanKept requests, whose table entries it keeps to the end.  512 requests,
// 48 of them with chunks and 32 released: 16.6 us, 15.7 in a graph (14.3 where the step was
// planned before and few pages move; 34.6 with one window at a time); four decoding
// requests, two of them onto a new page: 3.3 us in a graph, 2.8 where none takes one (3.7
// with 1024 threads).
// The kept entries are what 64 registers a thread hold: three requests a warp of up to 256
// blocks, so 96 chunks and released requests.  Those behind them, and longer rows, are
// read again in each stage: 250 of 512 requests 28 us, 450 of them 41.
constexpr int kPlanWide = 8 * 32, kPlanKept = 3;
constexpr int kPlanSmall = 128;  // requests that a block of as many threads plans

template <int NT, int PER>
__global__ void __launch_bounds__(NT) page_plan_kernel(const PlanArgs p, bool fill_rows) {
    extern __shared__ int sm[];
    __shared__ int s_bad, s_specials;
    __shared__ unsigned long long s_rows;
    int* s_cached = sm;                  // positions kept of every request (0 when released)
    int* s_new = s_cached + p.n_req;     // its new positions
    int* s_need = s_new + p.n_req;       // its blocks without a page, then their prefix
    int* s_back = s_need + p.n_req;      // pages it gives back, then their prefix
    int* s_cu = s_back + p.n_req;        // [n_req + 1]
    int* s_special = s_cu + p.n_req + 1; // requests that a warp looks after, 2 r + (released)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = NT / 32;
    const int shift = 31 - __clz(p.page);
    const long long cap = (long long)p.max_blocks << shift;
    auto held = [&](int e) { return (unsigned)e < (unsigned)p.n_pages; };
    auto row_of = [&](int r) { return p.table + (size_t)r * p.max_blocks; };
    auto first = [&](int r) { return s_cached[r] >> shift; };
    auto end = [&](int r) { return (int)(((long long)s_cached[r] + s_new[r] + p.page - 1) >> shift); };
    struct Entries { int e[kPlanWide / 32]; };
    auto entries = [&](const int32_t* row, int j0, int hi) {
        Entries x;
#pragma unroll
        for (int u = 0; u < kPlanWide / 32; ++u) x.e[u] = j0 + 32 * u + lane < hi ? row[j0 + 32 * u + lane] : -1;
        return x;
    };
    if (tid == 0) { s_bad = 0; s_rows = 0; s_specials = 0; }
    const int count0 = *p.free_count;
    const int count = min(max(count0, 0), p.n_pages);
    int cached[PER], fresh[PER], gone[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = tid + i * NT;
        if (r >= p.n_req) break;
        cached[i] = p.cached[r];
        fresh[i] = p.new_len[r];
        gone[i] = p.release ? p.release[r] : 0;
    }
    __syncthreads();
    unsigned want = 0;  // bit kPlanOwn i + j: block j of the thread's i-th request needs a page
    unsigned long long rows = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = tid + i * NT;
        if (r >= p.n_req) break;
        const bool rel = gone[i] != 0;
        const long long total = (long long)(rel ? 0 : cached[i]) + fresh[i];
        const bool bad = cached[i] < 0 || fresh[i] < 0 || total > cap || fresh[i] > p.rows;
        if (bad) s_bad = ST_BAD_LENGTH;
        const int kept = bad || rel ? 0 : cached[i], n = bad ? 0 : fresh[i];
        s_cached[r] = kept;
        s_new[r] = s_cu[r] = n;
        rows += n;
        const int lo = kept >> shift, hi = bad ? lo : (int)((total + p.page - 1) >> shift);
        s_need[r] = s_back[r] = 0;
        if (!bad && (rel || hi - lo > kPlanOwn)) {
            s_special[atomicAdd(&s_specials, 1)] = 2 * r + rel;
        } else {
            int need = 0;
#pragma unroll
            for (int j = 0; j < kPlanOwn; ++j)
                if (lo + j < hi && !held(row_of(r)[lo + j])) need |= 1 << j;
            want |= (unsigned)need << (kPlanOwn * i);
            s_need[r] = __popc(need);
        }
    }
    for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
    if (lane == 0 && rows) atomicAdd(&s_rows, rows);
    __syncthreads();
    const int specials = s_specials;  // in any order: what comes of them goes by the prefix sums
    // the warp's i-th: request, released or not, and its blocks lo .. hi - 1 that matter
    struct Special { int r, lo, hi; bool rel; };
    auto special = [&](int i) {
        Special s;
        s.r = s_special[i] >> 1;
        s.rel = s_special[i] & 1;
        s.lo = s.rel ? 0 : first(s.r);
        s.hi = s.rel ? p.max_blocks : end(s.r);
        return s;
    };
    Entries kept[kPlanKept];
#pragma unroll
    for (int k = 0; k < kPlanKept; ++k)
        if (warp + k * nwarp < specials) {
            const Special s = special(warp + k * nwarp);
            kept[k] = entries(row_of(s.r), s.lo, s.hi);
        }
    // f(special, entries, first block) over all blocks of the warp's specials, the kept entries first
    auto each = [&](auto begin, auto f, auto done) {
#pragma unroll
        for (int k = 0; k < kPlanKept; ++k)
            if (warp + k * nwarp < specials) {
                const Special s = special(warp + k * nwarp);
                begin(s);
                f(s, kept[k], s.lo);
                for (int j = s.lo + kPlanWide; j < s.hi; j += kPlanWide) f(s, entries(row_of(s.r), j, s.hi), j);
                done(s);
            }
        for (int i = warp + kPlanKept * nwarp; i < specials; i += nwarp) {
            const Special s = special(i);
            begin(s);
            for (int j = s.lo; j < s.hi; j += kPlanWide) f(s, entries(row_of(s.r), j, s.hi), j);
            done(s);
        }
    };
    int n = 0;
    each([&](const Special&) { n = 0; },
         [&](const Special& s, const Entries& x, int j0) {
#pragma unroll
             for (int u = 0; u < kPlanWide / 32; ++u) n += s.rel ? held(x.e[u]) : j0 + 32 * u + lane < s.hi && !held(x.e[u]);
         },
         [&](const Special& s) {
             n = __reduce_add_sync(0xffffffffu, n);
             if (lane == 0) {
                 s_need[s.r] = s.rel ? end(s.r) : n;
                 s_back[s.r] = s.rel ? n : 0;
             }
         });
    __syncthreads();
    int tot[3];
    plan_scan3<NT, PER>(s_need, s_back, s_cu, p.n_req, tot);
    const int need_all = tot[0], back_all = tot[1];
    const int grown = min(count + back_all, p.n_pages);
    int refused = s_bad;
    if (s_rows > (unsigned long long)p.rows) refused |= ST_BAD_LENGTH;
    if (!refused && need_all > grown) refused |= ST_OUT_OF_PAGES;
    if (refused) {  // nothing changes, and the step has no rows
        if (tid == 0) set_status(p.status, refused);
        for (int r = tid; r <= p.n_req; r += NT) {
            p.cu_rows[r] = 0;
            if (r < p.n_req) p.kv_len[r] = p.cached[r];
        }
        if (fill_rows)
            for (int i = tid; i < p.rows; i += NT) { p.positions[i] = 0; p.slots[i] = -1; }
        return;
    }
    if (tid == 0) {
        s_cu[p.n_req] = (int)s_rows;
        *p.free_count = grown - need_all;
        if (count != count0 || count + back_all > p.n_pages) set_status(p.status, ST_BAD_PAGE);
    }
    if (back_all) {
        int at = 0;
        each([&](const Special& s) { at = count + s_back[s.r]; },
             [&](const Special& s, const Entries& x, int j0) {
                 if (!s.rel) return;
#pragma unroll
                 for (int u = 0; u < kPlanWide / 32; ++u) {
                     const unsigned m = __ballot_sync(0xffffffffu, held(x.e[u]));
                     if (held(x.e[u])) {
                         const int to = at + __popc(m & ((1u << lane) - 1));
                         if (to < p.n_pages) p.free_pages[to] = x.e[u];
                         row_of(s.r)[j0 + 32 * u + lane] = -1;
                     }
                     at += __popc(m);
                 }
             },
             [&](const Special&) {});
    }
    __syncthreads();
    if (need_all) {
        int page[PER * kPlanOwn];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = tid + i * NT;
            if (r >= p.n_req) break;
            int from = grown - 1 - s_need[r];
#pragma unroll
            for (int j = 0; j < kPlanOwn; ++j)
                if (want >> (kPlanOwn * i + j) & 1) page[kPlanOwn * i + j] = p.free_pages[from--];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = tid + i * NT;
            if (r >= p.n_req) break;
#pragma unroll
            for (int j = 0; j < kPlanOwn; ++j)
                if (want >> (kPlanOwn * i + j) & 1) row_of(r)[first(r) + j] = page[kPlanOwn * i + j];
        }
        // every page's place first, all of the warp's loads on their way, then the table
        Entries got[kPlanKept];
        int from = 0;
        auto take = [&](const Special& s, const Entries& x, int j0, Entries& y) {
#pragma unroll
            for (int u = 0; u < kPlanWide / 32; ++u) {
                const int j = j0 + 32 * u + lane;
                const bool need = j < end(s.r) && (s.rel || !held(x.e[u]));  // a released row is empty by now
                const unsigned m = __ballot_sync(0xffffffffu, need);
                y.e[u] = need ? p.free_pages[from - __popc(m & ((1u << lane) - 1))] : INT_MIN;
                from -= __popc(m);
            }
        };
        auto put = [&](const Special& s, int j0, const Entries& y) {
#pragma unroll
            for (int u = 0; u < kPlanWide / 32; ++u)
                if (y.e[u] != INT_MIN) row_of(s.r)[j0 + 32 * u + lane] = y.e[u];
        };
        int next[kPlanKept];
#pragma unroll
        for (int k = 0; k < kPlanKept; ++k)
            if (warp + k * nwarp < specials) {
                const Special s = special(warp + k * nwarp);
                from = grown - 1 - s_need[s.r];
                take(s, kept[k], s.lo, got[k]);
                next[k] = from;
            }
#pragma unroll
        for (int k = 0; k < kPlanKept; ++k)
            if (warp + k * nwarp < specials) {
                const Special s = special(warp + k * nwarp);
                put(s, s.lo, got[k]);
                from = next[k];
                for (int j = s.lo + kPlanWide; j < end(s.r); j += kPlanWide) {
                    Entries y;
                    take(s, entries(row_of(s.r), j, s.hi), j, y);
                    put(s, j, y);
                }
            }
        for (int i = warp + kPlanKept * nwarp; i < specials; i += nwarp) {
            const Special s = special(i);
            from = grown - 1 - s_need[s.r];
            for (int j = s.lo; j < end(s.r); j += kPlanWide) {
                Entries y;
                take(s, entries(row_of(s.r), j, s.hi), j, y);
                put(s, j, y);
            }
        }
    }
    for (int r = tid; r <= p.n_req; r += NT) {
        p.cu_rows[r] = s_cu[r];
        if (r < p.n_req) p.kv_len[r] = s_cached[r] + s_new[r];
    }
    __syncthreads();
    if (fill_rows)
        for (int i = tid; i < p.rows; i += NT) plan_row(p, s_cu, s_cached, shift, i);
}

// Positions and slots of the rows, over many blocks.
__global__ void __launch_bounds__(256) page_rows_kernel(const PlanArgs p) {
    extern __shared__ int s_cu[];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is written
    for (int r = threadIdx.x; r <= p.n_req; r += blockDim.x) s_cu[r] = p.cu_rows[r];
    __syncthreads();
    const int shift = 31 - __clz(p.page);
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.rows; i += gridDim.x * blockDim.x)
        plan_row(p, s_cu, nullptr, shift, i);
}

// ---------------------------------------------------------------- cache writes
// (For the tensor-core attention of more than 16 query heads to a K/V head; the other kernels write
// the cache themselves.)
__global__ void __launch_bounds__(256) paged_append_kernel(const bf16* __restrict__ qkv, int H, int nkv, int hd, int rows,
                                                           const int32_t* __restrict__ slots, bf16* __restrict__ kc,
                                                           bf16* __restrict__ vc, int n_slots, int* status) {
    constexpr int VEC = Vec<bf16>::N;
    const int kvn = nkv * hd, per_row = 2 * kvn / VEC;  // vectors of k then v
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)rows * per_row) return;
    const int r = (int)(i / per_row), e = (int)(i % per_row) * VEC;
    const int slot = slots[r];
    if ((unsigned)slot >= (unsigned)n_slots) {
        if (slot >= 0) set_status(status, ST_BAD_PAGE);
        return;
    }
    const bf16* src = qkv + (size_t)r * ((H + 2 * nkv) * hd) + (size_t)H * hd + e;
    bf16* dst = (e < kvn ? kc : vc) + (size_t)slot * kvn + (e < kvn ? e : e - kvn);
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
// Request of packed row i < cu[n_req], by a whole warp, 32 ways at a time.
__device__ __forceinline__ int row_request_warp(const int32_t* __restrict__ cu, int n_req, int i, int lane) {
    int lo = 0, hi = n_req;  // cu[lo] <= i < cu[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && cu[at] <= i);
        const int k = m ? 31 - __clz(m) : 0;
        hi = min(hi, lo + (k + 1) * step);
        lo += k * step;
    }
    return lo;
}

// Heads and types that the tensor-core kernels do not take.  One block per (packed row,
// query head), four warps over the keys, 32 keys of a warp at a time: each lane forms
// one key's whole score, the warp keeps a running maximum and sum, and the lanes then
// own output dims while the 32 weights pass by shuffles.  The four warps are joined at
// the end.  The step's own keys and values are read from its rows, not from the cache,
// so the same launch writes them there.  Bound by latency at the sizes of such models
// (five requests of up to 110 positions, 4 fp32 heads of 16: 7.5 us a call, 5.5 in a graph).
// No key is shared between rows or heads: prompts of 4 x 256 rows on 512 positions take 65 us, with
// 10 heads of 128 1014.
template <typename A, int HD>
__global__ void __launch_bounds__(128) paged_attention_kernel(const A* __restrict__ qkv, int H, int nkv, int rows,
                                                              const int32_t* __restrict__ slots, const PagedKv kv,
                                                              float scale_log2, A* __restrict__ o, int* status) {
    constexpr int VEC = Vec<A>::N;
    constexpr int EPL = HD >= 32 ? HD / 32 : 1;
    constexpr int WAYS = HD >= 32 ? 1 : 32 / HD;  // keys that a warp's lanes take at once in the second product
    __shared__ float sq[HD], sm[4], sl[4], so[4][HD];
    const int row = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (row == rows) {  // the block behind the rows: every request's length and rows, whether it has any or not
        int lo, n, len;
        for (int r = threadIdx.x; h == 0 && r < kv.n_req; r += blockDim.x)
            if (!request(kv, rows, r, lo, n, len)) set_status(status, ST_BAD_LENGTH);
        return;
    }
    const int Nqkv = (H + 2 * nkv) * HD, kvn = nkv * HD;
    A* const kc = reinterpret_cast<A*>(kv.k);
    A* const vc = reinterpret_cast<A*>(kv.v);
    if (h == 0) {
        const int slot = slots[row];
        if ((unsigned)slot < (unsigned)(kv.n_pages * kv.page)) {
            for (int e = threadIdx.x * VEC; e < 2 * kvn; e += 128 * VEC)
                *reinterpret_cast<uint4*>((e < kvn ? kc + e : vc + (e - kvn)) + (size_t)slot * kvn) =
                    *reinterpret_cast<const uint4*>(qkv + (size_t)row * Nqkv + (size_t)H * HD + e);
        } else if (slot >= 0 && threadIdx.x == 0) {
            set_status(status, ST_BAD_PAGE);
        }
    }
    const int32_t* cu = kv.cu_rows;
    for (int c = threadIdx.x; c < HD; c += blockDim.x) sq[c] = tof(qkv[(size_t)row * Nqkv + (size_t)h * HD + c]) * scale_log2;
    if (row < cu[0] || row >= cu[kv.n_req]) return;  // behind the last sequence: stays as it was
    const int r = row_request_warp(cu, kv.n_req, row, lane);
    int lo, fresh, all;
    if (!request(kv, rows, r, lo, fresh, all)) return;
    const int before = all - fresh;  // positions in the cache
    __syncthreads();
    const int len = before + (row - lo) + 1;  // keys that the row sees
    const int32_t* table = kv.table + (size_t)r * kv.max_blocks;
    const int shift = 31 - __clz(kv.page), g = h / (H / nkv);
    float acc[EPL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
    for (int j0 = warp * 32; j0 < len; j0 += 128) {
        const int j = j0 + lane;
        const A *kr = nullptr, *vr = nullptr;  // null: a position without a page, which reads as zeros
        if (j >= before && j < len) {
            kr = qkv + (size_t)(lo + j - before) * Nqkv + (size_t)(H + g) * HD;
            vr = kr + kvn;
        } else if (j < len) {
            const int page = table[j >> shift];
            if ((unsigned)page < (unsigned)kv.n_pages) {
                const size_t at = ((size_t)(page << shift) + (j & (kv.page - 1))) * kvn + (size_t)g * HD;
                kr = kc + at;
                vr = vc + at;
            } else {
                set_status(status, ST_BAD_PAGE);
            }
        }
        float sc = j < len ? 0.f : -INFINITY;
        if (kr) {
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
#pragma unroll 8
        for (int k = 0; k < n; k += WAYS) {
            const int key = k + (WAYS > 1 ? lane / HD : 0);  // below 32; a key behind the last weighs nothing
            const float pk = __shfl_sync(0xffffffffu, pj, key);
            const A* from = reinterpret_cast<const A*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vr), key));
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (from) acc[i] = fmaf(pk, tof(from[WAYS > 1 ? lane % HD : lane + 32 * i]), acc[i]);
        }
    }
#pragma unroll
    for (int x = HD; x < 32; x <<= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], x);
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
    const float inv = 1.f / L;
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
// memory, each changed beam written once: 16 x 4 beams, 20 layers of 250 positions of 128
// (210 MB) take 41 us, 5.1 TB/s.
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

// More beams than a thread holds: 2 or 4 groups of threads share an element's changing
// beams, U each.  They load the parents' vectors, all on their way at once, meet, and
// store them.  Against one thread for up to 32 beams: 5 x 12 beams, 18 layers, 3
// positions of 128 in pages 39 -> 16 us; 10 x 9 beams, 6 layers, up to 118 positions of
// 512 bytes in pages 54 -> 28; 9 x 9 beams, 18 layers of 175 positions of 320, dense
// (472 MB) 121 -> 118.
template <int U, bool PAGED>
__global__ void __launch_bounds__(256) beam_reorder_many_kernel(const ReorderArgs a) {
    __shared__ int s_from[32], s_to[32], s_lo[32], s_hi[32];  // the changing beams: rows, positions
    __shared__ int s_n, s_first, s_last;
    const unsigned vecs = (unsigned)a.width >> 4;
    const int tid = threadIdx.x, shift = PAGED ? 31 - __clz(a.page) : 0;
    const int cap = PAGED ? (int)min((long long)a.max_blocks * a.page, 0x7fffffffll) : a.t_max;
    for (int pb = blockIdx.y; pb < a.planes * a.batch; pb += gridDim.y) {
        const int plane = pb / a.batch, b = pb % a.batch;
        __syncthreads();
        if (tid < 32) {
            const int row = b * a.beams + tid;
            int par = tid, lo = 0, hi = 0;
            if (tid < a.beams) {
                par = a.parents[row];
                lo = PAGED ? max(a.starts[row], 0) : a.start;
                hi = PAGED ? min(a.ends[row], cap) : a.end;
                if ((unsigned)par >= (unsigned)a.beams) {
                    set_status(a.status, ST_BAD_LENGTH);
                    par = tid;
                }
            }
            const bool moves = par != tid && lo < hi;
            const unsigned m = __ballot_sync(0xffffffffu, moves);
            if (moves) {
                const int k = __popc(m & ((1u << tid) - 1));
                s_from[k] = b * a.beams + par;
                s_to[k] = row;
                s_lo[k] = lo;
                s_hi[k] = hi;
            }
            const int first = __reduce_min_sync(0xffffffffu, moves ? lo : 0x7fffffff), last = __reduce_max_sync(0xffffffffu, moves ? hi : 0);
            if (tid == 0) { s_n = __popc(m); s_first = first; s_last = last; }
        }
        __syncthreads();
        const int n = s_n;
        if (n == 0) continue;
        const int lo = s_first, groups = n <= U ? 1 : n <= 2 * U ? 2 : 4, E = 256 / groups;
        const int x = tid & (E - 1), k0 = tid / E * U;  // element of the block's, first of the thread's beams
        const long long total = (long long)(s_last - lo) * vecs;
        char* base = a.base + (size_t)plane * a.plane_stride;
        for (long long at = (long long)blockIdx.x * E; at < total; at += (long long)gridDim.x * E) {
            const long long xx = at + x;
            // (32-bit division where the span allows it)
            const unsigned rel = total <= 0xffffffffll ? (unsigned)xx / vecs : (unsigned)(xx / vecs);
            const int pos = lo + (int)rel;
            const size_t e = (size_t)(xx - (long long)rel * vecs) << 4;
            uint4 v[U];
            char* to[U];
            auto addr = [&](int row) -> char* {  // null: the position has no page
                if (!PAGED) return base + ((size_t)row * a.t_max + pos) * a.width + e;
                const int page = a.table[(size_t)row * a.max_blocks + (pos >> shift)];
                if ((unsigned)page >= (unsigned)a.n_pages) return nullptr;
                return base + (((size_t)page << shift) + (pos & (a.page - 1))) * a.width + e;
            };
            const char* from[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u;
                const bool in = xx < total && k < n && pos >= s_lo[k] && pos < s_hi[k];
                from[u] = to[u] = nullptr;
                if (in) {
                    from[u] = addr(s_from[k]);
                    to[u] = addr(s_to[k]);
                    if (PAGED && (!from[u] || !to[u])) {
                        set_status(a.status, ST_BAD_PAGE);
                        to[u] = nullptr;
                    }
                    if (from[u] == to[u]) to[u] = nullptr;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u]) v[u] = *reinterpret_cast<const uint4*>(from[u]);
            if (groups > 1) __syncthreads();  // else a thread has all of an element's beams
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u]) *reinterpret_cast<uint4*>(to[u]) = v[u];
        }
    }
}

template <bool PAGED>
void reorder_launch(const ReorderArgs& a, dim3 grid, cudaStream_t s) {
    if (a.beams <= 4) beam_reorder_kernel<4, PAGED><<<grid, 256, 0, s>>>(a);
    else if (a.beams <= 8) beam_reorder_kernel<8, PAGED><<<grid, 256, 0, s>>>(a);
    else beam_reorder_many_kernel<8, PAGED><<<grid, 256, 0, s>>>(a);
}

template <typename A>
cudaError_t attention_simt_t(const void* qkv, int H, int nkv, int hd, int rows, const int32_t* slots, const PagedKv& kv,
                             void* o, int* status, cudaStream_t s) {
    const float sl = 1.44269504088896340736f / sqrtf((float)hd);
    const dim3 grid(rows + 1, H);
    const A* q = reinterpret_cast<const A*>(qkv);
    A* out = reinterpret_cast<A*>(o);
    switch (hd) {
        case 16: paged_attention_kernel<A, 16><<<grid, 128, 0, s>>>(q, H, nkv, rows, slots, kv, sl, out, status); break;
        case 32: paged_attention_kernel<A, 32><<<grid, 128, 0, s>>>(q, H, nkv, rows, slots, kv, sl, out, status); break;
        case 64: paged_attention_kernel<A, 64><<<grid, 128, 0, s>>>(q, H, nkv, rows, slots, kv, sl, out, status); break;
        case 128: paged_attention_kernel<A, 128><<<grid, 128, 0, s>>>(q, H, nkv, rows, slots, kv, sl, out, status); break;
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
    constexpr int kLarge = 1024;
    auto large = page_plan_kernel<kLarge, kMaxRequests / kLarge>;
    cudaError_t e = ensure_smem_limit((const void*)large, (6 * kMaxRequests + 1) * 4);
    if (e != cudaSuccess) return e;
    const bool fused = rows <= kPlanFusedRows;
    // few requests and rows: a small block starts and meets sooner
    if (n_req <= kPlanSmall && rows <= 4 * kPlanSmall) page_plan_kernel<kPlanSmall, 1><<<1, kPlanSmall, (6 * n_req + 1) * 4, s>>>(p, fused);
    else large<<<1, kLarge, (6 * n_req + 1) * 4, s>>>(p, fused);
    count_launch();
    if (!fused) {
        const int blocks = std::min((rows + 255) / 256, 4 * device_sm_count());
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(blocks);
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = (n_req + 1) * 4;
        cfg.stream = s;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&cfg, page_rows_kernel, p)) != cudaSuccess) return e;
        count_launch();
    }
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const bf16* qkv, int H, int nkv, int hd, int rows, const int32_t* slots, const PagedKv& kv,
                                int* status, cudaStream_t s) {
    const long long n = (long long)rows * (2ll * nkv * hd / Vec<bf16>::N);
    paged_append_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(qkv, H, nkv, hd, rows, slots, reinterpret_cast<bf16*>(kv.k),
                                                                    reinterpret_cast<bf16*>(kv.v), kv.n_pages * kv.page, status);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_paged_attention_simt(DType at, const void* qkv, int H, int nkv, int hd, int rows, const int32_t* slots,
                                        const PagedKv& kv, void* o, int* status, cudaStream_t s) {
    return at == DT_BF16 ? attention_simt_t<bf16>(qkv, H, nkv, hd, rows, slots, kv, o, status, s)
                         : attention_simt_t<float>(qkv, H, nkv, hd, rows, slots, kv, o, status, s);
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
    const long long want = std::max(1ll, (a.table && a.beams > 8 ? 8ll : 16ll) * device_sm_count() / gy);  // blocks along a span, enough to fill the GPU
    const dim3 grid((unsigned)std::min((n + 255) / 256, want), gy);
    if (a.table) reorder_launch<true>(a, grid, s);
    else reorder_launch<false>(a, grid, s);
    count_launch();
    return cudaGetLastError();
}

}  // namespace nc
