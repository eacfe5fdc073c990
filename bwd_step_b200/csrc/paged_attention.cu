// Attention of a step's new tokens over the paged cache, bf16.
//
// Decoding requests (one new token): per K/V head the group's query heads, 16 at
// most, are the rows of one small matrix product against every cached key, so
// each key and value is read once for all of them.  Bound by HBM.
//
// Work is cut evenly over the SMs: the requests' key tiles of all K/V heads form
// one line, and block c of G takes the tiles [c W / G, (c + 1) W / G) of its W.
// A (request, K/V head) that lies in one block is finished there; one that is cut
// leaves a partial output, row maximum and sum in each of its blocks, and a second
// kernel joins them in the blocks' order, so the result does not depend on timing.
// A block has at most two partial results: its first and its last piece.
#include "paged.h"
#include "tc_common.cuh"
#include <cudaTypedefs.h>
#include <algorithm>

namespace nc {
namespace {
using namespace tc;

constexpr int kTile = 64;        // keys of a decode tile
constexpr int kDecRows = 16;     // query heads of a K/V head that the decode kernel takes
constexpr int kDecThreads = 288; // 8 consumer warps, then the producer
constexpr float kLog2eF = 1.44269504088896340736f;

// Rows of a partial result: halves of `half` rows, row i of a half is token i / Hg of
// it and head i % Hg; `tokens` per half.  One int4 per block in `desc`, for the piece
// that begins in this block and goes on in the next ones: first packed row, K/V head,
// 2 * (number of blocks it lies in) + (its slot here), its tokens; z = 0: none.
struct Partials {
    float* o;      // [2 G, rows, HD] unnormalised
    float2* ml;    // [2 G, rows] maximum (log2 domain), sum
    int4* desc;    // [G]
};

struct DecodeArgs {
    const bf16* qkv;
    const int32_t* slots;
    PagedKv kv;
    bf16* o;
    Partials part;
    int H, nkv, Hg, rows, piece, max_new;  // piece: rows of one copy, min(page, kTile)
    float scale_log2;
    int* status;
};

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// d[16x8] += a[16x16] b[16x8]
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

// ---------------------------------------------------------------- requests
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

// Exclusive prefix sums of v(r), r < n, into pre[0..n] by all NT threads of the block.
template <int NT, typename T, typename F>
__device__ __forceinline__ void block_prefix(T* pre, int n, F v) {
    __shared__ T ws[NT / 32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    T run = 0;
    for (int base = 0; base < n; base += NT) {
        const int r = base + (int)threadIdx.x;
        const T x = r < n ? v(r) : T(0);
        T s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane == 31) ws[w] = s;
        __syncthreads();
        T before = 0, all = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            if (i < w) before += ws[i];
            all += ws[i];
        }
        if (r < n) pre[r] = run + before + s - x;
        run += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[n] = run;
    __syncthreads();
}

// The last r with pre[r] <= x < pre[r + 1].
template <typename T>
__device__ __forceinline__ int find_request(const T* pre, int n, T x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ long long cut(long long W, int G, int c) { return W * c / G; }  // first tile of block c
__device__ __forceinline__ int block_of(long long W, int G, long long x) { return (int)(((x + 1) * G - 1) / W); }

// ---------------------------------------------------------------- decode
template <int HD>
struct DecLayout {
    static constexpr int KV = kTile * HD * 2;               // one tile of K or V
    static constexpr int STAGE = 2 * KV;
    // Even: the two groups of consumers take the tiles in turn, so a stage is always the
    // same group's.  With an odd number one group could test a stage's barrier two phases
    // ahead, while the other's tile is still on its way, and see the phase before as its own.
    static constexpr int STAGES = HD == 128 ? 4 : 8;
    static_assert(STAGES % 2 == 0, "a stage belongs to one group of consumers");
    static constexpr int RED = STAGES * STAGE;              // 4 warps' accumulators and statistics
    static constexpr int RED_W = (HD / 2 + 4) * 32 * 4;
    static constexpr int BAR = RED + 4 * RED_W;
    static constexpr int PRE = BAR + 256;
    static constexpr int bytes(int n_req) { return PRE + (n_req + 1) * 4; }
};
static_assert(DecLayout<128>::bytes(kMaxRequests) <= 232448 && DecLayout<64>::bytes(kMaxRequests) <= 232448,
              "decode shared memory exceeds the per-block limit");

// One piece of a block's tiles: part of one (request, K/V head).
struct DecSeg {
    int r, g, row, len, tiles, k0, k1;
    long long unit;  // its (request, K/V head)'s first tile in the line
};
__device__ __forceinline__ DecSeg dec_seg(const DecodeArgs& a, const int* pre, int x, int x1) {
    DecSeg s;
    int n;
    s.r = find_request(pre, a.kv.n_req, x);
    request(a.kv, a.rows, s.r, s.row, n, s.len);
    s.tiles = (s.len + kTile - 1) / kTile;
    const int rem = x - pre[s.r];
    s.g = rem / s.tiles;
    s.k0 = rem % s.tiles;
    s.k1 = min(s.tiles, s.k0 + (x1 - x));
    s.unit = pre[s.r] + (long long)s.g * s.tiles;
    return s;
}

// Byte of 16-byte vector j of key `key` in a tile: pieces of `piece` rows, each
// [HD / 64][piece][128 bytes] with the 128-byte swizzle of the copies.
template <int HD>
__device__ __forceinline__ uint32_t dec_at(int key, int j, int pshift) {
    const int p = key >> pshift, rr = key & ((1 << pshift) - 1);
    return (uint32_t)(((p << pshift) * HD * 2) + ((j >> 3) << (pshift + 7)) + rr * 128 + (((j & 7) ^ (rr & 7)) << 4));
}

// Eight consumer warps in two groups that take the tiles in turn; a warp has 16 of
// its tile's 64 keys, a running maximum and sum, and a whole output, and the eight are
// joined at the end of a piece.  S = Q K^T and O += P V are mma.sync products of
// 16 rows: at 16 rows a tile's 64 KB of operands take 1400 cycles to arrive and
// some 300 to multiply, and tcgen05's 128 rows would be an eighth full.
template <int HD>
__global__ void __launch_bounds__(kDecThreads, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a) {
    using Lay = DecLayout<HD>;
    constexpr int ST = Lay::STAGES, NB = HD / 8;
    extern __shared__ __align__(1024) uint8_t smem_dyn[];
    if ((smem_u32(smem_dyn) & 1023u) != 0) {
        if (threadIdx.x == 0) set_status(a.status, ST_BAD_LAYOUT);
        return;
    }
    pdl_trigger();
    const uint32_t base = smem_u32(smem_dyn);
    float* red = reinterpret_cast<float*>(smem_dyn + Lay::RED);
    const uint32_t full = base + Lay::BAR, empty = full + 8 * ST;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_dyn + Lay::BAR + 16 * ST);
    int* pre = reinterpret_cast<int*>(smem_dyn + Lay::PRE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int st = 0; st < ST; ++st) {
            mbar_init(full + 8 * st, 1);
            mbar_init(empty + 8 * st, 4);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch(&tm_k);
        tma_prefetch(&tm_v);
    }
    block_prefix<kDecThreads>(pre, a.kv.n_req, [&](int r) {
        int lo, n, len;
        const bool ok = request(a.kv, a.rows, r, lo, n, len);
        if (blockIdx.x == 0 && (!ok || (a.max_new > 0 && n > a.max_new))) set_status(a.status, ST_BAD_LENGTH);
        return ok && n == 1 ? a.nkv * ((len + kTile - 1) / kTile) : 0;
    });
    const int W = pre[a.kv.n_req], G = max(1, min((int)gridDim.x, W));  // no block between two others is empty
    const bool busy = W > 0 && (int)blockIdx.x < G;
    const int x0 = busy ? (int)cut(W, G, blockIdx.x) : 0, x1 = busy ? (int)cut(W, G, blockIdx.x + 1) : 0;
    const int pshift = 31 - __clz(a.piece), shift = 31 - __clz(a.kv.page);

    if (warp == 8) {
        // ---------------- producer: a tile's pages, one copy per page piece
        int i = 0;
        bool ok = true;
        for (int x = x0; ok && x < x1;) {
            const DecSeg s = dec_seg(a, pre, x, x1);
            const int32_t* table = a.kv.table + (size_t)s.r * a.kv.max_blocks;
            const int per = kTile >> pshift;  // pieces of a tile
            int have = -1, entry = 0;         // 32 pieces' slots in the lanes, from piece `have` on
            for (int kt = s.k0; kt < s.k1; ++kt, ++i) {
                const int p0 = kt * per, np = min(per, (s.len - kt * kTile + a.piece - 1) >> pshift);
                if (have < 0 || p0 + np > have + 32) {
                    have = p0;
                    const int pos = (p0 + lane) << pshift;
                    entry = a.kv.n_pages << shift;  // past the end: reads as zeros
                    if (pos < s.len) {
                        const int page = table[pos >> shift];
                        if ((unsigned)page < (unsigned)a.kv.n_pages) entry = (page << shift) + (pos & (a.kv.page - 1));
                        else set_status(a.status, ST_BAD_PAGE);
                    }
                }
                const int st = i % ST;
                const uint32_t ph = (i / ST) & 1;
                ok = warp_wait(empty + 8 * st, ph ^ 1, abort_flag, a.status);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(full + 8 * st, (uint32_t)(2 * np) * a.piece * HD * 2);
                __syncwarp();
                const int p = lane >> 1, row = __shfl_sync(0xffffffffu, entry, p0 - have + (lane >> 1));
                if (p < np) {
                    const uint32_t dst = base + st * Lay::STAGE + (lane & 1) * Lay::KV + (uint32_t)(p << pshift) * HD * 2;
                    tma_load_3d(dst, lane & 1 ? &tm_v : &tm_k, 0, row, s.g * (HD / 64), full + 8 * st);
                }
            }
            x += s.k1 - s.k0;
        }
        if (!ok) {  // copies in flight land before the block exits
            for (int k = max(0, i - ST); k < i; ++k) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try(full + 8 * (k % ST), (k / ST) & 1) && globaltimer() - t0 < 1000000ull) {}
            }
        }
        pdl_wait();
        return;
    }

    // ---------------- consumers
    {   // every row's k, v to its slot, while the first tiles are on their way
        const int kvn = a.nkv * HD, per_row = kvn / 4;  // 16-byte vectors of k, then of v
        const long long total = (long long)a.rows * per_row;
        for (long long v = (long long)blockIdx.x * 256 + threadIdx.x; v < total; v += (long long)gridDim.x * 256) {
            const int row = (int)(v / per_row), e = (int)(v % per_row) * 8;
            const int slot = a.slots[row];
            if ((unsigned)slot >= (unsigned)(a.kv.n_pages << shift)) {
                if (slot >= 0) set_status(a.status, ST_BAD_PAGE);
                continue;
            }
            const bf16* src = a.qkv + (size_t)row * ((a.H + 2 * a.nkv) * HD) + (size_t)a.H * HD + e;
            bf16* dst = e < kvn ? (bf16*)a.kv.k + (size_t)slot * kvn + e : (bf16*)a.kv.v + (size_t)slot * kvn + (e - kvn);
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        }
    }
    const int grp = warp >> 2, w = warp & 3;
    int i = 0;
    bool ok = true;
    for (int x = x0; x < x1;) {
        const DecSeg s = dec_seg(a, pre, x, x1);
        const size_t qrow = (size_t)s.row * ((a.H + 2 * a.nkv) * HD);
        uint32_t q[HD / 16][4];
        {
            const bf16* p0 = a.qkv + qrow + (size_t)(s.g * a.Hg + (lane >> 2)) * HD + (lane & 3) * 2;
            const bool lo = (lane >> 2) < a.Hg, hi = (lane >> 2) + 8 < a.Hg;
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                q[k][0] = lo ? *reinterpret_cast<const uint32_t*>(p0 + 16 * k) : 0u;
                q[k][1] = hi ? *reinterpret_cast<const uint32_t*>(p0 + 8 * HD + 16 * k) : 0u;
                q[k][2] = lo ? *reinterpret_cast<const uint32_t*>(p0 + 16 * k + 8) : 0u;
                q[k][3] = hi ? *reinterpret_cast<const uint32_t*>(p0 + 8 * HD + 16 * k + 8) : 0u;
            }
        }
        float acc[NB][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
        for (int kt = s.k0; kt < s.k1; ++kt, ++i) {
            if ((i & 1) != grp) continue;
            const int st = i % ST;
            if (ok) ok = warp_wait(full + 8 * st, (i / ST) & 1, abort_flag, a.status);
            if (!ok) continue;
            const uint32_t sk = base + st * Lay::STAGE, sv = sk + Lay::KV;
            const int valid = s.len - kt * kTile - w * 16;  // of this warp's 16 keys
            if (valid > 0) {
                if (valid <= 16) {
                    // the request's end: the new key and value come from the step's rows, and values behind
                    // it are cleared (their weight is 0, but a page may hold anything there)
                    for (int v = lane; v < (16 - valid) * (HD / 8); v += 32)
                        *reinterpret_cast<uint4*>(smem_dyn + (sv - base) + dec_at<HD>(w * 16 + valid + v / (HD / 8), v % (HD / 8), pshift)) =
                            make_uint4(0, 0, 0, 0);
                    const bf16* src = a.qkv + qrow + (size_t)(a.H + s.g) * HD;
                    for (int v = lane; v < 2 * (HD / 8); v += 32) {
                        const bool isv = v >= HD / 8;
                        const int j = isv ? v - HD / 8 : v;
                        *reinterpret_cast<uint4*>(smem_dyn + ((isv ? sv : sk) - base) + dec_at<HD>(w * 16 + valid - 1, j, pshift)) =
                            *reinterpret_cast<const uint4*>(src + (isv ? (size_t)a.nkv * HD : 0) + 8 * j);
                    }
                    __syncwarp();
                }
                float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                const int kkey = w * 16 + ((lane >> 4) << 3) + (lane & 7), kj = (lane >> 3) & 1;
#pragma unroll
                for (int k = 0; k < HD / 16; ++k) {
                    uint32_t b[4];
                    ldmatrix4(sk + dec_at<HD>(kkey, 2 * k + kj, pshift), b);
                    mma16816(sc[0], q[k], b[0], b[1]);
                    mma16816(sc[1], q[k], b[2], b[3]);
                }
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = n * 8 + (lane & 3) * 2 + (e & 1);
                        sc[n][e] = key < valid ? sc[n][e] * a.scale_log2 : -INFINITY;
                        mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
                    }
                bool grow = false;
                float mu[2], al[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                    // the maximum moves only when it grows by more than 2^8: P stays below 2^8
                    const bool up = mx[h] > m[h] + 8.f;
                    al[h] = up ? ex2(m[h] - mx[h]) : 1.f;
                    if (up) m[h] = mx[h];
                    mu[h] = m[h] == -INFINITY ? 0.f : m[h];
                    grow |= up;
                }
                uint32_t p[4];
                float pe[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) pe[n][e] = ex2(sc[n][e] - mu[e >> 1]);
                l[0] = l[0] * al[0] + ((pe[0][0] + pe[0][1]) + (pe[1][0] + pe[1][1]));
                l[1] = l[1] * al[1] + ((pe[0][2] + pe[0][3]) + (pe[1][2] + pe[1][3]));
                p[0] = pack2(pe[0][0], pe[0][1]);
                p[1] = pack2(pe[0][2], pe[0][3]);
                p[2] = pack2(pe[1][0], pe[1][1]);
                p[3] = pack2(pe[1][2], pe[1][3]);
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        acc[n][0] *= al[0]; acc[n][1] *= al[0];
                        acc[n][2] *= al[1]; acc[n][3] *= al[1];
                    }
                }
                const int vkey = w * 16 + (lane & 15), vj = lane >> 4;
#pragma unroll
                for (int n = 0; n < NB / 2; ++n) {
                    uint32_t b[4];
                    ldmatrix4_t(sv + dec_at<HD>(vkey, 2 * n + vj, pshift), b);
                    mma16816(acc[2 * n], p, b[0], b[1]);
                    mma16816(acc[2 * n + 1], p, b[2], b[3]);
                }
                if (valid <= 16) fence_proxy_async_smem();  // this warp wrote to the stage
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * st);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        // the warps' outputs into one, the upper half of them at a time (the same order always)
#pragma unroll
        for (int half = 4; half > 0; half >>= 1) {
            if (warp >= half && warp < 2 * half) {
                float* to = red + (warp - half) * (Lay::RED_W / 4) + lane;
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) to[(4 * n + e) * 32] = acc[n][e];
                to[(4 * NB) * 32] = m[0]; to[(4 * NB + 1) * 32] = m[1];
                to[(4 * NB + 2) * 32] = l[0]; to[(4 * NB + 3) * 32] = l[1];
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (warp < half) {
                const float* from = red + warp * (Lay::RED_W / 4) + lane;
                float c0[2], c1[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float om = from[(4 * NB + h) * 32], ol = from[(4 * NB + 2 + h) * 32];
                    const float M = fmaxf(m[h], om);
                    c0[h] = m[h] == -INFINITY ? 0.f : ex2(m[h] - M);
                    c1[h] = om == -INFINITY ? 0.f : ex2(om - M);
                    l[h] = l[h] * c0[h] + ol * c1[h];
                    m[h] = M;
                }
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[n][e] = acc[n][e] * c0[e >> 1] + from[(4 * n + e) * 32] * c1[e >> 1];
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        if (warp == 0 && ok) {
            const bool whole = s.k0 == 0 && s.k1 == s.tiles;
            const int slot = 2 * (int)blockIdx.x + (x == x0 ? 0 : 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int hr = (lane >> 2) + 8 * h;
                if (hr >= a.Hg) continue;
                if (whole) {
                    const float inv = 1.f / l[h];
                    bf16* to = a.o + (size_t)s.row * a.H * HD + (size_t)(s.g * a.Hg + hr) * HD + (lane & 3) * 2;
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        *reinterpret_cast<uint32_t*>(to + 8 * n) = pack2(acc[n][2 * h] * inv, acc[n][2 * h + 1] * inv);
                } else {
                    float* to = a.part.o + ((size_t)slot * kDecRows + hr) * HD + (lane & 3) * 2;
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        *reinterpret_cast<float2*>(to + 8 * n) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
                    if ((lane & 3) == 0) a.part.ml[(size_t)slot * kDecRows + hr] = make_float2(m[h], l[h]);
                }
            }
        }
        x += s.k1 - s.k0;
    }
    if (threadIdx.x == 0) {
        int4 d = make_int4(0, 0, 0, 0);
        if (x0 < x1 && ok) {
            const DecSeg s = dec_seg(a, pre, x1 - 1, x1);  // the block's last (request, K/V head)
            const long long end = s.unit + s.tiles;
            if (s.unit >= x0 && end > x1)
                d = make_int4(s.row, s.g, 2 * (block_of(W, G, end - 1) - (int)blockIdx.x + 1) + (s.unit == x0 ? 0 : 1), 1);
        }
        a.part.desc[blockIdx.x] = d;
    }
    pdl_wait();
}

// ---------------------------------------------------------------- joining the pieces
// Block (c, y): rows of the output that begins in block c of the attention's grid and
// goes on in the next ones; WPR warps to a row, each with every WPR-th piece.
template <int HD, int WPR>
__global__ void __launch_bounds__(256) paged_join_kernel(const Partials part, int half, int tokens, int H, int Hg,
                                                         bf16* __restrict__ o) {
    constexpr int E = HD / 32, RPB = 8 / WPR;
    __shared__ float s_o[8][HD];
    __shared__ float2 s_ml[8];
    pdl_trigger();
    pdl_wait();
    const int4 d = part.desc[blockIdx.x];
    const int n = d.z >> 1;
    if (n == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = blockIdx.y * RPB + warp / WPR, rows = half * (tokens * Hg <= half && half > kDecRows ? 2 : 1);
    const int in = i % half, tok = (i / half) * tokens + in / Hg;
    const bool live = i < rows && in < tokens * Hg && tok < d.w;
    float acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (live) {
        for (int k = warp % WPR; k < n; k += WPR) {
            const size_t at = (size_t)(2 * (blockIdx.x + k) + (k == 0 ? d.z & 1 : 0)) * rows + i;
            const float2 ml = part.ml[at];
            float v[E];
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 t = *reinterpret_cast<const float2*>(part.o + at * HD + lane * E + e);
                v[e] = t.x; v[e + 1] = t.y;
            }
            const float M = fmaxf(m, ml.x);
            const float c0 = m == -INFINITY ? 0.f : ex2(m - M), c1 = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = acc[e] * c0 + (c1 > 0.f ? v[e] * c1 : 0.f);
            l = l * c0 + ml.y * c1;
            m = M;
        }
    }
    if (WPR > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (warp % WPR != 0) return;
#pragma unroll
        for (int k = 1; k < WPR; ++k) {
            const float2 ml = s_ml[warp + k];
            const float M = fmaxf(m, ml.x);
            const float c0 = m == -INFINITY ? 0.f : ex2(m - M), c1 = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = acc[e] * c0 + s_o[warp + k][lane * E + e] * c1;
            l = l * c0 + ml.y * c1;
            m = M;
        }
    }
    if (!live) return;
    const float inv = 1.f / l;
    bf16* to = o + (size_t)(d.x + tok) * H * HD + (size_t)(d.y * Hg + in % Hg) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(to + e) = pack2(acc[e] * inv, acc[e + 1] * inv);
}

// ---------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// bf16 tensor map with the 128-byte swizzle, zeros outside; strides in bytes of dims 1...
bool encode(CUtensorMap* map, const void* ptr, int nd, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, nd, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A page pool [slots, nkv * hd] as [64-column block][slot][64]: one copy brings
// `piece` slots of all of a head's column blocks.
bool map_pool(CUtensorMap* map, const void* ptr, int nkv, int hd, const PagedKv& kv, int piece) {
    const cuuint64_t ld = (cuuint64_t)nkv * hd * 2;
    const cuuint64_t dims[3] = {64, (cuuint64_t)kv.n_pages * kv.page, (cuuint64_t)nkv * hd / 64}, strides[2] = {ld, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)piece, (cuuint32_t)hd / 64};
    return encode(map, ptr, 3, dims, strides, box);
}

cudaError_t launch_pdl(const void* func, dim3 grid, int threads, int smem, cudaStream_t s, void** args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, func, args);
    if (e == cudaSuccess) count_launch();
    return e;
}

bool decode_takes(DType at, int H, int nkv, int hd, int max_new) {
    return at == DT_BF16 && (hd == 64 || hd == 128) && H / nkv <= kDecRows && max_new == 1;
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t partial_bytes(int blocks, int rows, int hd) {
    return al256((size_t)2 * blocks * rows * hd * 4) + al256((size_t)2 * blocks * rows * 8) + al256((size_t)blocks * 16);
}
Partials partials(char* ws, int blocks, int rows, int hd) {
    Partials p;
    p.o = reinterpret_cast<float*>(ws);
    ws += al256((size_t)2 * blocks * rows * hd * 4);
    p.ml = reinterpret_cast<float2*>(ws);
    ws += al256((size_t)2 * blocks * rows * 8);
    p.desc = reinterpret_cast<int4*>(ws);
    return p;
}

template <int HD>
cudaError_t decode(DecodeArgs a, void* ws, cudaStream_t s) {
    using Lay = DecLayout<HD>;
    cudaError_t e = ensure_smem_limit((const void*)paged_decode_kernel<HD>, Lay::bytes(kMaxRequests));
    if (e != cudaSuccess) return e;
    const int G = device_sm_count();
    a.part = partials((char*)ws, G, kDecRows, HD);
    a.piece = std::min(a.kv.page, kTile);
    CUtensorMap tk, tv;
    if (!map_pool(&tk, a.kv.k, a.nkv, HD, a.kv, a.piece) || !map_pool(&tv, a.kv.v, a.nkv, HD, a.kv, a.piece))
        return cudaErrorUnknown;
    paged_decode_kernel<HD><<<G, kDecThreads, Lay::bytes(a.kv.n_req), s>>>(tk, tv, a);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    int half = kDecRows, tokens = 1;
    void* args[] = {&a.part, &half, &tokens, &a.H, &a.Hg, &a.o};
    return launch_pdl((const void*)paged_join_kernel<HD, 4>, dim3(G, (a.Hg + 1) / 2), 256, 0, s, args);
}

}  // namespace

size_t paged_attention_workspace(DType at, int H, int nkv, int hd) {
    if (!decode_takes(at, H, nkv, hd, 1)) return 256;
    return partial_bytes(device_sm_count(), kDecRows, hd);
}

cudaError_t paged_attention(DType at, const void* qkv, int H, int nkv, int hd, int rows, int max_new,
                            const int32_t* slots, const PagedKv& kv, void* o, void* workspace, int* status,
                            cudaStream_t s) {
    if (decode_takes(at, H, nkv, hd, max_new)) {
        DecodeArgs a{};
        a.qkv = reinterpret_cast<const bf16*>(qkv);
        a.slots = slots;
        a.kv = kv;
        a.o = reinterpret_cast<bf16*>(o);
        a.H = H; a.nkv = nkv; a.Hg = H / nkv; a.rows = rows; a.max_new = max_new;
        a.scale_log2 = kLog2eF / sqrtf((float)hd);
        a.status = status;
        return hd == 128 ? decode<128>(a, workspace, s) : decode<64>(a, workspace, s);
    }
    cudaError_t e = launch_paged_append(at, qkv, H, nkv, hd, rows, slots, kv, status, s);
    if (e != cudaSuccess) return e;
    return launch_paged_attention_simt(at, qkv, H, nkv, hd, rows, kv, o, status, s);
}

}  // namespace nc
