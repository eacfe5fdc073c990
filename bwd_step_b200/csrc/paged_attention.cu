// Attention of a step's new tokens over the paged cache, bf16, on the tensor cores.
//
// Chunks (two new tokens or more) run on tcgen05 in tiles of 128 rows, a row being a
// (token, query head).  Bound by the cycle scores -> softmax -> output of a tile: two
// chunks of some 2000 rows on 5500 positions, 10 heads of 128, take 143 to 155 us, as the
// power limit lets the clock be (126 GFLOP, 815 to 880 TFLOP/s).
// Decoding requests (one new token): per K/V head the group's query heads, 16 at
// most, are the rows of one small matrix product against every cached key, so
// each key and value is read once for all of them.  Bound by HBM: 128 requests of 900
// to 8191 positions (290 MB) take 57 us, the kernel itself 52 (5.6 TB/s).
//
// Work is cut evenly over the SMs: the requests' key tiles of all K/V heads form
// one line, whose W tiles are dealt out in order, W / G to each of G blocks.
// A unit (a (request, K/V head), or a part of a chunk) that lies in one block is finished
// there; one that is cut leaves a partial output, row maximum and sum in each of its
// blocks, and a last kernel joins them in the blocks' order, so the result does not depend on timing.
// A block has at most two partial results: its first and its last piece.
#include "paged.h"
#include "tc_common.cuh"
#include <cudaTypedefs.h>
#include <algorithm>

namespace nc {
namespace {
using namespace tc;

constexpr int kTile = 64;        // keys of a decode tile
// Where the table has no more positions than this, nothing is cut over blocks and there is nothing to
// join.  Graph times, whole / cut, us, 10 heads of 128:
//   steps with chunks of some 225 rows on up to 700 positions: 8 requests 27 / 35, 64 requests 109 / 117;
//   one alone on 600 to 700 positions 27 / 22, the one case here that cutting would serve;
//   steps of decoding requests alone, 4 and 148 of them: table of 128 positions 6.3 / 7.8 and 8.0 / 8.2, of 256
//   7.6 / 7.7 and 12.2 / 13.7, of 512 9.5 / 8.4 and 15.6 / 17.2, of 1024 13.2 / 8.7 and 24.6 / 22.6.
constexpr int kWholePositions = 1024, kWholeDecoding = 256;
constexpr int kDecRows = 16;     // query heads of a K/V head that the decode kernel takes
constexpr int kDecThreads = 320; // 8 consumer warps, the producer, and one that writes the cache
constexpr float kLog2eF = 1.44269504088896340736f;

// Partial results of the G blocks, two pieces each.  `desc` tells of the unit that begins in a
// block and goes on in the next ones: first packed row, K/V head, 2 * (blocks it lies in) + (its
// piece's slot here; 0 in the others), tokens; z = 0: none.
struct Partials {
    float* o;    // [2 G, rows, HD] unnormalised
    float2* ml;  // [2 G, rows] maximum (log2 domain), sum
    int4* desc;  // [G]
};

struct DecodeArgs {
    const bf16* qkv;
    const int32_t* slots;
    PagedKv kv;
    bf16* o;
    Partials part;
    int H, nkv, Hg, rows, piece, max_new;  // piece: rows of one copy, min(page, kTile)
    bool whole;                            // no (request, K/V head) is cut
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

// The line of W tiles cut over G blocks: the first W % G of them have one tile more.
template <typename T>
struct Cut {
    T each;
    int more;
    __device__ __forceinline__ Cut(T W, int G) : each(W / (unsigned)G), more((int)(W - each * (unsigned)G)) {}
    __device__ __forceinline__ T first(int c) const { return each * (unsigned)c + (unsigned)min(c, more); }  // tile of block c
    __device__ __forceinline__ int block(T x) const {  // that has tile x
        const T big = (each + 1) * (unsigned)more;
        return x < big ? (int)(x / (each + 1)) : more + (int)((x - big) / each);
    }
};

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
    static constexpr int QS = 3;                            // pieces whose query rows, and new k and v, are brought ahead
    static constexpr int Q_BYTES = (kDecRows + 2) * HD * 2;
    static constexpr int Q = STAGES * STAGE;
    static constexpr int RED = Q + QS * Q_BYTES;            // 8 warps' outputs, 64 columns at a time
    static constexpr int RED_LD = 68;                       // floats of a row
    static constexpr int ML = RED + 8 * kDecRows * RED_LD * 4;  // [8][16] maximum, sum
    static constexpr int BAR = ML + 8 * kDecRows * 8;
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
// 16 rows: a tile's 32 KB of operands (head size 128) take 1400 cycles to arrive at an
// SM's share of the bandwidth and some 300 to multiply, and tcgen05's 128 rows would be an eighth full.
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
    float2* red_ml = reinterpret_cast<float2*>(smem_dyn + Lay::ML);
    const uint32_t full = base + Lay::BAR, empty = full + 8 * ST, q_full = empty + 8 * ST, q_empty = q_full + 8 * Lay::QS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_dyn + Lay::BAR + 16 * (ST + Lay::QS));
    int* pre = reinterpret_cast<int*>(smem_dyn + Lay::PRE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int st = 0; st < ST; ++st) {
            mbar_init(full + 8 * st, 1);
            mbar_init(empty + 8 * st, 4);
        }
        for (int st = 0; st < Lay::QS; ++st) {
            mbar_init(q_full + 8 * st, 1);
            mbar_init(q_empty + 8 * st, 8);
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
    const Cut<unsigned> line((unsigned)W, G);
    auto edge = [&](int c) {  // first tile of block c
        const int x = (int)line.first(c);
        if (!a.whole || x >= W) return x;
        const DecSeg s = dec_seg(a, pre, x, W);
        return s.k0 ? x - s.k0 + s.tiles : x;
    };
    const int x0 = busy ? edge(blockIdx.x) : 0, x1 = busy ? edge(blockIdx.x + 1) : 0;
    const int pshift = 31 - __clz(a.piece), shift = 31 - __clz(a.kv.page);

    if (warp == 8) {
        // ---------------- producer: a tile's pages, one copy per page piece
        int i = 0, k = 0;
        bool ok = true;
        for (int x = x0; ok && x < x1; ++k) {
            const DecSeg s = dec_seg(a, pre, x, x1);
            const int32_t* table = a.kv.table + (size_t)s.r * a.kv.max_blocks;
            const int per = kTile >> pshift;  // pieces of a tile
            int have, entry;                  // 32 pieces' slots in the lanes, from piece `have` on
            auto entries = [&](int p0) {
                have = p0;
                const int pos = (p0 + lane) << pshift;
                entry = a.kv.n_pages << shift;  // past the end: reads as zeros
                if (pos < s.len) {
                    const int page = table[pos >> shift];
                    if ((unsigned)page < (unsigned)a.kv.n_pages) entry = (page << shift) + (pos & (a.kv.page - 1));
                    else set_status(a.status, ST_BAD_PAGE);
                }
            };
            entries(s.k0 * per);
            ok = warp_wait(q_empty + 8 * (k % Lay::QS), ((k / Lay::QS) & 1) ^ 1, abort_flag, a.status);
            if (!ok) break;
            if (lane == 0) {
                const uint32_t to = base + Lay::Q + (k % Lay::QS) * Lay::Q_BYTES, bar = q_full + 8 * (k % Lay::QS);
                const bf16* from = a.qkv + (size_t)s.row * ((a.H + 2 * a.nkv) * HD);
                mbar_expect_tx(bar, (uint32_t)(a.Hg + 2) * HD * 2);
                bulk_load(to, from + (size_t)s.g * a.Hg * HD, (uint32_t)a.Hg * HD * 2, bar);
                bulk_load(to + kDecRows * HD * 2, from + (size_t)(a.H + s.g) * HD, HD * 2, bar);
                bulk_load(to + (kDecRows + 1) * HD * 2, from + (size_t)(a.H + a.nkv + s.g) * HD, HD * 2, bar);
            }
            __syncwarp();
            for (int kt = s.k0; kt < s.k1; ++kt, ++i) {
                const int p0 = kt * per, np = min(per, (s.len - kt * kTile + a.piece - 1) >> pshift);
                if (p0 + np > have + 32) entries(p0);
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
            auto drain = [&](uint32_t bar, uint32_t parity) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try(bar, parity) && globaltimer() - t0 < 1000000ull) {}
            };
            for (int t = max(0, i - ST); t < i; ++t) drain(full + 8 * (t % ST), (t / ST) & 1);
            for (int t = max(0, k + 1 - Lay::QS); t <= k; ++t) drain(q_full + 8 * (t % Lay::QS), (t / Lay::QS) & 1);
        }
        pdl_wait();
        return;
    }
    if (warp == 9) {
        // ---------------- every row's k, v to its slot, eight vectors of a thread on their way
        constexpr int U = 8;
        const int kvn = a.nkv * HD, per_row = kvn / 4;  // 16-byte vectors of k, then of v
        const long long total = (long long)a.rows * per_row, step = (long long)gridDim.x * 32;
        for (long long v0 = (long long)blockIdx.x * 32 + lane; v0 < total; v0 += U * step) {
            int slot[U], e[U];
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long v = v0 + u * step;
                slot[u] = -1;
                if (v >= total) continue;
                const int row = (int)(v / per_row);
                e[u] = (int)(v % per_row) * 8;
                slot[u] = a.slots[row];
                x[u] = *reinterpret_cast<const uint4*>(a.qkv + (size_t)row * ((a.H + 2 * a.nkv) * HD) + (size_t)a.H * HD + e[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if ((unsigned)slot[u] < (unsigned)(a.kv.n_pages << shift))
                    *reinterpret_cast<uint4*>(e[u] < kvn ? (bf16*)a.kv.k + (size_t)slot[u] * kvn + e[u]
                                                         : (bf16*)a.kv.v + (size_t)slot[u] * kvn + (e[u] - kvn)) = x[u];
                else if (slot[u] >= 0)
                    set_status(a.status, ST_BAD_PAGE);
            }
        }
        if (lane == 0) {
            int4 d = make_int4(0, 0, 0, 0);
            if (x0 < x1) {
                const DecSeg s = dec_seg(a, pre, x1 - 1, x1);  // the block's last (request, K/V head)
                const long long end = s.unit + s.tiles;
                if (s.unit >= x0 && end > x1)
                    d = make_int4(s.row, s.g, 2 * (line.block((unsigned)(end - 1)) - (int)blockIdx.x + 1) + (s.unit == x0 ? 0 : 1), 1);
            }
            a.part.desc[blockIdx.x] = d;
        }
        pdl_wait();
        return;
    }

    // ---------------- consumers
    const int grp = warp >> 2, w = warp & 3;
    int i = 0, piece = 0;
    bool ok = true;
    for (int x = x0; x < x1; ++piece) {
        const DecSeg s = dec_seg(a, pre, x, x1);
        const uint32_t q_at = Lay::Q + (piece % Lay::QS) * Lay::Q_BYTES;  // query rows, then the new k and v
        if (ok) ok = warp_wait(q_full + 8 * (piece % Lay::QS), (piece / Lay::QS) & 1, abort_flag, a.status);
        uint32_t q[HD / 16][4];
        {
            const uint8_t* p0 = smem_dyn + q_at + (lane >> 2) * (HD * 2) + (lane & 3) * 4;
            const bool lo = (lane >> 2) < a.Hg, hi = (lane >> 2) + 8 < a.Hg;
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                q[k][0] = lo ? *reinterpret_cast<const uint32_t*>(p0 + 32 * k) : 0u;
                q[k][1] = hi ? *reinterpret_cast<const uint32_t*>(p0 + 16 * HD + 32 * k) : 0u;
                q[k][2] = lo ? *reinterpret_cast<const uint32_t*>(p0 + 32 * k + 16) : 0u;
                q[k][3] = hi ? *reinterpret_cast<const uint32_t*>(p0 + 16 * HD + 32 * k + 16) : 0u;
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
                    for (int v = lane; v < 2 * (HD / 8); v += 32) {
                        const bool isv = v >= HD / 8;
                        const int j = isv ? v - HD / 8 : v;
                        *reinterpret_cast<uint4*>(smem_dyn + ((isv ? sv : sk) - base) + dec_at<HD>(w * 16 + valid - 1, j, pshift)) =
                            *reinterpret_cast<const uint4*>(smem_dyn + q_at + kDecRows * HD * 2 + 16 * v);
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
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty + 8 * (piece % Lay::QS));
        // the warps' outputs into one, 64 columns at a time, the warps always in the same order
        if ((lane & 3) == 0) {
            red_ml[warp * kDecRows + (lane >> 2)] = make_float2(m[0], l[0]);
            red_ml[warp * kDecRows + 8 + (lane >> 2)] = make_float2(m[1], l[1]);
        }
        const bool whole = s.k0 == 0 && s.k1 == s.tiles;
        const int slot = 2 * (int)blockIdx.x + (x == x0 ? 0 : 1);
        const int row = threadIdx.x >> 4, col = (threadIdx.x & 15) * 4;  // of the joined output, and 64 c more columns
        float f[8], L = 0.f, M = -INFINITY;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                float* to = red + (warp * kDecRows + (lane >> 2)) * Lay::RED_LD + 8 * n + 2 * (lane & 3);
                *reinterpret_cast<float2*>(to) = make_float2(acc[8 * c + n][0], acc[8 * c + n][1]);
                *reinterpret_cast<float2*>(to + 8 * Lay::RED_LD) = make_float2(acc[8 * c + n][2], acc[8 * c + n][3]);
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (c == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k) M = fmaxf(M, red_ml[k * kDecRows + row].x);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 ml = red_ml[k * kDecRows + row];
                    f[k] = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
                    L += ml.y * f[k];
                }
            }
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(red + (k * kDecRows + row) * Lay::RED_LD + col);
                o.x = fmaf(v.x, f[k], o.x); o.y = fmaf(v.y, f[k], o.y);
                o.z = fmaf(v.z, f[k], o.z); o.w = fmaf(v.w, f[k], o.w);
            }
            if (row < a.Hg && ok) {
                if (whole) {
                    const float inv = 1.f / L;
                    *reinterpret_cast<uint2*>(a.o + (size_t)s.row * a.H * HD + (size_t)(s.g * a.Hg + row) * HD + 64 * c + col) =
                        make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
                } else {
                    *reinterpret_cast<float4*>(a.part.o + ((size_t)slot * kDecRows + row) * HD + 64 * c + col) = o;
                    if (c == 0 && col == 0) a.part.ml[(size_t)slot * kDecRows + row] = make_float2(M, L);
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        x += s.k1 - s.k0;
    }
    pdl_wait();
}

// ---------------------------------------------------------------- chunks
// A unit is 2 x `tt` new tokens of a request with the Hg query heads of one K/V head:
// two halves of tt * Hg <= 128 rows (row i: token i / Hg, head i % Hg) that share the
// unit's K and V tiles of 128 keys, so that a chunk fills the tensor core's 128 rows
// whatever its length and K and V are read once for all heads.  The units' key tiles
// form the line that is cut over the SMs.
//   warp 8     TMA: Q of both halves (a [tt][Hg][64] box per 64 columns), then K_j and
//              V_j into two rings, one copy per page piece and 64 columns, K one tile
//              ahead of V; the lanes hold 32 pieces' slots and issue a copy each;
//   warp 9     tcgen05.mma in the order ... O_a += P_a(j) V_j, S_a(j+1), O_b += P_b(j)
//              V_j, S_b(j+1) ...: S = Q K^T into the half's 128 TMEM score columns,
//              O += P V with P read from TMEM over the first half of them and V as an
//              MN-major operand;
//   warps 0-3  softmax of half a, warps 4-7 of half b: a row per thread, running maximum
//              in the log2 domain that moves only when it grows by 2^8, P as packed bf16.
// A half's scores, softmax and output wait for each other; the other half's run meanwhile.
// Both take some 3200 cycles a tile (long chunks, 55 tiles a block), where the products alone take 2048
// and the softmax of both halves 2000.  That is 176 thousand of a block's 207 thousand cycles; its start
// takes 9, the pieces' first copies and products 11 and their output 11.
constexpr int kChunkThreads = 320;  // softmax of half a, of half b (a warpgroup each); producer, MMA
constexpr int kChunkRows = 256;
// Units of so many key tiles are not cut: 8 requests of some 900 positions 33.9 -> 30.5 us.  The rule does not ask
// how many units there are: chunks of 20 rows on 1200 positions take, whole / cut, 36.3 / 37.1 us for 64 requests, but
// 31.5 / 20.9 for 8 and 30.1 / 18.5 for one, in whose ten tiles one SM walks while the others idle.
constexpr int kWholeTiles = 10;

struct ChunkArgs {
    PagedKv kv;
    bf16* o;
    Partials part;
    int H, nkv, Hg, tt, rows, piece, max_new;  // piece: rows of one copy, min(page, 128)
    bool skip_one;                             // requests with one new row are the decode kernel's
    float scale_log2;
    int* status;

    // Whether request r is this kernel's, and its first row, new rows and length.
    __device__ __forceinline__ bool takes(int r, int& row, int& n, int& len) const {
        return request(kv, rows, r, row, n, len) && n > (skip_one ? 1 : 0);
    }
    // Key tiles of request r over all K/V heads.
    __device__ __forceinline__ long long tiles(int r) const;
};

constexpr int kGroup = 16;  // requests that one entry of the chunk kernel's prefix sums stands for

template <int HD>
struct ChunkLayout {
    static constexpr int KB = HD / 64;
    static constexpr int TILE = KB * 16384;  // [128 x HD] bf16, 128B-swizzled
    static constexpr int KVSTG = HD == 128 ? 2 : 3;
    static constexpr int K = 2 * TILE;
    static constexpr int V = K + KVSTG * TILE;
    static constexpr int BAR = V + KVSTG * TILE;
    static constexpr int OUT = BAR + 256;         // 4 KB a softmax warp: its output's way to whole lines
    static constexpr int PRE = OUT + 8 * 4096;    // [groups of requests + 1]
    static constexpr int bytes(int n_req) { return PRE + ((n_req + kGroup - 1) / kGroup + 1) * 8; }
};
static_assert(ChunkLayout<128>::bytes(kMaxRequests) <= 232448, "chunk shared memory exceeds the per-block limit");

// sum of floor((a i + b) / 128) over i < n, for a <= 256 (the floor sum of an arithmetic progression, by
// the Euclidean algorithm): the whole parts are taken out, then what is left counts the lattice points
// under a line, whose axes are exchanged until none is.
__device__ __forceinline__ long long floor_sum128(unsigned n, unsigned a, unsigned b) {
    long long sum = (long long)n * (b >> 7);
    unsigned m = 128;
    b &= 127;
    while (n) {
        if (a >= m) { sum += (long long)n * (n - 1) / 2 * (a / m); a %= m; }
        if (b >= m) { sum += (long long)n * (b / m); b %= m; }
        const unsigned y = a * n + b;  // a < 128, n < 2^24: below 2^31
        n = y / m;
        b = y % m;
        const unsigned t = m;
        m = a;
        a = t;
    }
    return sum;
}

// Key tiles of a request's chunk for one K/V head: over its units, the tiles up to each one's last token.
__device__ __forceinline__ long long chunk_tiles(int n, int len, int unit) {
    const int full = (n - 1) / unit;  // all but the chunk's last unit end `unit` tokens further on
    return (full ? floor_sum128(full, unit, len - n + unit + 127) : 0) + ((len + 127) >> 7);
}

__device__ __forceinline__ long long ChunkArgs::tiles(int r) const {
    int row, n, len;
    return r < kv.n_req && takes(r, row, n, len) ? nkv * chunk_tiles(n, len, 2 * tt) : 0;
}

// Walks the pieces of a block's part [x, x1) of the line; every role of the block walks alike.
struct ChunkWalk {
    long long x, x1, unit;     // unit: the current unit's first tile in the line
    int r, g, b, row, n, len;  // request, K/V head, unit of the chunk; its first packed row, new rows, length
    bool whole;                // pieces are whole units: those that begin in the part
    int tok0, toks, end, tiles, k0, k1;  // the unit's tokens [tok0, tok0 + toks), keys and tiles; the piece's tiles

    __device__ __forceinline__ void set(const ChunkArgs& a) {
        tok0 = b * 2 * a.tt;
        toks = min(n - tok0, 2 * a.tt);
        end = len - n + tok0 + toks;
        tiles = (end + 127) >> 7;
    }
    // Out of line, so that the walk's state waits in local memory while a piece is worked on.
    // By whole warps: the lanes look at a group's requests, then at 32 units, at once.
    __device__ __forceinline__ void start(const ChunkArgs& a, const long long* pre, long long from, long long to, bool units) {
        x = from; x1 = to;
        whole = units;
        if (x >= x1) return;
        const int lane = threadIdx.x & 31, groups = (a.kv.n_req + kGroup - 1) / kGroup;
        const int gr = find_request(pre, groups, x);
        const long long mine = lane < kGroup ? a.tiles(gr * kGroup + lane) : 0;
        long long before = mine;
#pragma unroll
        for (int o = 1; o < kGroup; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        before += pre[gr] - mine;
        const unsigned in = __ballot_sync(0xffffffffu, lane < kGroup && before <= x && x < before + mine);
        const int at = __ffs(in) - 1;
        r = gr * kGroup + at;
        long long rem = x - __shfl_sync(0xffffffffu, before, at);
        const long long per = __shfl_sync(0xffffffffu, mine, at) / a.nkv;
        request(a.kv, a.rows, r, row, n, len);
        g = (int)(rem / per);
        rem -= g * per;
        // the unit that has tile rem, 32 units at a time
        for (b = 0;; b += 32) {
            const int e = min(n, (b + lane + 1) * 2 * a.tt);
            const int mine = (b + lane) * 2 * a.tt < n ? (len - n + e + 127) >> 7 : 0;
            long long t = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += y;
            }
            const unsigned in = __ballot_sync(0xffffffffu, rem < t);
            if (in) {
                const int at = __ffs(in) - 1;
                rem -= __shfl_sync(0xffffffffu, t - mine, at);
                b += at;
                break;
            }
            rem -= __shfl_sync(0xffffffffu, t, 31);
        }
        set(a);
        k0 = (int)rem;
        unit = x - k0;
        k1 = whole ? tiles : (int)min((long long)tiles, k0 + (x1 - x));
        if (whole && k0 > 0) next(a);  // it began in the block before
    }
    __device__ __forceinline__ void next(const ChunkArgs& a) {
        x += k1 - k0;
        if (x >= x1) return;
        if (tok0 + toks >= n) {
            b = 0;
            if (++g == a.nkv) {
                g = 0;
                while (!a.takes(++r, row, n, len)) {}
            }
        } else {
            ++b;
        }
        set(a);
        unit = x;
        k0 = 0;
        k1 = whole ? tiles : (int)min((long long)tiles, x1 - x);
    }
};

// The three-input maximum.
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 8 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
    tmem_wait_ld();
}

// The one thread of the warp that issues its products.  Chosen by elect.sync, not by its lane, so that
// the compiler knows them to be uniform: beside busy warps a group of eight takes 520 cycles (the tensor
// core's own time) where a branch on the lane takes 960.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// D = A B^T over four K-steps of 16 (64 columns of the tiles), the descriptors 32 bytes apart.
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 q, 0, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        " add.u64 x, %1, 2;\n add.u64 y, %2, 2;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
        " add.u64 x, %1, 4;\n add.u64 y, %2, 4;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n"
        " add.u64 x, %1, 6;\n add.u64 y, %2, 6;\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, q;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D += A B over four K-steps of 16 keys: A in TMEM, 8 columns apart, B MN-major, 2048 bytes apart.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b32 x;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 q, 0, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        " add.u32 x, %1, 8;\n add.u64 y, %2, 128;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n"
        " add.u32 x, %1, 16;\n add.u64 y, %2, 256;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n"
        " add.u32 x, %1, 24;\n add.u64 y, %2, 384;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, q;\n}\n"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int HD>
__global__ void __launch_bounds__(kChunkThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const ChunkArgs a) {
    using Lay = ChunkLayout<HD>;
    constexpr int KB = Lay::KB, TILE = Lay::TILE, KVSTG = Lay::KVSTG;
    extern __shared__ __align__(1024) uint8_t smem_dyn[];
    if ((smem_u32(smem_dyn) & 1023u) != 0) {
        if (threadIdx.x == 0) set_status(a.status, ST_BAD_LAYOUT);
        return;
    }
    pdl_trigger();
    const uint32_t sQ = smem_u32(smem_dyn), sK = sQ + Lay::K, sV = sQ + Lay::V;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem_dyn + Lay::BAR);
    const uint32_t b0 = smem_u32(bars);
    const uint32_t q_full = b0, q_empty = b0 + 8;
    const uint32_t k_full = b0 + 16, k_empty = k_full + 8 * KVSTG;
    const uint32_t v_full = k_empty + 8 * KVSTG, v_empty = v_full + 8 * KVSTG;
    const uint32_t s_full = v_empty + 8 * KVSTG;  // [2] per half
    const uint32_t p_full = s_full + 16, o_full = p_full + 32;  // [2][2] per half, its keys 0-63 and 64-127; [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 10 + 4 * KVSTG);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    long long* pre = reinterpret_cast<long long*>(smem_dyn + Lay::PRE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int st = 0; st < KVSTG; ++st) {
            mbar_init(k_full + 8 * st, 1); mbar_init(k_empty + 8 * st, 1);
            mbar_init(v_full + 8 * st, 1); mbar_init(v_empty + 8 * st, 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full + 8 * x, 1);
            mbar_init(p_full + 16 * x, 4);
            mbar_init(p_full + 16 * x + 8, 4);
            mbar_init(o_full + 8 * x, 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch(&tm_q);
        tma_prefetch(&tm_k);
        tma_prefetch(&tm_v);
    }
    const int groups = (a.kv.n_req + kGroup - 1) / kGroup;
    bool cuts = false;
    for (int base = 0; base < groups * kGroup; base += kChunkThreads) {
        const int r = base + (int)threadIdx.x;
        long long t = a.tiles(r);
        cuts |= t > 0 && a.kv.kv_len[r] > 128 * kWholeTiles;
        if (blockIdx.x == 0 && r < a.kv.n_req) {
            int lo, n, len;
            if (!request(a.kv, a.rows, r, lo, n, len) || (a.max_new > 0 && n > a.max_new)) set_status(a.status, ST_BAD_LENGTH);
        }
#pragma unroll
        for (int o = kGroup / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (r % kGroup == 0 && r / kGroup < groups) pre[r / kGroup] = t;
    }
    // Short units are not cut: a piece saved would cost more to join than it takes.
    const bool units = !__syncthreads_or(cuts);
    if (warp == 0) {  // exclusive prefix sums, 32 groups at a time
        long long run = 0;
        for (int base = 0; base < groups; base += 32) {
            const long long v = base + lane < groups ? pre[base + lane] : 0;
            long long t = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += y;
            }
            if (base + lane < groups) pre[base + lane] = run + t - v;
            run += __shfl_sync(0xffffffffu, t, 31);
        }
        if (lane == 0) pre[groups] = run;
    }
    __syncthreads();
    const long long W = pre[groups];
    const int G = (int)max(1ll, min((long long)gridDim.x, W));
    pdl_wait();  // the new keys and values are in their pages
    if (W == 0 || (int)blockIdx.x >= G) {
        if (threadIdx.x == 0) a.part.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    const Cut<unsigned long long> line(W, G);
    const long long x0 = line.first(blockIdx.x), x1 = line.first(blockIdx.x + 1);
    if (warp == 9) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM: scores (then P) of halves a and b in columns [0, 128) and [128, 256), their
    // outputs O in [256, 256 + HD) and [256 + HD, 256 + 2 HD)

    ChunkWalk w;
    w.start(a, pre, x0, x1, units);
    if (warp == 8) {
        const int pshift = 31 - __clz(a.piece), shift = 31 - __clz(a.kv.page);
        const int per = 128 >> pshift;  // pieces of a tile
        const int p = lane / KB, c = lane % KB;
        const uint32_t bytes_q = (uint32_t)(a.tt * a.Hg) * HD * 2;
        int k = 0, ki = 0, vi = 0, have, entry, k_row = 0, k_np = 0;
        bool ok = true;
        // the tile's first piece's slot of this lane, from the table entries kept in the lanes
        auto load = [&](bool isv, int i, int row, int np) -> bool {
            const int st = i % KVSTG;
            const uint32_t full_b = (isv ? v_full : k_full) + 8 * st, empty_b = (isv ? v_empty : k_empty) + 8 * st;
            if (!warp_wait(empty_b, ((i / KVSTG) & 1) ^ 1, abort_flag, a.status)) return false;
            if (lane == 0) mbar_expect_tx(full_b, (uint32_t)(np << pshift) * HD * 2);
            __syncwarp();
            if (p < np)
                tma_load_2d((isv ? sV : sK) + st * TILE + c * 16384 + (p << pshift) * 128, isv ? &tm_v : &tm_k,
                            w.g * HD + 64 * c, row, full_b);
            return true;
        };
        for (; ok && w.x < w.x1; w.next(a), ++k) {
            if (!warp_wait(q_empty, (k & 1) ^ 1, abort_flag, a.status)) { ok = false; break; }
            const bool two = w.toks > a.tt;
            if (lane == 0) {
                mbar_expect_tx(q_full, two ? 2 * bytes_q : bytes_q);
                for (int h = 0; h < (two ? 2 : 1); ++h)
#pragma unroll
                    for (int cc = 0; cc < KB; ++cc)
                        tma_load_3d(sQ + h * TILE + cc * 16384, &tm_q, 64 * cc, w.g * a.Hg, w.row + w.tok0 + h * a.tt, q_full);
            }
            __syncwarp();
            const int32_t* table = a.kv.table + (size_t)w.r * a.kv.max_blocks;
            have = -1;
            entry = 0;
            auto fetch = [&](int kt) {  // the slots of tile kt's pieces: k_row of this lane, k_np pieces
                const int p0 = kt * per;
                k_np = min(per, (w.end - kt * 128 + a.piece - 1) >> pshift);
                if (have < 0 || p0 + k_np > have + 32) {
                    have = p0;
                    const int pos = (p0 + lane) << pshift;
                    entry = a.kv.n_pages << shift;  // past the end: reads as zeros
                    if (pos < w.end) {
                        const int page = table[pos >> shift];
                        if ((unsigned)page < (unsigned)a.kv.n_pages) entry = (page << shift) + (pos & (a.kv.page - 1));
                        else set_status(a.status, ST_BAD_PAGE);
                    }
                }
                k_row = __shfl_sync(0xffffffffu, entry, p0 - have + p);
            };
            fetch(w.k0);
            if (!load(false, ki++, k_row, k_np)) { ok = false; break; }
            for (int kt = w.k0; kt < w.k1; ++kt) {
                const int row = k_row, np = k_np;
                if (kt + 1 < w.k1) {
                    fetch(kt + 1);
                    if (!load(false, ki++, k_row, k_np)) { ok = false; break; }
                }
                if (!load(true, vi++, row, np)) { ok = false; break; }
            }
        }
        if (!ok && lane == 0) {  // copies in flight land before the block exits (1 ms each at most)
            auto drain = [&](uint32_t bar, uint32_t parity) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try(bar, parity) && globaltimer() - t0 < 1000000ull) {}
            };
            drain(q_full, k & 1);
            for (int i = max(0, ki - KVSTG); i < ki; ++i) drain(k_full + 8 * (i % KVSTG), (i / KVSTG) & 1);
            for (int i = max(0, vi - KVSTG); i < vi; ++i) drain(v_full + 8 * (i % KVSTG), (i / KVSTG) & 1);
        }
    } else if (warp == 9) {
        if (elect_one()) {
            const uint32_t id_s = idesc_bf16(128, 128, false, false);
            const uint32_t id_o = idesc_bf16(128, HD, false, true);
            int k = 0, ki = 0, vi = 0;
            uint32_t pcnt0 = 0, pcnt1 = 0;  // P hand-overs waited for, per half
            bool ok = true;
            auto ready = [&](bool isv, int i) -> bool {
                return mbar_wait((isv ? v_full : k_full) + 8 * (i % KVSTG), (i / KVSTG) & 1, abort_flag, a.status);
            };
            auto scores = [&](int x, int st) {
                const uint64_t dq = smem_desc(sQ + x * TILE, 16, 1024), dk = smem_desc(sK + st * TILE, 16, 1024);
#pragma unroll
                for (int c = 0; c < KB; ++c) mma4(tmem + 128 * x, dq + c * 1024, dk + c * 1024, id_s, c > 0 ? 1u : 0u);
                mma_commit(s_full + 8 * x);
            };
            // O_x += P_x V: keys 16kk..16kk+15 sit in the packed columns 8kk..8kk+7
            auto pv = [&](int x, int st, bool acc) -> bool {
                const uint32_t par = (x ? pcnt1++ : pcnt0++) & 1;
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) {  // the first keys' products run while the others' weights are formed
                    if (!mbar_wait(p_full + 16 * x + 8 * hk, par, abort_flag, a.status)) return false;
                    tc_fence_after();
                    mma4_ts(tmem + 256 + x * HD, tmem + 128 * x + 32 * hk, smem_desc(sV + st * TILE + hk * 8192, 16384, 1024), id_o,
                            acc || hk > 0 ? 1u : 0u);
                }
                return true;
            };
            for (; ok && w.x < w.x1; w.next(a), ++k) {
                const bool two = w.toks > a.tt;
                const int nblk = w.k1 - w.k0;
                if (!mbar_wait(q_full, k & 1, abort_flag, a.status) || !ready(false, ki)) { ok = false; break; }
                tc_fence_after();
                scores(0, ki % KVSTG);
                if (two) scores(1, ki % KVSTG);
                mma_commit(k_empty + 8 * (ki % KVSTG));
                ++ki;
                if (nblk == 1) mma_commit(q_empty);  // the piece's last products that read Q
                for (int j = 0; j < nblk; ++j) {
                    const bool more = j + 1 < nblk;
                    const int vst = vi % KVSTG;
                    if (!ready(true, vi)) { ok = false; break; }
                    // half a: O += P(j) V_j, then S(j+1) (which overwrites P(j) after it, in issue order)
                    if (!pv(0, vst, j > 0)) { ok = false; break; }
                    if (more) {
                        if (!ready(false, ki)) { ok = false; break; }
                        tc_fence_after();
                        scores(0, ki % KVSTG);
                    } else {
                        mma_commit(o_full);
                    }
                    // half b likewise; V_j and (after both halves' scores) K_{j+1} are then released
                    if (two && !pv(1, vst, j > 0)) { ok = false; break; }
                    mma_commit(v_empty + 8 * vst);
                    ++vi;
                    if (more) {
                        if (two) scores(1, ki % KVSTG);
                        mma_commit(k_empty + 8 * (ki % KVSTG));
                        ++ki;
                    } else if (two) {
                        mma_commit(o_full + 8);
                    }
                    if (j + 2 == nblk) mma_commit(q_empty);
                }
            }
        }
    } else if (warp < 8) {
        // ---------------- softmax: half x, TMEM lane quarter q, one row per thread
        const int x = warp >> 2, q = warp & 3;
        const int r = q * 32 + lane;
        const int rt = r / a.Hg;  // token of the half
        const bool in = r < a.tt * a.Hg;
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        const uint32_t tS = tmem + lane_off + 128 * x, tO = tmem + lane_off + 256 + x * HD;
        uint32_t scnt = 0, ocnt = 0;
        int4 d = make_int4(0, 0, 0, 0);
        for (; w.x < w.x1; w.next(a)) {
            if (!w.whole && w.unit >= x0 && w.unit + w.tiles > x1)
                d = make_int4(w.row + w.tok0, w.g,
                              2 * (line.block(w.unit + w.tiles - 1) - (int)blockIdx.x + 1) + (w.unit == x0 ? 0 : 1), w.toks);
            if (x == 1 && w.toks <= a.tt) continue;
            const bool live = in && x * a.tt + rt < w.toks;
            const int k0 = w.k0, k1 = w.k1;
            int first = w.len - w.n + w.tok0 + x * a.tt - k0 * 128;  // position of the half's first token, from the tile's first key
            int lim = live ? first + rt : -1;                        // key c of the tile is visible iff c <= lim
            // the unit's last tile, where it ends inside the tile, and its keys there
            const int cut_tile = x == 0 && k1 == w.tiles && (w.end & 127) ? k1 - 1 : -1, cut_keys = w.end & 127;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int kt = k0; kt < k1; ++kt, first -= 128, lim -= 128) {
                if (!warp_wait(s_full + 8 * x, scnt & 1, abort_flag, a.status)) { ok = false; break; }
                tc_fence_after();
                const bool diag = 127 > first;
                if (kt == cut_tile) {
                    // values behind the unit's keys are cleared (their weight is 0, but a page may
                    // hold anything there).  V_j is released after P(j) V_j, so its barrier is in this tile's phase.
                    const int st = scnt % KVSTG;
                    if (!warp_wait(v_full + 8 * st, (scnt / KVSTG) & 1, abort_flag, a.status)) ok = false;
                    if (ok) {
                        for (int i = cut_keys * 8 + warp * 32 + lane; i < 128 * 8; i += 128)
#pragma unroll
                            for (int c = 0; c < KB; ++c)
                                *reinterpret_cast<uint4*>(smem_dyn + Lay::V + st * TILE + c * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                    }
                }
                if (!ok) break;
                uint32_t sr[128];
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) tmem_ld32_issue(tS + 32 * q4, sr + 32 * q4);
                ++scnt;
                tmem_wait_ld();
                float mx4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) mx4[k] = -INFINITY;
                if (diag) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > lim) sr[c] = 0xff800000u;  // -inf
                }
#pragma unroll
                for (int c = 0; c < 128; c += 2)
                    mx4[(c >> 1) & 3] = max3f(mx4[(c >> 1) & 3], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                mx *= a.scale_log2;
                const bool rescale = live && mx > m + 8.f;  // rows of nothing hold anything
                const float mu = rescale ? mx : m;
                const float alpha = rescale ? ex2(m - mx) : 1.f;
                const float nmu = mu == -INFINITY ? 0.f : -mu;  // no key seen yet: every weight is 2^-inf = 0
                const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), nmu2 = f2_pack(nmu, nmu);
                if (kt > k0 && __any_sync(0xffffffffu, rescale)) {
                    // O_x += P(j-1) V has completed (S(j) was issued after it and has landed);
                    // O_x += P(j) V waits for this warp's hand-over below
#pragma unroll 1
                    for (int c = 0; c < HD; c += 8) {  // few at a time: the scores are live
                        uint32_t o[8];
                        tmem_ld8(tO + c, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st8_nowait(tO + c, o);
                    }
                    tmem_wait_st();
                }
                uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                // P = 2^(s * scale - mu) as packed bf16 over the score columns, 64 keys handed over at a time
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) {
#pragma unroll
                    for (int q8 = 4 * hk; q8 < 4 * hk + 4; ++q8) {
                        uint32_t pk[8];
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const int cc = 16 * q8 + c;
                            const uint64_t y = f2_fma(f2_pack(__uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1])), sc2, nmu2);
                            float e0, e1;
                            f2_unpack(y, e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            sum2[(c >> 1) & 1] = f2_add(sum2[(c >> 1) & 1], f2_pack(e0, e1));
                            pk[c >> 1] = pack2(e0, e1);
                        }
                        tmem_st8_nowait(tS + 8 * q8, pk);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 16 * x + 8 * hk);
                }
                float s00, s01, s10, s11;
                f2_unpack(sum2[0], s00, s01);
                f2_unpack(sum2[1], s10, s11);
                l = l * alpha + ((s00 + s01) + (s10 + s11));
                m = mu;
            }
            if (!ok || !warp_wait(o_full + 8 * x, ocnt & 1, abort_flag, a.status)) break;
            ++ocnt;
            tc_fence_after();
            // Out by whole 128-byte lines: a warp's 32 rows x 128 bytes pass through shared memory (16-byte
            // vectors exchanged by row, so that neither side meets in a bank), four rows to a store.
            uint4* const pass = reinterpret_cast<uint4*>(smem_dyn + Lay::OUT + warp * 4096);
            const bool whole = k0 == 0 && k1 == w.tiles;
            const float inv = 1.f / l;
            const size_t at = (size_t)(2 * blockIdx.x + (w.x == x0 ? 0 : 1)) * kChunkRows + x * 128 + r;
            char* const mine = whole ? reinterpret_cast<char*>(a.o + (size_t)(w.row + w.tok0 + x * a.tt + rt) * a.H * HD + (size_t)(w.g * a.Hg + r % a.Hg) * HD)
                                     : reinterpret_cast<char*>(a.part.o + at * HD);
            const unsigned lives = __ballot_sync(0xffffffffu, live);
            // (little code: it runs once a piece, from a cold instruction cache)
#pragma unroll 1
            for (int t = 0; t < HD / 32; ++t) {  // 32 columns: a line of the workspace, half a line of o
                float o[32];
                tmem_ld32(tO + 32 * t, o);
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        pass[lane * 8 + ((4 * (t & 1) + i) ^ (lane & 7))] =
                            make_uint4(pack2(o[8 * i] * inv, o[8 * i + 1] * inv), pack2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                       pack2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                    if (!(t & 1)) continue;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(&pass[lane * 8 + (i ^ (lane & 7))]) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
                __syncwarp();
                const int off = 128 * (whole ? t >> 1 : t) + 16 * (lane & 7);
#pragma unroll 2
                for (int i = 0; i < 8; ++i) {
                    const int row = 4 * i + (lane >> 3);
                    char* to = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), row));
                    if (lives >> row & 1) *reinterpret_cast<uint4*>(to + off) = pass[row * 8 + ((lane & 7) ^ (row & 7))];
                }
                __syncwarp();
            }
            if (!whole && live) a.part.ml[at] = make_float2(m, l);
            tc_fence_before();
            // the next piece's first product overwrites O: it waits for this half's P, handed over after these reads
        }
        if (threadIdx.x == 0) a.part.desc[blockIdx.x] = *abort_flag ? make_int4(0, 0, 0, 0) : d;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- joining the pieces
// How one attention kernel's partial results lie (see Partials): its rows per piece, in halves of
// `half` rows and `tokens` tokens, and how many blocks along y join them.
struct JoinSet {
    Partials part;
    int rows, half, tokens, blocks;
};

// Rows of the output that begins in block c of the attention's grid and goes on in the next
// ones, one row after another: WPR warps to a row, each with every WPR-th piece.
template <int HD, int WPR>
__device__ __forceinline__ void join_rows(const JoinSet& s, int y, int H, int Hg, bf16* __restrict__ o, float (*s_o)[HD],
                                          float2* s_ml) {
    constexpr int E = HD / 32, RPB = 8 / WPR;
    const int4 d = s.part.desc[blockIdx.x];
    const int n = d.z >> 1;
    if (n == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i0 = y * RPB; i0 < s.rows; i0 += s.blocks * RPB) {
        const int i = i0 + warp / WPR, in = i % s.half, tok = (i / s.half) * s.tokens + in / Hg;
        const bool live = in < s.tokens * Hg && tok < d.w;
        float acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        auto add = [&](float om, float ol, const float* v) {
            const float M = fmaxf(m, om);
            const float c0 = m == -INFINITY ? 0.f : ex2(m - M), c1 = om == -INFINITY ? 0.f : ex2(om - M);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = acc[e] * c0 + v[e] * c1;
            l = l * c0 + ol * c1;
            m = M;
        };
        if (live) {
#pragma unroll 2
            for (int k = warp % WPR; k < n; k += WPR) {
                const size_t at = (size_t)(2 * (blockIdx.x + k) + (k == 0 ? d.z & 1 : 0)) * s.rows + i;
                const float2 ml = s.part.ml[at];
                float v[E];
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 t = *reinterpret_cast<const float2*>(s.part.o + at * HD + lane * E + e);
                    v[e] = t.x; v[e + 1] = t.y;
                }
                add(ml.x, ml.y, v);
            }
        }
        if (WPR > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
            if (lane == 0) s_ml[warp] = make_float2(m, l);
            __syncthreads();
            if (warp % WPR != 0) continue;
#pragma unroll
            for (int k = 1; k < WPR; ++k) add(s_ml[warp + k].x, s_ml[warp + k].y, &s_o[warp + k][lane * E]);
        }
        if (!live) continue;
        const float inv = 1.f / l;
        bf16* to = o + (size_t)(d.x + tok) * H * HD + (size_t)(d.y * Hg + in % Hg) * HD + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(to + e) = pack2(acc[e] * inv, acc[e + 1] * inv);
    }
}

// Both attention kernels' pieces: blocks y < dec.blocks the decoding requests' (few rows, up to as
// many pieces as there are SMs), the others the chunks' (up to 256 rows, seldom more than three pieces).
template <int HD>
__global__ void __launch_bounds__(256) paged_join_kernel(const JoinSet dec, const JoinSet chunk, int H, int Hg, bf16* __restrict__ o) {
    __shared__ float s_o[8][HD];
    __shared__ float2 s_ml[8];
    pdl_wait();
    if ((int)blockIdx.y < dec.blocks) join_rows<HD, 4>(dec, blockIdx.y, H, Hg, o, s_o, s_ml);
    else join_rows<HD, 1>(chunk, blockIdx.y - dec.blocks, H, Hg, o, s_o, s_ml);
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

bool tensor_core_takes(DType at, int H, int nkv, int hd) { return at == DT_BF16 && (hd == 64 || hd == 128) && H / nkv <= 128; }

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
cudaError_t attention(const bf16* qkv, int H, int nkv, int rows, int max_new, const int32_t* slots, const PagedKv& kv, bf16* o,
                      char* ws, int* status, cudaStream_t s) {
    const int Hg = H / nkv, G = device_sm_count();
    const float scale_log2 = kLog2eF / sqrtf((float)HD);
    const bool decodes = Hg <= kDecRows, chunks = !decodes || max_new != 1;
    const bool whole = (long long)kv.max_blocks * kv.page <= (chunks ? kWholePositions : kWholeDecoding);
    static_assert(kWholePositions <= 128 * kWholeTiles, "the chunk kernel cuts nothing either");
    JoinSet jd{}, jc{};
    cudaError_t e;
    if (decodes) {
        if ((e = ensure_smem_limit((const void*)paged_decode_kernel<HD>, DecLayout<HD>::bytes(kMaxRequests))) != cudaSuccess) return e;
        jd = {partials(ws, G, kDecRows, HD), kDecRows, kDecRows, 1, (Hg + 1) / 2};
        ws += partial_bytes(G, kDecRows, HD);
        DecodeArgs a{qkv, slots, kv, o, jd.part, H, nkv, Hg, rows, std::min(kv.page, kTile), max_new, whole, scale_log2, status};
        CUtensorMap tk, tv;
        if (!map_pool(&tk, kv.k, nkv, HD, kv, a.piece) || !map_pool(&tv, kv.v, nkv, HD, kv, a.piece)) return cudaErrorUnknown;
        paged_decode_kernel<HD><<<G, kDecThreads, DecLayout<HD>::bytes(kv.n_req), s>>>(tk, tv, a);
        count_launch();
        e = cudaGetLastError();
    } else {
        e = launch_paged_append(qkv, H, nkv, HD, rows, slots, kv, status, s);
    }
    if (e != cudaSuccess) return e;
    if (chunks) {
        if ((e = ensure_smem_limit((const void*)paged_chunk_kernel<HD>, ChunkLayout<HD>::bytes(kMaxRequests))) != cudaSuccess) return e;
        const int tt = 128 / Hg;
        jc = {partials(ws, G, kChunkRows, HD), kChunkRows, 128, tt, 32};
        ChunkArgs a{kv, o, jc.part, H, nkv, Hg, tt, rows, std::min(kv.page, 128), max_new, decodes, scale_log2, status};
        CUtensorMap tq, tk, tv;
        const cuuint64_t ld = (cuuint64_t)(H + 2 * nkv) * HD * 2;
        const cuuint64_t dq[3] = {HD, (cuuint64_t)(H + 2 * nkv), (cuuint64_t)rows}, sq[2] = {HD * 2, ld};
        const cuuint32_t bq[3] = {64, (cuuint32_t)Hg, (cuuint32_t)tt};
        const cuuint64_t dk[2] = {(cuuint64_t)nkv * HD, (cuuint64_t)kv.n_pages * kv.page}, sk[1] = {(cuuint64_t)nkv * HD * 2};
        const cuuint32_t bk[2] = {64, (cuuint32_t)a.piece};
        if (!encode(&tq, qkv, 3, dq, sq, bq) || !encode(&tk, kv.k, 2, dk, sk, bk) || !encode(&tv, kv.v, 2, dk, sk, bk))
            return cudaErrorUnknown;
        void* args[] = {&tq, &tk, &tv, &a};
        e = launch_pdl((const void*)paged_chunk_kernel<HD>, dim3(G), kChunkThreads, ChunkLayout<HD>::bytes(kv.n_req), s, args);
        if (e != cudaSuccess) return e;
    }
    if (whole) return cudaSuccess;
    void* args[] = {&jd, &jc, &H, const_cast<int*>(&Hg), &o};
    return launch_pdl((const void*)paged_join_kernel<HD>, dim3(G, jd.blocks + jc.blocks), 256, 0, s, args);
}

}  // namespace

size_t paged_attention_workspace(DType at, int H, int nkv, int hd) {
    if (!tensor_core_takes(at, H, nkv, hd)) return 256;
    const int G = device_sm_count();
    return partial_bytes(G, kDecRows, hd) + partial_bytes(G, kChunkRows, hd);
}

cudaError_t paged_attention(DType at, const void* qkv, int H, int nkv, int hd, int rows, int max_new,
                            const int32_t* slots, const PagedKv& kv, void* o, void* workspace, int* status,
                            cudaStream_t s) {
    if (tensor_core_takes(at, H, nkv, hd)) {
        auto f = hd == 128 ? attention<128> : attention<64>;
        return f(reinterpret_cast<const bf16*>(qkv), H, nkv, rows, max_new, slots, kv, reinterpret_cast<bf16*>(o), (char*)workspace,
                 status, s);
    }
    return launch_paged_attention_simt(at, qkv, H, nkv, hd, rows, slots, kv, o, status, s);
}

}  // namespace nc
