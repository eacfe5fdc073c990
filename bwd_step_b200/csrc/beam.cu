// Beam search's selection over beams and vocabulary.
//
// A candidate (beam k, id v) has the score s_k + z_kv - lse_k, lse_k the
// log-sum-exp of beam k's logits; a finished beam has one candidate, its end
// again at its score.  The K best of a batch row's candidates are wanted, so at
// most the K best logits of each beam matter.
//
// One cluster of blocks per batch row, every block a slice of the vocabulary, every
// warp a part of it; nothing meets while the logits stream through shared memory:
//   1. bulk copies bring 16 KB chunks of one beam after another, and every thread
//      keeps its values' maximum and, against its warp's maximum, the sum of their
//      exponentials;
//   2. the slices' maxima of every beam and lane meet through distributed shared memory:
//      each lane's best score over beams, slices and warps is some candidate's, so the
//      K-th largest of the 32 bounds the K-th best score from below;
//   3. only the threads whose maximum reaches that bound, some K of all, read their
//      values again (from L2) and hand the first block the candidates that reach it;
//   4. the first block ranks those by counting the better ones.
// The sums are kept in 32 bits.  A term e^d is off by 2.3 |d| 2^-24 of itself (the difference, the factor and
// the product rounded; the mean of |d| over the terms by their weight is at most ln V) and by 2^-22
// (ex2.approx), each change of the maximum on its way by 5 2^-24, each sum by 2^-24: some 60 2^-24 in
// all for 65536 ids, so the log-sum-exp is within 2^-18 whatever the size of the logits.  Measured over
// normal logits of deviations 0.01 to 1000, 4160 to 262400 ids: 1.2 2^-24 root mean square, 4.4 2^-24 at most.
// One launch, no workspace.  64 x 8 beams of 65536 ids (62 MB) take 28 us (25.8 in a graph): the
// stream 11.5, bound by HBM, and what follows it by the latency of its steps; 1 x 4 beams 12 us (9.6).
// The slow way that many equal or masked candidates take (more than 256 that reach the bound, as where
// 40 ids are left of 65536) is K passes: 64 x 8 beams 1.0 ms, a vocabulary masked throughout 1.1 ms.
#include "paged.h"
#include "tc_common.cuh"

#include <cooperative_groups.h>
#include <algorithm>

namespace nc {
namespace {
namespace cg = cooperative_groups;

constexpr int kWarps = 8, kThreads = 32 * kWarps;  // and one warp more that copies
constexpr int kChunk = 16384;  // bytes of a beam's logits brought at once
constexpr int kStages = 2;     // chunks on their way: at four blocks an SM, 128 KB
constexpr int kCand = 256;     // gathered candidates; more (many alike) take the slow way
// Blocks of a cluster, at most.  1x4 beams of 65536 ids: 12.4 us with 4, 9.2 with 8, 9.4 with 16;
// 64x8 beams: 24.9, 24.6, 51 us.  Smaller vocabularies take fewer (see launch_beam_select).
constexpr int kCluster = 8;
constexpr float kLog2e = 1.44269504088896340736f;
typedef unsigned long long u64;

// Floats in the order of unsigned integers, NaN as -inf and -0 as +0; 0 is below all of them.
__device__ __forceinline__ uint32_t ordered(float z) {
    const uint32_t b = __float_as_uint(fmaxf(z, -INFINITY) + 0.f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) { return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu)); }
// A key orders candidates of one beam: by logit, then the lower id first.  0 stands for none.
__device__ __forceinline__ u64 make_key(uint32_t z, uint32_t id) { return (u64)z << 32 | (uint32_t)~id; }
__device__ __forceinline__ float key_logit(u64 key) { return unordered((uint32_t)(key >> 32)); }
__device__ __forceinline__ uint32_t key_id(u64 key) { return ~(uint32_t)key; }

// The K-th largest of the lanes' values (bitonic sort over the warp).
__device__ __forceinline__ uint32_t lane_kth(uint32_t v, int k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, v, d);
            const bool high = ((lane & d) == 0) == ((lane & size) == 0);  // descending runs
            v = high ? max(v, o) : min(v, o);
        }
    return __shfl_sync(0xffffffffu, v, k - 1);
}

// Maximum of a 16-byte vector's values, NaN passed over.
__device__ __forceinline__ float vec_max(const uint4& u, bf16) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
}
__device__ __forceinline__ float vec_max(const uint4& u, float) {
    return fmaxf(fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w))), -INFINITY);
}

struct SelectArgs {
    int batch, beams, V, eos, slice;  // slice: ids of a block
    const float* scores;
    const int32_t* finished;
    float* scores_out;
    int32_t* tokens;
    int32_t* parents;
    int32_t* finished_out;
    int* status;
};

// A candidate as the ranking sees it: score, ordered (0: none), beam, key.
struct Candidate {
    u64 score, key;
    int beam;
};
__device__ __forceinline__ bool better(u64 s, int b, u64 k, u64 s2, int b2, u64 k2) {
    return s > s2 || (s == s2 && (b < b2 || (b == b2 && k > k2)));
}

struct Shared {
    uint8_t stage[kStages][kChunk];
    u64 score[kCand], key[kCand];  // the first block's: the gathered candidates
    int beam[kCand];
    int count, pushed;        // candidates gathered; those that this block gave
    int pushes[kCluster];     // what every block gave
    float sum[kMaxBeams], mx[kMaxBeams];       // this slice's maximum, and sum of exp(z - mx)
    double lse[kMaxBeams];
    uint32_t least[kMaxBeams];
    float part[kMaxBeams][kWarps], top[kMaxBeams][kWarps];
    uint32_t warp_best[kWarps + 1][32];
    uint32_t lane_max[kMaxBeams][32];
    float s0[kMaxBeams];
    int finished[kMaxBeams];
    int active[kMaxBeams];
    int n_active;
    int abort_flag;
    Candidate best[2], warp_cand[kWarps + 1];
    uint64_t full[kStages], empty[kStages];
    uint32_t tmax[1];              // [K][kThreads]: thread maxima, ordered; 0 where a thread has no value
};
inline size_t shared_bytes(int K) { return sizeof(Shared) + (size_t)K * kThreads * 4; }

__device__ __forceinline__ u64 ordered(double x) {
    const u64 u = (u64)__double_as_longlong(x + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered(u64 o) { return __longlong_as_double((long long)(o ^ ((o >> 63) ? 1ull << 63 : ~0ull))); }

template <typename A>
__global__ void __launch_bounds__(kThreads + 32, 4) beam_select_kernel(const A* __restrict__ logits, const SelectArgs a) {
    constexpr int VEC = Vec<A>::N, NV = kChunk / 16 / kThreads, EL = kChunk / (int)sizeof(A);  // a thread's vectors, a chunk's ids
    extern __shared__ __align__(128) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), S = (int)cluster.num_blocks(), K = a.beams;
    const int b = blockIdx.x / S, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lo = min(a.V, rank * a.slice), hi = min(a.V, lo + a.slice);
    const int nch = (hi - lo + EL - 1) / EL;
    const A* row = logits + (size_t)b * K * a.V;
    uint32_t* tmax = sh.tmax;
    volatile int* abort_flag = &sh.abort_flag;
    if (warp == 0) {
        const bool fin = lane < K && a.finished && a.finished[b * K + lane] != 0;
        const unsigned m = __ballot_sync(0xffffffffu, lane < K && !fin);
        if (lane < K && !fin) sh.active[__popc(m & ((1u << lane) - 1))] = lane;
        sh.finished[lane] = fin;
        sh.s0[lane] = lane < K ? a.scores[b * K + lane] : 0.f;
        sh.mx[lane] = -INFINITY;
        sh.sum[lane] = 0.f;
        if (lane < kStages) {
            tc::mbar_init(tc::smem_u32(&sh.full[lane]), 1);
            tc::mbar_init(tc::smem_u32(&sh.empty[lane]), kWarps);
        }
        if (lane == 0) {
            sh.n_active = __popc(m);
            sh.abort_flag = 0;
            sh.count = sh.pushed = 0;
            tc::fence_barrier_init();
        }
    }
    __syncthreads();
    const int n_active = hi > lo ? sh.n_active : 0, T = n_active * nch;
    // ---------------- 1: the stream
    if (warp == kWarps) {
        int ak = 0, ch = 0, t = 0;
        for (; t < T; ++t) {
            const int st = t % kStages, c0 = lo + ch * EL;
            if (!tc::warp_wait(tc::smem_u32(&sh.empty[st]), ((t / kStages) & 1) ^ 1, abort_flag, a.status)) break;
            if (lane == 0) {
                const uint32_t bytes = (uint32_t)min(EL, hi - c0) * sizeof(A), bar = tc::smem_u32(&sh.full[st]);
                tc::mbar_expect_tx(bar, bytes);
                tc::bulk_load(tc::smem_u32(sh.stage[st]), row + (size_t)sh.active[ak] * a.V + c0, bytes, bar);
            }
            if (++ch == nch) { ch = 0; ++ak; }
        }
        if (t < T && lane == 0)  // copies in flight land before the memory is used again (1 ms each at most)
            for (int d = max(0, t - kStages); d < t; ++d) {
                const uint64_t t0 = tc::globaltimer();
                while (tc::globaltimer() - t0 < 1000000ull && !tc::mbar_test(tc::smem_u32(&sh.full[d % kStages]), (d / kStages) & 1)) {}
            }
    } else {
        bool ok = true;
        for (int ak = 0, t = 0; ok && ak < n_active; ++ak) {
            const int k = sh.active[ak];
            float own = -INFINITY, top = -INFINITY, sum = 0.f;  // top, sum: of the warp's maximum so far, of this lane
            for (int ch = 0; ch < nch; ++ch, ++t) {
                const int st = t % kStages, n = min(EL, hi - lo - ch * EL);
                ok = tc::warp_wait(tc::smem_u32(&sh.full[st]), (t / kStages) & 1, abort_flag, a.status);
                if (!ok) break;
                const uint4* z = reinterpret_cast<const uint4*>(sh.stage[st]) + tid;
                uint4 raw[NV];
#pragma unroll
                for (int q = 0; q < NV; ++q) raw[q] = z[q * kThreads];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.empty[st]));
#pragma unroll
                for (int q = 0; q < NV; ++q)  // n is a multiple of a vector: it is in or out
                    if ((q * kThreads + tid) * VEC < n) own = fmaxf(own, vec_max(raw[q], A{}));
                const float up = unordered(__reduce_max_sync(0xffffffffu, ordered(own)));
                if (up > top) {
                    sum *= tc::ex2((top - up) * kLog2e);  // top = -inf: 0
                    top = up;
                }
                if (top == -INFINITY) continue;
                // The difference before the factor: it is exact near the maximum, where -top * log2 e, rounded beside
                // fma(z, log2 e, .), would leave |top| 2^-24 in the sum (and infinities at the type's largest values).
                const uint64_t l2 = tc::f2_pack(kLog2e, kLog2e), less = tc::f2_pack(-top, -top);
                uint64_t s2[2] = {tc::f2_pack(0.f, 0.f), tc::f2_pack(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    float v[VEC];
                    load_vec(reinterpret_cast<const A*>(&raw[q]), v);
                    if ((q * kThreads + tid) * VEC < n)
#pragma unroll
                        for (int e = 0; e < VEC; e += 2) {
                            float x0, x1;
                            tc::f2_unpack(tc::f2_mul(tc::f2_add(tc::f2_pack(v[e], v[e + 1]), less), l2), x0, x1);
                            s2[(e >> 1) & 1] = tc::f2_add(s2[(e >> 1) & 1], tc::f2_pack(tc::ex2(x0), tc::ex2(x1)));
                        }
                }
                float x0, x1, x2, x3;
                tc::f2_unpack(s2[0], x0, x1);
                tc::f2_unpack(s2[1], x2, x3);
                float add = (x0 + x1) + (x2 + x3);
                if (add != add && top < INFINITY) {  // NaN counts as -inf: without them
                    add = 0.f;
#pragma unroll
                    for (int q = 0; q < NV; ++q) {
                        float v[VEC];
                        load_vec(reinterpret_cast<const A*>(&raw[q]), v);
                        if ((q * kThreads + tid) * VEC < n)
#pragma unroll
                            for (int e = 0; e < VEC; ++e) add += tc::ex2((fmaxf(v[e], -INFINITY) - top) * kLog2e);
                    }
                }
                sum += add;
            }
            tmax[k * kThreads + tid] = ordered(own);
            sum = warp_sum(sum);
            if (lane == 0) { sh.part[k][warp] = sum; sh.top[k][warp] = top; }
        }
    }
    __syncthreads();
    // ---------------- 2: the slice's maxima and sums, then the bound from all slices'
    for (int k = warp; k < K; k += kWarps + 1) {
        uint32_t m = 0;
        if (!sh.finished[k] && hi > lo) {
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                uint32_t v = tmax[k * kThreads + 32 * i + lane];
                if ((32 * i + lane) * VEC >= hi - lo) tmax[k * kThreads + 32 * i + lane] = v = 0;  // it had no value
                m = max(m, v);
            }
            const float pt = lane < kWarps ? sh.top[k][lane] : -INFINITY;
            const float top = unordered(__reduce_max_sync(0xffffffffu, ordered(pt)));
            const float s = warp_sum(pt > -INFINITY ? sh.part[k][lane] * tc::ex2((pt - top) * kLog2e) : 0.f);
            if (lane == 0) { sh.mx[k] = top; sh.sum[k] = s; }
        }
        sh.lane_max[k][lane] = m;
    }
    cluster.sync();
    auto score_of = [&](int k, float z) -> double {
        const double v = (double)sh.s0[k] + ((double)z - sh.lse[k]);
        return v != v ? -INFINITY : v;
    };
    uint32_t best = 0;  // the lane's best score, rounded down to 32 bits and ordered
    for (int k = warp; k < K; k += kWarps + 1) {
        if (sh.finished[k]) {
            const float v = sh.s0[k];
            if (lane == k) best = max(best, ordered(v));
            continue;
        }
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < kCluster; ++s)
            if (s < S) m = max(m, cluster.map_shared_rank(&sh, s)->lane_max[k][lane]);
        const Shared* o = cluster.map_shared_rank(&sh, lane < S ? lane : 0);
        const float mx = lane < S ? o->mx[k] : -INFINITY;
        const float p = lane < S ? o->sum[k] : 0.f;
        const float top = unordered(__reduce_max_sync(0xffffffffu, ordered(mx)));
        double sum = mx > -INFINITY ? (double)(p * tc::ex2((mx - top) * kLog2e)) : 0.0;
#pragma unroll
        for (int d = kCluster / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        // no candidate of weight (or +inf among them): every score is -inf
        if (lane == 0) sh.lse[k] = top > -INFINITY && top < INFINITY ? (double)top + log(sum) : (double)INFINITY;
        __syncwarp();
        if (m) best = max(best, ordered(__double2float_rd(score_of(k, unordered(m)))));
    }
    sh.warp_best[warp][lane] = best;
    __syncthreads();
#pragma unroll
    for (int i = 0; i <= kWarps; ++i) best = max(best, sh.warp_best[i][lane]);
    // where fewer than K lanes have a finite score, finite candidates are tried for
    const double bound = (double)unordered(max(lane_kth(best, K, lane), ordered(-INFINITY) + 1));
    // ---------------- 3: the candidates that reach the bound, to the first block
    Shared* first = cluster.map_shared_rank(&sh, 0);
    if (tid < K) {
        // the least logit of beam tid that may reach the bound: the difference in 64 bits, and a margin for its
        // rounding and the score's (both far below 2^-40 of the larger part)
        const double d = (double)sh.s0[tid] - sh.lse[tid], least = bound - d;
        const double margin = (fabs(bound) + fabs(d)) * 0x1p-40;
        sh.least[tid] = least == least && margin < INFINITY ? max(1u, ordered(__double2float_rd(least - margin))) : 1u;
    }
    __syncthreads();
    auto push = [&](double v, u64 key, int k) {
        atomicAdd(&sh.pushed, 1);
        const int to = atomicAdd(&first->count, 1);
        if (to < kCand) { first->score[to] = ordered(v); first->key[to] = key; first->beam[to] = k; }
    };
    // calls f(key, score) for this thread's values of beam k
    auto values = [&](int k, auto f) {
        const A* z = row + (size_t)k * a.V;
        for (int ch = 0; ch < nch; ++ch) {
            const int c0 = lo + ch * EL;
            uint4 raw[NV];
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int id = c0 + (q * kThreads + tid) * VEC;
                if (id < hi) raw[q] = *reinterpret_cast<const uint4*>(z + id);
            }
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int id = c0 + (q * kThreads + tid) * VEC;
                if (id >= hi) continue;
                float v[VEC];
                load_vec(reinterpret_cast<const A*>(&raw[q]), v);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const uint32_t o = ordered(v[e]);
                    f(make_key(o, id + e), score_of(k, unordered(o)));
                }
            }
        }
    };
    if (warp < kWarps && hi > lo) {
        // Only a few threads' values are looked at; the warp reads a thread's together, a value to a lane.
        const int in_chunk = (lane / VEC * kThreads + 32 * warp) * VEC + lane % VEC;
        for (int k = 0; k < K; ++k) {
            const uint32_t least = sh.least[k];
            unsigned m = __ballot_sync(0xffffffffu, !sh.finished[k] && tmax[k * kThreads + tid] >= least);
            for (; m; m &= m - 1) {
                const A* z = row + (size_t)k * a.V;
                for (int ch = 0; ch < nch; ++ch) {
                    const int id = lo + ch * EL + in_chunk + (__ffs(m) - 1) * VEC;
                    if (lane >= NV * VEC || id >= hi) continue;
                    const uint32_t o = ordered(tof(z[id]));
                    if (o < least) continue;
                    const double sc = score_of(k, unordered(o));
                    if (sc >= bound) push(sc, make_key(o, id), k);
                }
            }
        }
    }
    if (rank == 0 && tid < K && sh.finished[tid] && (double)sh.s0[tid] >= bound) push((double)sh.s0[tid], make_key(1u, a.eos), tid);
    __syncthreads();
    if (tid < S) cluster.map_shared_rank(&sh, tid)->pushes[rank] = sh.pushed;
    cluster.sync();
    // ---------------- 4: the candidates in their order
    auto put = [&](int i, u64 score, u64 key, int beam) {
        const int to = b * K + i, token = (int)key_id(key);
        a.scores_out[to] = (float)unordered(score);
        a.tokens[to] = token;
        a.parents[to] = beam;
        if (a.finished_out) a.finished_out[to] = sh.finished[beam] || token == a.eos;
    };
    int c = 0;
    for (int s = 0; s < S; ++s) c += sh.pushes[s];
    if (c >= K && c <= kCand) {  // no block reads another's memory from here on
        if (rank == 0)
            for (int i = warp; i < c; i += kWarps + 1) {  // a warp to a candidate, the better ones counted by the lanes
                const u64 sc = sh.score[i], ke = sh.key[i];
                const int be = sh.beam[i];
                int above = 0;
                for (int o = lane; o - lane < c; o += 32)
                    above += __popc(__ballot_sync(0xffffffffu, o < c && better(sh.score[o], sh.beam[o], sh.key[o], sc, be, ke)));
                if (lane == 0 && above < K) put(above, sc, ke, be);
            }
    } else {
        // Too many alike, or too few of finite score: K times the best candidate behind the last one, each
        // block's threads over their own values, the blocks' bests through distributed shared memory.
        u64 last_s = ~0ull, last_k = ~0ull;
        int last_b = -1;
        for (int i = 0; i < K; ++i) {
            u64 bs = 0, bk = 0;
            int bb = kMaxBeams;
            auto offer = [&](u64 s, u64 ke, int k) {
                if (better(last_s, last_b, last_k, s, k, ke) && better(s, k, ke, bs, bb, bk)) { bs = s; bk = ke; bb = k; }
            };
            for (int k = 0; k < K; ++k) {
                if (sh.finished[k]) {
                    if (rank == 0 && tid == k) offer(ordered(sh.s0[k] != sh.s0[k] ? -INFINITY : (double)sh.s0[k]), make_key(1u, a.eos), k);
                } else if (warp < kWarps && hi > lo) {
                    const uint32_t m = tmax[k * kThreads + tid];
                    // a thread whose best value is no better than what it holds has nothing to offer
                    if (m && ordered(score_of(k, unordered(m))) >= bs)
                        values(k, [&](u64 key, double sc) { offer(ordered(sc), key, k); });
                }
            }
            auto take = [&](u64 s, u64 ke, int k) {
                if (better(s, k, ke, bs, bb, bk)) { bs = s; bk = ke; bb = k; }
            };
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                take(__shfl_xor_sync(0xffffffffu, bs, d), __shfl_xor_sync(0xffffffffu, bk, d), __shfl_xor_sync(0xffffffffu, bb, d));
            if (lane == 0) sh.warp_cand[warp] = {bs, bk, bb};
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w <= kWarps; ++w) take(sh.warp_cand[w].score, sh.warp_cand[w].key, sh.warp_cand[w].beam);
                sh.best[i & 1] = {bs, bk, bb};  // read until the next round's barrier, written again after it
            }
            cluster.sync();
            bs = bk = 0;
            bb = kMaxBeams;
            for (int s = 0; s < S; ++s) {
                const Candidate& o = cluster.map_shared_rank(&sh, s)->best[i & 1];
                take(o.score, o.key, o.beam);
            }
            if (rank == 0 && tid == 0) put(i, bs, bk, bb);
            last_s = bs; last_k = bk; last_b = bb;
        }
        cluster.sync();  // every block's shared memory has been read
    }
}

template <typename A>
cudaError_t select_t(const void* logits, const SelectArgs& a, int cluster, cudaStream_t s) {
    cudaError_t e = ensure_smem_limit((const void*)beam_select_kernel<A>, (int)shared_bytes(kMaxBeams));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.batch * cluster));
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = shared_bytes(a.beams);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, beam_select_kernel<A>, reinterpret_cast<const A*>(logits), a);
    if (e != cudaSuccess) return e;
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(DType at, const void* logits, int batch, int beams, int V, const float* scores,
                               const int32_t* finished, int eos, float* scores_out, int32_t* tokens, int32_t* parents,
                               int32_t* finished_out, int* status, cudaStream_t s) {
    SelectArgs a{};
    a.batch = batch; a.beams = beams; a.V = V; a.eos = eos;
    a.scores = scores; a.finished = finished;
    a.scores_out = scores_out; a.tokens = tokens; a.parents = parents; a.finished_out = finished_out;
    a.status = status;
    // A small vocabulary gains nothing by more blocks, and many rows pay for each.  Graph times, us, with 1, 2, 4, 8 blocks:
    // 1 x 4 beams of 1024 ids 8.6, 8.9, 8.9, 9.0, of 4096 9.2, 8.9, 8.6, 8.8, of 16384 12.5, 9.8, 9.1, 9.0; 64 x 8 beams of 1024
    // ids 14.1, 14.7, 15.6, 18.9, of 4096 14.6, 13.8, 14.4, 18.5, of 16384 21.4, 15.3, 15.9, 20.2 (few rows decide from 8192 on).
    const int cluster = V >= 8192 ? kCluster : V >= 4096 ? 4 : V >= 2048 ? 2 : 1;
    a.slice = ((V + cluster - 1) / cluster + 7) & ~7;
    return at == DT_BF16 ? select_t<bf16>(logits, a, cluster, s) : select_t<float>(logits, a, cluster, s);
}

}  // namespace nc
