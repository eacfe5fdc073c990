// Beam search's selection over beams and vocabulary.
//
// A candidate (beam k, id v) has the score s_k + z_kv - lse_k, lse_k the
// log-sum-exp of beam k's logits; a finished beam has one candidate, its end
// again at its score.  The K best of a batch row's candidates are wanted, so at
// most the K best logits of each beam matter: one pass over the logits keeps,
// per beam, a running maximum and sum of exponentials and a sorted list of the
// best (logit, id) keys, and the lists of K beams are merged by score.
//
// One cluster of blocks per batch row, every block a slice of the vocabulary,
// every warp a part of a beam's slice; lists and sums meet in the first block
// through distributed shared memory, so there is one launch and no workspace.
// Bound by reading the logits once.
#include "paged.h"
#include "common.cuh"

#include <cooperative_groups.h>
#include <algorithm>

namespace nc {
namespace {
namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTasks = 32;  // (beam, part of its slice) lists of a block
constexpr float kLog2e = 1.44269504088896340736f;
typedef unsigned long long u64;

// A key orders candidates of one beam: by logit, then the lower id first.
// NaN counts as -inf, and -0 as +0.  0 stands for none.
__device__ __forceinline__ float clean(float z) { return z != z ? -INFINITY : z + 0.f; }
__device__ __forceinline__ u64 make_key(float z, uint32_t id) {
    const uint32_t b = __float_as_uint(z);
    return (u64)(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float key_logit(u64 key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t key_id(u64 key) { return ~(uint32_t)key; }

// A warp's sorted list: lane i holds the i-th best key, `last` the K-th.
struct List {
    u64 key = 0, last = 0;
    int k;
    __device__ __forceinline__ void insert(u64 c, int lane) {  // c is the same in every lane
        const int at = __popc(__ballot_sync(0xffffffffu, key > c));
        const u64 up = __shfl_up_sync(0xffffffffu, key, 1);
        if (lane == at) key = c;
        else if (lane > at) key = up;
        last = __shfl_sync(0xffffffffu, key, k - 1);
    }
    // every lane offers one key (0: none)
    __device__ __forceinline__ void offer(u64 c, int lane) {
        unsigned m = __ballot_sync(0xffffffffu, c > last);
        while (m) {
            insert(__shfl_sync(0xffffffffu, c, __ffs(m) - 1), lane);
            m &= m - 1;
            m &= __ballot_sync(0xffffffffu, c > last);
        }
    }
};

__device__ __forceinline__ float exp2a(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The K-th largest of the lanes' values (bitonic sort over the warp).
__device__ __forceinline__ float lane_kth(float v, int k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, v, d);
            const bool high = ((lane & d) == 0) == ((lane & size) == 0);  // descending runs
            v = high ? fmaxf(v, o) : fminf(v, o);
        }
    return __shfl_sync(0xffffffffu, v, k - 1);
}

struct SelectArgs {
    int batch, beams, V, eos, cluster, slice, parts;  // ids of a block's slice, parts of a slice per beam
    const float* scores;
    const int32_t* finished;
    float* scores_out;
    int32_t* tokens;
    int32_t* parents;
    int32_t* finished_out;
};

struct Shared {
    u64 task_key[kMaxTasks][32];
    float task_max[kMaxTasks];
    float task_sum[kMaxTasks];
    u64 key[kMaxBeams][32];  // per beam: the block's best keys
    float mx[kMaxBeams];
    double sum[kMaxBeams];
    double lse[kMaxBeams];
};

// One warp over ids [lo, hi) of a beam's logits.  lo is a multiple of a 16-byte
// vector and the row starts on a 16-byte boundary.
template <typename A>
__device__ __forceinline__ void scan_logits(const A* __restrict__ z, int lo, int hi, int lane, List& list, float& mx,
                                            float& sum) {
    constexpr int VEC = Vec<A>::N, NV = 4, STEP = 32 * VEC;  // NV vectors of a lane in flight
    mx = -INFINITY;
    sum = 0.f;
    uint4 next[NV];
    auto fetch = [&](int at) {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = at + q * STEP + lane * VEC;
            if (i < hi) next[q] = __ldcs(reinterpret_cast<const uint4*>(z + i));
        }
    };
    fetch(lo);
    float floor_v = -INFINITY;
    bool first = true;
    for (int at = lo; at < hi; at += NV * STEP) {
        float v[NV][VEC];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = at + q * STEP + lane * VEC;  // hi - lo is a multiple of VEC: a vector is in or out
            float w[VEC];
            load_vec(reinterpret_cast<const A*>(&next[q]), w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[q][e] = i < hi ? clean(w[e]) : -INFINITY;
        }
        if (at + NV * STEP < hi) fetch(at + NV * STEP);
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int e = 0; e < VEC; ++e) top = fmaxf(top, v[q][e]);
        if (top > mx) {
            sum *= exp2a((mx - top) * kLog2e);  // mx = -inf: 0
            mx = top;
        }
        if (mx > -INFINITY) {
            const float sh = -mx * kLog2e;
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s4[e & 3] += exp2a(fmaf(v[q][e], kLog2e, sh));
            sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        }
        // at least K of the first values are no less than the K-th largest of the lanes' maxima
        if (first) {
            floor_v = lane_kth(top, list.k, lane);
            first = false;
        }
        if (!__any_sync(0xffffffffu, top >= floor_v)) continue;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = at + q * STEP + lane * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (__any_sync(0xffffffffu, v[q][e] >= floor_v))
                    list.offer(v[q][e] >= floor_v && i < hi ? make_key(v[q][e], i + e) : 0, lane);
        }
        if (list.last) floor_v = fmaxf(floor_v, key_logit(list.last));
    }
}

template <typename A>
__global__ void __launch_bounds__(kThreads) beam_select_kernel(const A* __restrict__ logits, const SelectArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), C = a.cluster, K = a.beams;
    const int b = blockIdx.x / C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto finished = [&](int k) { return a.finished && a.finished[b * K + k] != 0; };
    const int lo = min(a.V, rank * a.slice), hi = min(a.V, lo + a.slice);
    const int step = ((hi - lo + a.parts - 1) / a.parts + 7) & ~7;
    for (int t = warp; t < K * a.parts; t += kWarps) {
        const int k = t / a.parts, l0 = min(hi, lo + (t % a.parts) * step), l1 = min(hi, l0 + step);
        List list;
        list.k = K;
        float mx = -INFINITY, sum = 0.f;
        if (!finished(k) && l0 < l1) scan_logits(logits + (size_t)(b * K + k) * a.V, l0, l1, lane, list, mx, sum);
        sh.task_key[t][lane] = lane < K ? list.key : 0;
        const float top = warp_max(mx);
        sum = warp_sum(mx > -INFINITY ? sum * exp2a((mx - top) * kLog2e) : 0.f);
        if (lane == 0) { sh.task_max[t] = top; sh.task_sum[t] = sum; }
    }
    __syncthreads();
    // a beam's parts
    for (int k = warp; k < K; k += kWarps) {
        List list;
        list.k = K;
        float top = -INFINITY;
        for (int q = 0; q < a.parts; ++q) {
            list.offer(sh.task_key[k * a.parts + q][lane], lane);
            top = fmaxf(top, sh.task_max[k * a.parts + q]);
        }
        double sum = 0.0;
        if (top > -INFINITY)
            for (int q = 0; q < a.parts; ++q)
                sum += (double)sh.task_sum[k * a.parts + q] * (double)exp2f((sh.task_max[k * a.parts + q] - top) * kLog2e);
        sh.key[k][lane] = lane < K ? list.key : 0;
        if (lane == 0) { sh.mx[k] = top; sh.sum[k] = sum; }
    }
    cluster.sync();
    if (rank == 0) {
        for (int k = warp; k < K; k += kWarps) {
            List list;
            list.k = K;
            float top = -INFINITY;
            for (int c = 0; c < C; ++c) {
                const Shared* o = cluster.map_shared_rank(&sh, c);
                list.offer(o->key[k][lane], lane);
                top = fmaxf(top, o->mx[k]);
            }
            double sum = 0.0;
            if (top > -INFINITY)
                for (int c = 0; c < C; ++c) {
                    const Shared* o = cluster.map_shared_rank(&sh, c);
                    sum += o->sum[k] * exp((double)o->mx[k] - (double)top);
                }
            __syncwarp();
            sh.task_key[k][lane] = lane < K ? list.key : 0;  // this block's task lists have been read
            if (lane == 0) sh.lse[k] = top > -INFINITY ? (double)top + log(sum) : (double)INFINITY;
        }
        __syncthreads();
        if (warp == 0) {
            // lane k walks beam k's list; K times the best head, ties to the lower beam
            const bool beam = lane < K;
            const bool fin = beam && finished(lane);
            const double s0 = beam ? (double)a.scores[b * K + lane] : 0.0;
            int at = 0, token = 0;
            double head = 0.0;
            bool have = false;
            auto peek = [&]() {
                if (!beam) return;
                const u64 key = at < K ? sh.task_key[lane][at] : 0;
                have = fin ? at == 0 : key != 0;
                token = fin ? a.eos : (int)key_id(key);
                head = fin ? s0 : s0 + ((double)key_logit(key) - sh.lse[lane]);
                if (head != head) head = -INFINITY;
            };
            peek();
            float out_s = 0.f;
            int out_t = 0, out_p = 0, out_f = 0;
            for (int i = 0; i < K; ++i) {
                double s = head;
                int who = have ? lane : 64 + lane;  // one without a candidate loses against every other
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const double s2 = __shfl_xor_sync(0xffffffffu, s, o);
                    const int w2 = __shfl_xor_sync(0xffffffffu, who, o);
                    const bool take = (w2 < 64) != (who < 64) ? w2 < 64 : (s2 > s || (s2 == s && w2 < who));
                    if (take) { s = s2; who = w2; }
                }
                who &= 31;
                const int t = __shfl_sync(0xffffffffu, token, who);
                const int f = __shfl_sync(0xffffffffu, (int)fin, who);
                if (lane == i) {
                    out_s = (float)s;
                    out_t = t;
                    out_p = who;
                    out_f = f || t == a.eos;
                }
                if (lane == who) { ++at; peek(); }
            }
            if (beam) {
                const int to = b * K + lane;
                a.scores_out[to] = out_s;
                a.tokens[to] = out_t;
                a.parents[to] = out_p;
                if (a.finished_out) a.finished_out[to] = out_f;
            }
        }
    }
    cluster.sync();  // the first block has read every block's lists
}

template <typename A>
cudaError_t select_t(const void* logits, SelectArgs a, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.batch * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)a.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, beam_select_kernel<A>, reinterpret_cast<const A*>(logits), a);
    if (e != cudaSuccess) return e;
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(DType at, const void* logits, int batch, int beams, int V, const float* scores,
                               const int32_t* finished, int eos, float* scores_out, int32_t* tokens, int32_t* parents,
                               int32_t* finished_out, cudaStream_t s) {
    SelectArgs a{};
    a.batch = batch; a.beams = beams; a.V = V; a.eos = eos;
    a.scores = scores; a.finished = finished;
    a.scores_out = scores_out; a.tokens = tokens; a.parents = parents; a.finished_out = finished_out;
    a.cluster = V >= 8192 ? 8 : V >= 1024 ? 2 : 1;
    a.slice = ((V + a.cluster - 1) / a.cluster + 7) & ~7;
    a.parts = std::max(1, 16 / beams);
    return at == DT_BF16 ? select_t<bf16>(logits, a, s) : select_t<float>(logits, a, s);
}

}  // namespace nc
