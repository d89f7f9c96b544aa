// tree_accept.cu -- greedy acceptance down a tree of drafted tokens (sm_103a).
//
// From node 0 (the last emitted token): t = argmax of the target's logits at
// the node, ties to the smaller token; the walk goes on to the lowest child
// whose token is t, and ends, emitting t, where there is none.  Only the rows of
// the visited nodes are read: (n_acc + 1) * V * 4 bytes per sequence, one after
// the other, since each row's argmax says which is next.
//
// A cluster of CTAs shares a row: each takes a slice, and the slices' best keys
// (value, then lower index, packed in 64 bits) are exchanged through distributed
// shared memory with one cluster barrier per level.
//
// Bound: HBM while all sequences are at it, a chain of latencies (a row's loads, two
// reductions, the barrier: about 2 us) when few are.  V = 128,256, logits from HBM, 128
// sequences that accept 0 to 4 nodes: 43.9 us on the GPU, of 29 us at the measured copy rate;
// 6 nodes each: 76 us, of 68; one sequence, V = 152,064, four rows: 9.3 us.  Copies through
// shared memory in place of the loads, 96 KB a CTA under way, measured slower (55 us, where the
// loads alone then took 46): what a CTA does for a piece of 16 KB costs more than the loads' latency.
#include <climits>

#include "common.cuh"

namespace magicdec {

constexpr int kTaThreads = 512;
constexpr int kTaMaxCluster = 16;
constexpr int kTaMaxNodes = 256;
constexpr int kTaPerSm = 2;             // CTAs an SM holds
constexpr int kTaAsk = 2048;            // 16-byte vectors of a prefetch
constexpr int kTaAhead = 4;             // loads of a thread under way
static_assert(kTaMaxNodes <= kTaThreads, "one thread holds a node's token and parent");

struct TreeAcceptParams {
    const float *target;             // [B, n, V]
    const int32_t *tok, *parent, *n_nodes;
    int32_t *n_acc, *path, *out_tok;
    int *err;
    int n, V;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The two halves of a cluster barrier, for whole warps.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// Store to the same shared-memory variable of CTA `rank` of the cluster, which has to be known to run.
__device__ __forceinline__ void st_cluster_u64(uint64_t *p, uint32_t rank, uint64_t v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// Order-preserving key: larger value first, then the smaller index.  -0 counts
// as +0 (they compare equal, so the smaller index has to win); 0 stands for no
// value above -infinity.
__device__ __forceinline__ uint64_t best_key(float v, uint32_t idx) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return v > -INFINITY ? ((uint64_t)o << 32) | (uint32_t)~idx : 0;
}
// The largest key of a warp, as two 32-bit reductions.
__device__ __forceinline__ uint64_t warp_best(uint64_t key) {
    const uint32_t hi = (uint32_t)(key >> 32), top = __reduce_max_sync(0xffffffffu, hi);
    return ((uint64_t)top << 32) | __reduce_max_sync(0xffffffffu, hi == top ? (uint32_t)key : 0u);
}

__global__ void __launch_bounds__(kTaThreads, kTaPerSm) tree_accept_kernel(const TreeAcceptParams p) {
    __shared__ uint64_t slot[2][kTaMaxCluster];
    __shared__ uint64_t wbest[kTaThreads / 32];
    __shared__ int wnext[kTaMaxNodes / 32];
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Every CTA says here that it runs.  Another one's shared memory is there only from then on, so
    // the first store to it waits for all of them; the first row's loads lie between.
    cluster_arrive();
    pdl_trigger();
    pdl_wait();
    const int raw = p.n_nodes ? checked(ld_dep(p.n_nodes + b), 0, p.n, p.err) : p.n;
    const int nn = raw < 0 ? 0 : (raw > p.n ? p.n : raw);
    int my_tok = -1, my_par = -1;
    if (tid < nn) {
        my_tok = ld_dep(p.tok + (long long)b * p.n + tid);
        my_par = p.parent ? checked(ld_dep(p.parent + (long long)b * p.n + tid), INT_MIN, tid - 1, p.err) : tid - 1;
        if (my_par >= tid) my_par = -1;
    }
    int32_t *path = p.path + (long long)b * p.n, *out = p.out_tok + (long long)b * p.n;
    int u = nn > 0 ? 0 : -1, level = 0;
    while (u >= 0) {
        const float *row = p.target + ((long long)b * p.n + u) * p.V;
        // The first elements up to a 16-byte boundary and the last ones go one by one.
        const int mis = (int)((reinterpret_cast<uintptr_t>(row) >> 2) & 3);
        const int pre = min(p.V, (4 - mis) & 3), nv = (p.V - pre) / 4, post = pre + nv * 4;
        const int v0 = (int)((long long)nv * rank / C), v1 = (int)((long long)nv * (rank + 1) / C);
        const float4 *vec = reinterpret_cast<const float4 *>(row + pre);
        // The slice is on its way to L2 as a whole while the threads load it bit by bit, as long
        // as there are few sequences, whose rate hangs on how much of a row is under way.  With,
        // and without it (V = 128,256, us on the GPU, logits from HBM, of sequences that accept
        // 0 to 4 nodes evenly, 6 each, none): 16 sequences 18.4, 40.6, 6.6 and 18.9, 41.6, 7.2;
        // 50 sequences 25.5, 38.0, 7.8 and 27.0, 41.7, 7.5; 76 sequences 33.8, 74.5, 13.5 and
        // 34.4, 81.2, 13.2; 100 sequences, two CTAs a row, 40.5, 69.2, 13.1 and 40.4, 65.3, 11.1;
        // 128 sequences 46.3, 85.8, 14.9 and 43.8, 75.8, 12.7.
        if (C >= 4)
            for (int at = v0 + tid * kTaAsk; at < v1; at += kTaThreads * kTaAsk)
                bulk_prefetch_l2(vec + at, (uint32_t)min(kTaAsk, v1 - at) * 16);
        // The largest of a thread's vectors, the first of equal ones.
        float best = -INFINITY;
        float4 at = make_float4(best, best, best, best);
        int vi = 0;
        auto see = [&](float4 x, int i) {
            const float m = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
            if (m > best) {
                best = m;
                at = x;
                vi = i;
            }
        };
        int i = v0 + tid;
        for (; i + (kTaAhead - 1) * kTaThreads < v1; i += kTaAhead * kTaThreads) {
            float4 x[kTaAhead];
#pragma unroll
            for (int k = 0; k < kTaAhead; ++k) x[k] = ld_dep_f4(vec + i + k * kTaThreads);
#pragma unroll
            for (int k = 0; k < kTaAhead; ++k) see(x[k], i + k * kTaThreads);
        }
        {
            float4 x[kTaAhead];
#pragma unroll
            for (int k = 0; k < kTaAhead - 1; ++k)
                if (i + k * kTaThreads < v1) x[k] = ld_dep_f4(vec + i + k * kTaThreads);
#pragma unroll
            for (int k = 0; k < kTaAhead - 1; ++k)
                if (i + k * kTaThreads < v1) see(x[k], i + k * kTaThreads);
        }
        const uint32_t first = pre + 4 * vi;
        uint64_t key = best_key(best, first + (at.x == best ? 0 : at.y == best ? 1 : at.z == best ? 2 : 3));
        if (rank == 0 && tid < pre) key = max(key, best_key(ld_dep_f(row + tid), tid));
        if (rank == C - 1 && tid < p.V - post) key = max(key, best_key(ld_dep_f(row + post + tid), post + tid));
        key = warp_best(key);
        if (level == 0) cluster_wait();                         // from now on all CTAs of the cluster run
        if (lane == 0) wbest[warp] = key;
        __syncthreads();
        if (warp == 0) {
            key = warp_best(lane < kTaThreads / 32 ? wbest[lane] : 0);
            if (lane < C) st_cluster_u64(&slot[level & 1][rank], lane, key);
        }
        // One barrier per level: a slot is written again two levels on, after the next
        // barrier, which no CTA reaches before it has read this level's slots.
        cluster_sync();
        key = warp_best(lane < C ? slot[level & 1][lane] : 0);
        const int t = key ? (int)~(uint32_t)key : 0;            // nothing above -infinity: all are equal
        const bool go = tid < nn && my_par == u && my_tok == t;
        const unsigned m = __ballot_sync(0xffffffffu, go);
        if (lane == 0 && warp < kTaMaxNodes / 32) wnext[warp] = m ? warp * 32 + __ffs(m) - 1 : -1;
        __syncthreads();
        int next = -1;
        for (int w = kTaMaxNodes / 32 - 1; w >= 0; --w) next = wnext[w] >= 0 ? wnext[w] : next;
        if (rank == 0 && tid == 0) {
            path[level] = u;
            out[level] = t;
        }
        u = next;
        ++level;
    }
    if (level == 0) cluster_wait();                             // no nodes: the arrival's other half
    if (rank == 0) {
        if (tid == 0) p.n_acc[b] = level - 1;
        for (int i = level + tid; i < p.n; i += kTaThreads) {
            path[i] = -1;
            out[i] = -1;
        }
    }
}

magicdec_status launch_tree_accept(int B, int n, int V, const float *target, const int32_t *tok,
                                   const int32_t *parent, const int32_t *n_nodes, int32_t *n_acc, int32_t *path,
                                   int32_t *out_tok, cudaStream_t st) {
    TreeAcceptParams p{};
    p.target = target;
    p.tok = tok;
    p.parent = parent;
    p.n_nodes = n_nodes;
    p.n_acc = n_acc;
    p.path = path;
    p.out_tok = out_tok;
    p.err = magicdec_host::device_error_word();
    p.n = n;
    p.V = V;
    // As many CTAs a row as there are places for.  So, and with twice as many (inputs as above):
    // 38 sequences 20.5, 49.9, 9.3 and 33.0, 63.8, 11.6 us; 50 sequences 25.5, 38.0, 7.8 and
    // 27.7, 54.6, 9.9; 128 sequences 44.0, 76.1, 12.8 and 48.6, 87.0, 16.8; 200 sequences 70.6,
    // 116.7, 18.9 and 66.3, 137.2, 21.8.
    int C = kTaMaxCluster;
    while (C > 1 && (long long)B * C > (long long)kTaPerSm * magicdec_host::sm_count()) C /= 2;
    if (!magicdec_host::allow_wide_cluster_once<tree_accept_kernel>()) return MAGICDEC_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B * C);
    cfg.blockDim = dim3(kTaThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, tree_accept_kernel, p) != cudaSuccess) return MAGICDEC_ERR_CUDA;
    return magicdec_host::launch_status();
}

}  // namespace magicdec
