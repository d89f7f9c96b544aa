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
#include "common.cuh"

namespace magicdec {

constexpr int kTaThreads = 512;
constexpr int kTaMaxCluster = 16;
constexpr int kTaMaxNodes = 256;
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
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store to the same shared-memory variable of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_u64(uint64_t *p, uint32_t rank, uint64_t v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// Order-preserving key: larger value first, then the smaller index.  -0 counts
// as +0 (they compare equal, so the smaller index has to win).
__device__ __forceinline__ uint64_t best_key(float v, uint32_t idx) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~idx;
}

struct Best {
    float v;
    uint32_t idx;
    __device__ __forceinline__ void see(float x, uint32_t i) {
        if (x > v || idx == 0xffffffffu) {       // a thread meets its indices in ascending order
            v = x;
            idx = i;
        }
    }
};

__global__ void __launch_bounds__(kTaThreads) tree_accept_kernel(const TreeAcceptParams p) {
    __shared__ uint64_t slot[2][kTaMaxCluster];
    __shared__ uint64_t wbest[kTaThreads / 32];
    __shared__ int wnext[kTaMaxNodes / 32];
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    const int raw = p.n_nodes ? checked(ld_dep(p.n_nodes + b), 0, p.n, p.err) : p.n;
    const int nn = raw < 0 ? 0 : (raw > p.n ? p.n : raw);
    int my_tok = -1, my_par = -1;
    if (tid < nn) {
        my_tok = ld_dep(p.tok + (long long)b * p.n + tid);
        my_par = p.parent ? checked(ld_dep(p.parent + (long long)b * p.n + tid), -1, tid - 1, p.err) : tid - 1;
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
        Best best{-INFINITY, 0xffffffffu};
        if (rank == 0 && tid < pre) best.see(ld_dep_f(row + tid), tid);
#pragma unroll 8
        for (int i = v0 + tid; i < v1; i += kTaThreads) {
            const float4 x = ld_dep_f4(vec + i);
            const uint32_t e = pre + 4 * i;
            best.see(x.x, e);
            best.see(x.y, e + 1);
            best.see(x.z, e + 2);
            best.see(x.w, e + 3);
        }
        if (rank == C - 1 && tid < p.V - post) best.see(ld_dep_f(row + post + tid), post + tid);
        uint64_t key = best.idx == 0xffffffffu ? 0 : best_key(best.v, best.idx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
        if (lane == 0) wbest[warp] = key;
        __syncthreads();
        if (warp == 0) {
            key = lane < kTaThreads / 32 ? wbest[lane] : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
            if (lane < C) st_cluster_u64(&slot[level & 1][rank], lane, key);
        }
        // One barrier per level: a slot is written again two levels on, after the next
        // barrier, which no CTA reaches before it has read this level's slots.
        cluster_sync();
        key = slot[level & 1][0];
        for (uint32_t c = 1; c < C; ++c) key = max(key, slot[level & 1][c]);
        const int t = (int)~(uint32_t)key;
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
    // As many CTAs a row as there are places for all sequences at once (four CTAs an SM).
    int C = kTaMaxCluster;
    while (C > 1 && (long long)B * C > 4ll * magicdec_host::sm_count()) C /= 2;
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
