// heavy.cu -- a draft cache that keeps its heavy hitters: attention that adds every
// row's attention weight up, and eviction of the rows of least weight (sm_103a).
//
//   out_r = sum_j p_rj v_j,  p_r = softmax_j(q_r . k_j / sqrt(d)),  weight_j += sum_r p_rj
//
// over the rows j of a KV head's compact cache and the R = n * G query rows that read it.
#include <cfloat>
#include <climits>

#include "common.cuh"

namespace magicdec {

// ----------------------------------------------------------------- attention
// Bound: HBM, 4 d + 8 bytes a cache row (K, V, the weight read and written) for 4 d R flops.
// A row's weight needs the whole softmax's maximum and sum, which are known when all keys have
// been seen; so the scores stay on chip until then: a cluster of C CTAs takes a (sequence, KV
// head), each a stretch of its keys and keeps their R scores in shared memory.  Then the CTAs
// exchange (max, sum), every row's weight is written once, and the O of all warps are summed in
// a fixed order.  No workspace, no atomics, one launch.
//
// A warp takes 16 keys at a time, straight from global memory into the fragments of
// mma.sync (m16n8k16): the order of the channels inside a product and of the output's
// columns is free, so that a lane's fragments are whole 16-byte words of a K row (channels
// 8 (lane % 4) .. of every 32) and of a V row (channels 8 (lane / 4) .. of every 64).  The
// products are a few percent of the time; what counts is the bytes under way: the K of the
// warp's next keys and the V of these.
constexpr int kHvWarps = 4;
constexpr int kHvThreads = kHvWarps * 32;
constexpr float kHvLazy = 24.0f;     // log2 growth of a row's maximum that is put up with

struct HeavyParams {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *weight;
    int32_t *pos;
    const int32_t *len, *next_pos;
    int *err;
    int B, H_q, H_kv, G, n, cap, R;
    int stride;                      // floats between two query rows' scores
    float scale_log2;                // log2(e) / sqrt(d)
};

__device__ __forceinline__ uint32_t hv_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t hv_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void hv_cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `p` in the shared memory of CTA `rank` of the cluster, and loads from there.
__device__ __forceinline__ uint32_t hv_at(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 hv_ld2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 hv_ld4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// A 16-byte load of K or V.  With two row tiles two warps read the same keys, the second from L1.
template <int MT>
__device__ __forceinline__ uint4 hv_ld(const uint4 *p) {
    if (MT == 1) return ld_dep_u4(p);
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// ROWS: query rows of a warp's tile that can be real, 8 or 16; MT: row tiles (a warp has one).
template <int D, int ROWS, int MT>
__global__ void __launch_bounds__(kHvThreads, ROWS == 8 ? 3 : 2) heavy_attn_kernel(const HeavyParams p) {
    constexpr int SP = D / 32;                          // spans of 32 channels
    constexpr int HV = D / 64;                          // halves of 64 channels
    constexpr int HR = ROWS / 8;                        // rows of a lane: lane / 4, and 8 more
    constexpr int KW = kHvWarps / MT;                   // warps that share the keys
    extern __shared__ __align__(16) uint8_t smem[];
    float *scores = reinterpret_cast<float *>(smem);    // [R][stride]; later the warps' O
    __shared__ float2 wstat[kHvWarps][16];              // of a warp's rows: (max, sum)
    __shared__ float2 cstat[32];                        // of this CTA
    __shared__ float2 all[32];                          // of the cluster: (max, 1 / sum)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lq = lane & 3, lr = lane >> 2;
    const int b = blockIdx.z, h = blockIdx.y;
    const uint32_t rank = hv_rank(), C = hv_ctas();
    const int mt = warp % MT, kw = warp / MT;
    const float sl = p.scale_log2;
    pdl_trigger();
    pdl_wait();
    const int len0 = checked(ld_dep(p.len + b), 0, p.cap, p.err);
    const int len = len0 < 0 ? 0 : (len0 > p.cap ? p.cap : len0);
    // This CTA's keys: [k0, k1), in groups of 16.
    const int per = ((len + (int)C - 1) / (int)C + 15) & ~15;
    const int k0 = min(len, (int)rank * per), k1 = min(len, k0 + per);
    const long long row0 = ((long long)b * p.H_kv + h) * p.cap;
    const uint4 *kb = reinterpret_cast<const uint4 *>(p.k + row0 * D);
    const uint4 *vb = reinterpret_cast<const uint4 *>(p.v + row0 * D);

    // The lane's query rows (i * G + g: token i, head g of the group), and how many keys they see.
    uint4 qf[SP][HR];
    int see[HR];
#pragma unroll
    for (int e = 0; e < HR; ++e) {
        const int r = mt * 16 + lr + 8 * e, i = r / p.G;
        see[e] = r < p.R ? len - p.n + 1 + i : 0;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (((long long)b * p.n + i) * p.H_q + h * p.G + (r - i * p.G)) * D);
#pragma unroll
        for (int s = 0; s < SP; ++s) qf[s][e] = r < p.R ? ld_dep_u4(src + s * 4 + lq) : make_uint4(0, 0, 0, 0);
    }
    float o[HV][8][2 * HR];                             // [half][channel][columns, rows]
#pragma unroll
    for (int f = 0; f < HV; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2 * HR; ++e) o[f][j][e] = 0.f;
    float m[HR], l[HR];
#pragma unroll
    for (int e = 0; e < HR; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
    }

    // D(16x8) += A(16x16) B(16x8); with 8 real rows the lower half of A and of D is not there.
    auto mma = [&](float *c, const uint32_t a0, const uint32_t a1, const uint32_t a2, const uint32_t a3, uint32_t b0,
                   uint32_t b1) {
        if (HR == 2) {
            asm volatile(
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                "{%0,%1,%2,%3};"
                : "+f"(c[0]), "+f"(c[1]), "+f"(c[2 * HR - 2]), "+f"(c[2 * HR - 1])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
        } else {
            asm volatile(
                "{\n\t.reg .f32 x, y;\n\t"
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,x,y}, {%2,%3,%4,%5}, {%6,%7}, "
                "{%0,%1,%8,%8};\n\t}"
                : "+f"(c[0]), "+f"(c[1])
                : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1), "f"(0.f));
        }
    };
    uint4 kf[2][SP];
    auto load_k = [&](int g) {                          // keys g .. g + 15; a row behind the last reads as zeros
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
            const int key = g + nb * 8 + lr;
#pragma unroll
            for (int s = 0; s < SP; ++s)
                kf[nb][s] = key < k1 ? hv_ld<MT>(kb + (long long)key * (D / 8) + s * 4 + lq) : make_uint4(0, 0, 0, 0);
        }
    };
    // The scores' place: row r of this warp's tile, key g.
    float *my = scores + (long long)(mt * 16 + lr) * p.stride - k0;
    int g = k0 + 16 * kw;
    if (g < k1) load_k(g);
    for (; g < k1; g += 16 * KW) {
        uint4 vf[4][HV];                                // V of keys 2 lq, 2 lq + 1, 2 lq + 8, 2 lq + 9
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int key = g + 2 * lq + (x & 1) + (x >> 1) * 8;
#pragma unroll
            for (int f = 0; f < HV; ++f)
                vf[x][f] = key < k1 ? hv_ld<MT>(vb + (long long)key * (D / 8) + f * 8 + lr) : make_uint4(0, 0, 0, 0);
        }
        float s[2][2 * HR];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
            for (int e = 0; e < 2 * HR; ++e) s[nb][e] = 0.f;
#pragma unroll
            for (int c = 0; c < SP; ++c) {
                const uint4 &a = qf[c][0], &a8 = qf[c][HR - 1];
                mma(s[nb], a.x, a8.x, a.y, a8.y, kf[nb][c].x, kf[nb][c].y);
                mma(s[nb], a.z, a8.z, a.w, a8.w, kf[nb][c].z, kf[nb][c].w);
            }
        }
        if (g + 16 * KW < k1) load_k(g + 16 * KW);
        // Keys that not every row sees: behind the last one, or of the block's own tokens.
        const bool edge = g + 16 > len - p.n + 1 || g + 16 > k1;
        float top[HR];
#pragma unroll
        for (int e = 0; e < HR; ++e) top[e] = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int e = 0; e < HR; ++e) {
                float &x = s[nb][2 * e], &y = s[nb][2 * e + 1];
                x *= sl;
                y *= sl;
                if (edge) {
                    const int key = g + nb * 8 + 2 * lq;
                    if (key >= min(see[e], k1)) x = -INFINITY;
                    if (key + 1 >= min(see[e], k1)) y = -INFINITY;
                }
                if (mt * 16 + lr + 8 * e < p.R)
                    *reinterpret_cast<float2 *>(my + (long long)(8 * e) * p.stride + g + nb * 8 + 2 * lq) =
                        make_float2(x, y);
                top[e] = fmaxf(top[e], fmaxf(x, y));
            }
        // The maximum moves, and O and the sum are scaled, only where it has grown by more than
        // 2^kHvLazy: weights up to 2^24 instead of 1 cost a floating sum nothing.
        bool move = false;
#pragma unroll
        for (int e = 0; e < HR; ++e) {
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
            move |= top[e] > m[e] + kHvLazy || (m[e] == -INFINITY && top[e] > m[e]);
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int e = 0; e < HR; ++e) {
                const float to = fmaxf(m[e], top[e]);
                const float f = to == -INFINITY ? 1.f : fast_exp2(m[e] - to);
                m[e] = to;
                l[e] *= f;
#pragma unroll
                for (int x = 0; x < HV; ++x)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        o[x][j][2 * e] *= f;
                        o[x][j][2 * e + 1] *= f;
                    }
            }
        }
        // P in bf16 for the second product: off by at most 2^-9 of itself, as the output's
        // rounding; the sum is of the unrounded values.
        uint32_t a[2][2] = {{0, 0}, {0, 0}};
#pragma unroll
        for (int e = 0; e < HR; ++e) {
            const float mu = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                const float x = fast_exp2(s[nb][2 * e] - mu), y = fast_exp2(s[nb][2 * e + 1] - mu);
                s[nb][2 * e] = x;
                s[nb][2 * e + 1] = y;
                l[e] += x + y;
                a[nb][e] = pack_bf16(x, y);
            }
        }
        if (p.n > 1 && g + 16 > len - p.n + 1) {
            // Keys of the block's own tokens, which earlier tokens must not see whatever they hold
            // (0 * inf is NaN): by scalars, and only where a row sees them.
            const int last = min(16, k1 - g);
            for (int x = 0; x < last; ++x) {
                const int key = g + x, from = (lane & ~3) | ((x & 7) >> 1);
                float w[HR];
#pragma unroll
                for (int e = 0; e < HR; ++e) {
                    const float even = x < 8 ? s[0][2 * e] : s[1][2 * e], odd = x < 8 ? s[0][2 * e + 1] : s[1][2 * e + 1];
                    w[e] = __shfl_sync(0xffffffffu, x & 1 ? odd : even, from);
                }
#pragma unroll
                for (int f = 0; f < HV; ++f)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {       // 8 channels of column 2 lq + c
                        const uint4 y = hv_ld<MT>(vb + (long long)key * (D / 8) + f * 8 + 2 * lq + c);
                        const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float vj = __uint_as_float(j & 1 ? z[j / 2] & 0xffff0000u : z[j / 2] << 16);
#pragma unroll
                            for (int e = 0; e < HR; ++e)
                                if (key < see[e]) o[f][j][2 * e + c] = fmaf(w[e], vj, o[f][j][2 * e + c]);
                        }
                    }
            }
            continue;
        }
#pragma unroll
        for (int f = 0; f < HV; ++f) {
            const uint32_t v0[4] = {vf[0][f].x, vf[0][f].y, vf[0][f].z, vf[0][f].w};
            const uint32_t v1[4] = {vf[1][f].x, vf[1][f].y, vf[1][f].z, vf[1][f].w};
            const uint32_t v8[4] = {vf[2][f].x, vf[2][f].y, vf[2][f].z, vf[2][f].w};
            const uint32_t v9[4] = {vf[3][f].x, vf[3][f].y, vf[3][f].z, vf[3][f].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {               // two keys' values of a channel side by side
                const uint32_t pick = j & 1 ? 0x7632u : 0x5410u;
                mma(o[f][j], a[0][0], a[0][HR - 1], a[1][0], a[1][HR - 1], __byte_perm(v0[j / 2], v1[j / 2], pick),
                    __byte_perm(v8[j / 2], v9[j / 2], pick));
            }
        }
    }

    // The warps' maxima and sums, the CTA's, the cluster's.
#pragma unroll
    for (int e = 0; e < HR; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if (lq == 0) wstat[warp][lr + 8 * e] = make_float2(m[e], l[e]);
    }
    __syncthreads();
    auto join = [](float2 &s, float2 x) {
        const float mx = fmaxf(s.x, x.x), mu = mx == -INFINITY ? 0.f : mx;
        s = make_float2(mx, s.y * fast_exp2(s.x - mu) + x.y * fast_exp2(x.x - mu));
    };
    if (tid < p.R) {
        float2 s = make_float2(-INFINITY, 0.f);
        for (int w = 0; w < KW; ++w) join(s, wstat[w * MT + tid / 16][tid % 16]);
        cstat[tid] = s;
    }
    if (C > 1) hv_cluster_sync();
    if (tid < p.R) {
        float2 s = make_float2(-INFINITY, 0.f);
        if (C > 1)
            for (uint32_t c = 0; c < C; ++c) join(s, hv_ld2(hv_at(&cstat[tid], c)));
        else
            s = cstat[tid];
        all[tid] = make_float2(s.x == -INFINITY ? 0.f : s.x, s.y > 0.f ? 1.f / s.y : 0.f);
    }
    __syncthreads();

    // Every row's weight, summed over the query rows in their order.
    const int first_new = p.next_pos ? len - p.n : INT_MAX;
    for (int j = k0 + tid; j < k1; j += kHvThreads) {
        float *w = p.weight + row0 + j;
        float sum = 0.f;
        const float old = j >= first_new ? 0.f : *w;
        for (int r = 0; r < p.R; ++r) sum = fmaf(fast_exp2(scores[(long long)r * p.stride + j - k0] - all[r].x), all[r].y, sum);
        *w = old + sum;
        if (j >= first_new) p.pos[row0 + j] = ld_dep(p.next_pos + b) + (j - first_new);
    }
    __syncthreads();

    // O of the warps, in the softmax's own scale: to shared memory, then summed over the warps
    // and over the CTAs, each of which has a share of the channels.
    float *osum = scores;                               // [KW][R][D]
#pragma unroll
    for (int e = 0; e < HR; ++e) {
        const int r = mt * 16 + lr + 8 * e;
        if (r >= p.R) continue;
        const float f = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - all[r].x) * all[r].y;
        float *to = osum + ((long long)kw * p.R + r) * D;
#pragma unroll
        for (int x = 0; x < HV; ++x)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4 *>(to + x * 64 + (2 * lq + c) * 8 + j) =
                        make_float4(o[x][j][2 * e + c] * f, o[x][j + 1][2 * e + c] * f, o[x][j + 2][2 * e + c] * f,
                                    o[x][j + 3][2 * e + c] * f);
    }
    if (C > 1) hv_cluster_sync();
    else __syncthreads();
    const int vecs = p.R * (D / 4), share = (vecs + (int)C - 1) / (int)C;
    for (int i = (int)rank * share + tid; i < min(vecs, (int)(rank + 1) * share); i += kHvThreads) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t c = 0; c < C; ++c) {
            const uint32_t base = hv_at(osum, c);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const float4 x = hv_ld4(base + (uint32_t)(w * vecs + i) * 16);
                s.x += x.x;
                s.y += x.y;
                s.z += x.z;
                s.w += x.w;
            }
        }
        const int r = i / (D / 4), c4 = i - r * (D / 4), t = r / p.G;
        *reinterpret_cast<uint2 *>(p.out + (((long long)b * p.n + t) * p.H_q + h * p.G + (r - t * p.G)) * D + c4 * 4) =
            make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
    if (C > 1) hv_cluster_sync();                       // no CTA ends while another reads its O
}

// ----------------------------------------------------------------- host side
constexpr int kHvMaxCluster = 16;

// Shared memory of a CTA whose cluster is C wide: the scores of its keys, or later the warps' O.
static size_t hv_smem(int cap, int R, int D, int C, int *stride) {
    const int warps = R <= 16 ? kHvWarps : kHvWarps / 2;
    const long long per = (((long long)cap + C - 1) / C + 15) / 16 * 16;
    // 8 floats more than a multiple of 32: neighbouring rows' scores lie in other banks.
    const long long st = (per + 23) / 32 * 32 + 8;
    *stride = (int)st;
    const long long a = st * R * 4, o = (long long)warps * R * D * 4;
    return (size_t)(a > o ? a : o);
}

template <int D, int ROWS, int MT>
static magicdec_status launch_heavy_t(const HeavyParams &p, int C, size_t smem, cudaStream_t st) {
    auto kern = heavy_attn_kernel<D, ROWS, MT>;
    if (!magicdec_host::allow_smem_once<heavy_attn_kernel<D, ROWS, MT>>(magicdec_host::max_smem_optin() - 2048) ||
        !magicdec_host::allow_wide_cluster_once<heavy_attn_kernel<D, ROWS, MT>>())
        return MAGICDEC_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, (unsigned)p.H_kv, (unsigned)p.B);
    cfg.blockDim = dim3(kHvThreads);
    cfg.dynamicSmemBytes = smem;
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
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return MAGICDEC_ERR_CUDA;
    return magicdec_host::launch_status();
}

magicdec_status launch_heavy_attn(int B, int H_q, int H_kv, int D, int cap, int n, const uint16_t *q,
                                  const uint16_t *k, const uint16_t *v, const int32_t *len, const int32_t *next_pos,
                                  float *weight, int32_t *pos, uint16_t *out, cudaStream_t st) {
    HeavyParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = out;
    p.weight = weight;
    p.pos = pos;
    p.len = len;
    p.next_pos = next_pos;
    p.err = magicdec_host::device_error_word();
    p.B = B;
    p.H_q = H_q;
    p.H_kv = H_kv;
    p.G = H_q / H_kv;
    p.n = n;
    p.cap = cap;
    p.R = n * p.G;
    p.scale_log2 = kLog2e / sqrtf((float)D);
    // As wide a cluster as it takes to have 8 CTAs an SM in all, with 64 keys each at least, and for
    // the scores to leave room for three CTAs an SM.
    const int limit = magicdec_host::max_smem_optin() - 2048;
    int C = 1;
    while (C < 8 && (long long)B * H_kv * C < 8ll * magicdec_host::sm_count() && cap > C * 64) C *= 2;
    size_t smem = hv_smem(cap, p.R, D, C, &p.stride);
    while (C < kHvMaxCluster && smem > 72 * 1024) smem = hv_smem(cap, p.R, D, C *= 2, &p.stride);
    if (smem > (size_t)limit) return MAGICDEC_ERR_UNSUPPORTED;
    if (D == 128)
        return p.R <= 8 ? launch_heavy_t<128, 8, 1>(p, C, smem, st)
                        : p.R <= 16 ? launch_heavy_t<128, 16, 1>(p, C, smem, st) : launch_heavy_t<128, 16, 2>(p, C, smem, st);
    return p.R <= 8 ? launch_heavy_t<64, 8, 1>(p, C, smem, st)
                    : p.R <= 16 ? launch_heavy_t<64, 16, 1>(p, C, smem, st) : launch_heavy_t<64, 16, 2>(p, C, smem, st);
}

// ------------------------------------------------------------------ eviction
// Of a (layer, sequence, KV head)'s len rows the `budget` with the largest key stay.  A row's
// key is its weight, infinity for the protected ones; equal keys: the smaller position stays, then
// the smaller row.  Seen from the other end, the E = len - budget least go; the border is found
// digit by digit over (weight, position, row), most significant first, from counts of the rows
// that agree with the border so far.  Rows that stay behind the budget then fill the holes below
// it, in ascending order of both, so that a step that evicts E rows moves at most E.
// Bound: 8 bytes a row (weight, position) from HBM, in practice the chain of a CTA's passes.
constexpr int kEvThreads = 256;
constexpr int kEvMoves = 512;            // moves listed at a time
constexpr int kEvBits = 8;

struct EvictParams {
    uint4 *kc, *vc;
    float *weight;
    int32_t *pos;
    const int32_t *len, *seq_len;
    int32_t *len_out;
    int *err;
    int B, H_kv, cap, vecs, budget, n_sink, n_recent;
    int keep;                            // rows whose keys fit shared memory
};

// Order of fp32 as unsigned integers; both zeros are one.
__device__ __forceinline__ uint32_t ev_key(float w) {
    const uint32_t x = __float_as_uint(w + 0.f);
    return x & 0x80000000u ? ~x : x | 0x80000000u;
}

__global__ void __launch_bounds__(kEvThreads) heavy_evict_kernel(const EvictParams p) {
    extern __shared__ uint32_t kept[];                       // keys of the first p.keep rows
    __shared__ int hist[1 << kEvBits];
    __shared__ int found[2];                                 // the border's digit, rows below it
    __shared__ int src[kEvMoves], dst[kEvMoves];
    __shared__ int wsum[2][kEvThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x, b = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    const int len0 = checked(ld_dep(p.len + b), 0, p.cap, p.err);
    const int len = len0 < 0 ? 0 : (len0 > p.cap ? p.cap : len0);
    if (h == 0 && blockIdx.z == 0 && tid == 0) p.len_out[b] = min(len, p.budget);
    int E = len - p.budget;                                  // rows to go
    if (E <= 0) return;
    const long long row0 = (((long long)blockIdx.z * p.B + b) * p.H_kv + h) * p.cap;
    float *weight = p.weight + row0;
    int32_t *pos = p.pos + row0;
    const long long recent = (long long)ld_dep(p.seq_len + b) - p.n_recent;
    auto fresh = [&](int j) {
        const int at = ld_dep(pos + j);
        return at < p.n_sink || at >= recent ? ev_key(INFINITY) : ev_key(__uint_as_float(ld_dep_u32(
                                                   reinterpret_cast<const unsigned *>(weight + j))));
    };
    for (int j = tid; j < min(len, p.keep); j += kEvThreads) kept[j] = fresh(j);
    auto key = [&](int j) { return j < p.keep ? kept[j] : fresh(j); };
    // What goes first: small weights, large positions, high rows.
    auto part = [&](int word, int j) {
        return word == 0 ? key(j) : word == 1 ? ~((uint32_t)ld_dep(pos + j) ^ 0x80000000u) : ~(uint32_t)j;
    };
    uint32_t border[3] = {0, 0, 0};
    int words = 3;                                           // words of the border that count
    bool whole = false;                                      // everything that agrees with the border goes
    uint32_t mask = 0;                                       // digits of the current word that are settled
    int left = E;
    for (int word = 0; word < 3 && !whole; ++word) {
        mask = 0;
        for (int shift = 32 - kEvBits; shift >= 0 && !whole; shift -= kEvBits) {
            __syncthreads();
            for (int i = tid; i < 1 << kEvBits; i += kEvThreads) hist[i] = 0;
            __syncthreads();
            for (int j = tid; j < len; j += kEvThreads) {
                bool same = true;
                for (int w = 0; w < word && same; ++w) same = part(w, j) == border[w];
                if (!same) continue;
                const uint32_t x = part(word, j);
                if ((x & mask) == (border[word] & mask)) atomicAdd(&hist[x >> shift & ((1 << kEvBits) - 1)], 1);
            }
            __syncthreads();
            // The digit at which the running count reaches `left`.
            const int c = hist[tid];
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane == 31) wsum[0][warp] = incl;
            __syncthreads();
            for (int w = 0; w < warp; ++w) incl += wsum[0][w];
            if (incl >= left && incl - c < left) {
                found[0] = tid;
                found[1] = incl - c;
            }
            __syncthreads();
            const int digit = found[0];
            border[word] |= (uint32_t)digit << shift;
            mask |= (uint32_t)((1 << kEvBits) - 1) << shift;
            left -= found[1];
            whole = hist[digit] == left;
            words = word + 1;
        }
    }
    static_assert(kEvThreads == 1 << kEvBits, "a thread has a digit");
    // Whether row j goes: below the border, or in agreement with it as far as it was settled.
    auto goes = [&](int j) {
        for (int w = 0; w < words; ++w) {
            const uint32_t m = w + 1 == words ? mask : 0xffffffffu;
            const uint32_t x = part(w, j) & m, y = border[w] & m;
            if (x != y) return x < y;
        }
        return true;
    };
    // One bit a row, so that weights and positions may move afterwards.
    uint32_t *gone = kept + p.keep;
    const int nw = (len + 31) / 32;
    for (int w = warp; w < nw; w += kEvThreads / 32) {
        const int j = w * 32 + lane;
        const unsigned m = __ballot_sync(0xffffffffu, j < len && goes(j));
        if (lane == 0) gone[w] = m;
    }
    __syncthreads();
    // Holes below the budget and the rows to fill them, listed kEvMoves at a time.
    const int per = 2 * p.vecs, rows = kEvThreads / per, c = tid % per;   // threads of a row of K and V
    uint4 *base = (c < p.vecs ? p.kc + c : p.vc + (c - p.vecs)) + row0 * p.vecs;
    for (int done = 0, holes = 1; done < holes; done += kEvMoves) {
        holes = 0;
        int late = 0;                                        // found so far, alike in all threads
        for (int w0 = 0; w0 < nw; w0 += kEvThreads) {
            const int w = w0 + tid;
            unsigned hole = 0, stay = 0;
            if (w < nw) {
                const int under = p.budget - w * 32, in = len - w * 32;
                const unsigned below = under >= 32 ? ~0u : under <= 0 ? 0u : (1u << under) - 1u;
                const unsigned real = in >= 32 ? ~0u : (1u << in) - 1u;
                hole = gone[w] & below;
                stay = ~gone[w] & real & ~below;
            }
            int ih = __popc(hole), is = __popc(stay);
            const int ch = ih, cs = is;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, ih, o), y = __shfl_up_sync(0xffffffffu, is, o);
                if (lane >= o) {
                    ih += x;
                    is += y;
                }
            }
            if (lane == 31) {
                wsum[0][warp] = ih;
                wsum[1][warp] = is;
            }
            __syncthreads();
            int ah = holes + ih - ch, as = late + is - cs;
            for (int x = 0; x < kEvThreads / 32; ++x) {
                if (x < warp) {
                    ah += wsum[0][x];
                    as += wsum[1][x];
                }
                holes += wsum[0][x];
                late += wsum[1][x];
            }
            for (; hole; hole &= hole - 1, ++ah)
                if (ah >= done && ah < done + kEvMoves) dst[ah - done] = w * 32 + __ffs(hole) - 1;
            for (; stay; stay &= stay - 1, ++as)
                if (as >= done && as < done + kEvMoves) src[as - done] = w * 32 + __ffs(stay) - 1;
            __syncthreads();
        }
        const int moves = min(holes - done, kEvMoves);       // there are as many holes as rows to fill them
        for (int i = tid / per; i < moves; i += rows)
            base[(long long)dst[i] * p.vecs] = ld_dep_u4(base + (long long)src[i] * p.vecs);
        for (int i = tid; i < moves; i += kEvThreads) {
            weight[dst[i]] = weight[src[i]];
            pos[dst[i]] = pos[src[i]];
        }
        __syncthreads();
    }
}

constexpr int kEvKeep = 24 * 1024;       // keys in shared memory at most
constexpr int kEvMaxRows = 1 << 20;

magicdec_status launch_heavy_evict(int layers, int B, int H_kv, int D, int cap, const int32_t *len,
                                   const int32_t *seq_len, int budget, int n_sink, int n_recent, uint16_t *kc,
                                   uint16_t *vc, float *weight, int32_t *pos, int32_t *len_out, cudaStream_t st) {
    if (cap > kEvMaxRows) return MAGICDEC_ERR_UNSUPPORTED;
    EvictParams p{};
    p.kc = reinterpret_cast<uint4 *>(kc);
    p.vc = reinterpret_cast<uint4 *>(vc);
    p.weight = weight;
    p.pos = pos;
    p.len = len;
    p.seq_len = seq_len;
    p.len_out = len_out;
    p.err = magicdec_host::device_error_word();
    p.B = B;
    p.H_kv = H_kv;
    p.cap = cap;
    p.vecs = D / 8;
    p.budget = budget;
    p.n_sink = n_sink;
    p.n_recent = n_recent;
    p.keep = cap < kEvKeep ? cap : cap <= kEvMaxRows / 2 ? kEvKeep : kEvKeep / 2;
    const int smem = (p.keep + (cap + 31) / 32) * 4;         // at most 192 KB
    if (!magicdec_host::allow_smem_once<heavy_evict_kernel>(200 * 1024)) return MAGICDEC_ERR_CUDA;
    return magicdec_host::launch_pdl(heavy_evict_kernel, dim3((unsigned)H_kv, (unsigned)B, (unsigned)layers),
                                     dim3(kEvThreads), (size_t)smem, st, p);
}

}  // namespace magicdec
