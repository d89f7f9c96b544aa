// heavy.cu -- a draft cache that keeps its heavy hitters: attention that adds every
// row's attention weight up, and eviction of the rows of least weight (sm_103a).
//
//   out_r = sum_j p_rj v_j,  p_r = softmax_j(q_r . k_j / sqrt(d)),  weight_j += sum_r p_rj
//
// over the rows j of a KV head's compact cache and the R = n * G query rows that read it.
#include <cfloat>
#include <climits>

#include "few_rows.cuh"
#include "heavy.cuh"

namespace magicdec {

// ----------------------------------------------------------------- attention
// Bound: HBM, 4 d + 8 bytes a cache row (K, V, the weight read and written) for 4 d R flops.
// A row's weight needs the whole softmax's maximum and sum, which are known when all keys have
// been seen.  So a cluster of C CTAs takes a (sequence, KV head), each a stretch of its keys, and
// after one pass over K and V the CTAs exchange (max, sum); then every row's weight is written
// once, from the scores, which stay in shared memory until then.  The O of all warps are summed in
// a fixed order.  No workspace, no atomics, one launch.  This is the way of up to 8 query rows whose
// scores fit; the others' is heavy_tc.cu.
//
// A producer warp keeps a ring of stages filled by TMA, 64 keys' K and V each; 4 consumer warps take 16
// keys of a stage each through ldmatrix and mma.sync (m16n8k16, the lower half of A empty): at 8 rows
// the products are a few percent of the time.  128 sequences over 2053 rows, R = 4: 179 us,
// 6.1 TB/s; with keys straight from global memory into the fragments, which left too few bytes
// under way, 207; on tcgen05 223.
constexpr int kHvKeys = 64;          // keys of a stage
constexpr int kHvHalf = kHvKeys * 128;   // bytes of 64 channels of them
constexpr int kHvStages = 8;         // stages of a ring at most
constexpr int kHvRows = 8;           // query rows at most
constexpr int kHvWarps = 4;          // consumer warps
constexpr int kHvThreads = kHvWarps * 32 + 32;

template <int D>
__global__ void __launch_bounds__(kHvThreads, 2)
    heavy_attn_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ CUtensorMap tmk16, const __grid_constant__ CUtensorMap tmv16,
                      const HeavyParams p) {
    constexpr int KS = D / 16, HV = D / 64, NB = D / 8;
    constexpr int OPER = HV * kHvHalf, STAGE = 2 * OPER;
    constexpr int OROW = D + 8;                         // floats of a row of O: rows lie in other banks
    constexpr int QHALF = kHvRows * 128;                // bytes of 64 channels of the query rows
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem;                               // later the warps' O
    float *scores = reinterpret_cast<float *>(smem + p.stages * STAGE);     // [R][stride]
    __shared__ __align__(1024) uint8_t qs[HV * QHALF];
    __shared__ uint64_t full[kHvStages], empty[kHvStages];
    __shared__ float2 wstat[kHvWarps][kHvRows];         // of a warp's keys: (max, sum)
    __shared__ float2 cstat[kHvRows];                   // of this CTA
    __shared__ float2 all[kHvRows];                     // of the cluster: (max, 1 / sum)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lq = lane & 3, lr = lane >> 2;            // fragments: columns 2 lq, row lr
    const int b = blockIdx.z, h = blockIdx.y;
    const uint32_t rank = few_rank(), C = few_ctas();
    const float sl = p.scale_log2;
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kHvWarps);
        }
        mbar_fence_init();
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    pdl_trigger();
    pdl_wait();
    // The query rows (row i * G + g: token i, head g of the group), swizzled as the keys.
    static_assert(kHvRows * (D / 8) <= kHvThreads, "a thread has a 16-byte word of the query rows");
    const int qr = tid / (D / 8), qc = tid % (D / 8), qi = qr / p.G;
    const uint16_t *qsrc = p.q + (((long long)b * p.n + qi) * p.H_q + h * p.G + (qr - qi * p.G)) * D + qc * 8;
    const uint4 qv = qr < p.R ? ld_dep_u4(reinterpret_cast<const uint4 *>(qsrc)) : make_uint4(0, 0, 0, 0);
    const int len0 = checked(ld_dep(p.len + b), 0, p.cap, p.err);
    if (qr < kHvRows) *reinterpret_cast<uint4 *>(qs + (qc >> 3) * QHALF + swz128(qr, qc & 7)) = qv;
    __syncthreads();
    const int len = len0 < 0 ? 0 : (len0 > p.cap ? p.cap : len0);
    // This CTA's keys: [k0, k1), in groups of 16.
    const int per = ((len + (int)C - 1) / (int)C + 15) & ~15;
    const int k0 = min(len, (int)rank * per), k1 = min(len, k0 + per), tiles = (k1 - k0 + kHvKeys - 1) / kHvKeys;
    const long long row0 = ((long long)b * p.H_kv + h) * p.cap;
    bool ok = smem_u32(smem) % 1024 == 0;
    if (!ok && tid == 0) raise_error(p.err, kErrState);

    if (warp == kHvWarps) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            const uint64_t once = policy_evict_first();
            for (int t = 0; ok && t < tiles; ++t) {
                const uint32_t st = (uint32_t)t % p.stages;
                ok = mbar_poll(&empty[st], ((uint32_t)t / p.stages & 1) ^ 1, p.err);
                if (!ok) break;
                const int key = k0 + t * kHvKeys, groups = (min(kHvKeys, k1 - key) + 15) / 16;
                uint8_t *to = ring + st * STAGE;
                mbar_arrive_expect_tx(&full[st], (uint32_t)(groups * 2 * HV * 2048));
                for (int f = 0; f < HV; ++f) {
                    if (groups == 4) {
                        tma_load_4d(to + f * kHvHalf, &tmk, f * 64, key, h, b, &full[st], once);
                        tma_load_4d(to + OPER + f * kHvHalf, &tmv, f * 64, key, h, b, &full[st], once);
                    } else {
                        for (int g = 0; g < groups; ++g) {
                            tma_load_4d(to + f * kHvHalf + g * 2048, &tmk16, f * 64, key + g * 16, h, b, &full[st], once);
                            tma_load_4d(to + OPER + f * kHvHalf + g * 2048, &tmv16, f * 64, key + g * 16, h, b, &full[st],
                                        once);
                        }
                    }
                }
            }
            // No copy may be in flight when the CTA ends, or when O takes the ring.
            for (int t = max(0, tiles - p.stages); t < tiles; ++t)
                mbar_poll(&full[t % p.stages], (uint32_t)t / p.stages & 1, p.err);
        }
        __syncwarp();
    }
    float o[NB][2], m = -INFINITY, l = 0.f;
    if (warp < kHvWarps) {
        // Query row r sees keys below this.
        const int see = lr < p.R ? min(len - p.n + 1 + lr / p.G, k1) : 0;
        uint32_t qf[KS][2];
#pragma unroll
        for (int c = 0; c < KS; c += 2)
            ldsm_x4(smem_u32(qs) + (c >> 2) * QHALF + (swz128(lane & 7, lane >> 3) ^ ((c & 3) * 32)), qf[c][0], qf[c][1],
                    qf[c + 1][0], qf[c + 1][1]);
#pragma unroll
        for (int j = 0; j < NB; ++j) o[j][0] = o[j][1] = 0.f;
        // The scores' place: row lr, key g.
        float *my = scores + (long long)lr * p.stride - k0;
        // A lane's address in a K tile, and in a V tile: 16-byte chunk c of its row is at c * 16 away from
        // chunk 0 in the sense of an exclusive or (8 chunks a half).
        const int x4 = lane >> 3, r0 = 16 * warp;
        const uint32_t k_lane = swz128(r0 + (x4 >> 1) * 8 + (lane & 7), x4 & 1);
        const uint32_t v_lane = swz128(r0 + (x4 & 1) * 8 + (lane & 7), x4 >> 1);
        for (int t = 0; t < tiles; ++t) {
            const uint32_t st = (uint32_t)t % p.stages, kt = smem_u32(ring + st * STAGE), vt = kt + OPER;
            ok = few_wait(&full[st], (uint32_t)t / p.stages & 1, p.err, ok, lane);
            const int g = k0 + t * kHvKeys + r0;
            if (g < k1) {
                // Two chains of products a score, so that half as many wait for one another.
                float s[2][2] = {}, s2[2][2] = {};
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                    uint32_t f0, f1, f2, f3;
                    ldsm_x4(((kt + k_lane) ^ ((c & 3) * 32)) + (c >> 2) * kHvHalf, f0, f1, f2, f3);
                    few_mma<1>(c & 1 ? s2[0] : s[0], qf[c], f0, f1);
                    few_mma<1>(c & 1 ? s2[1] : s[1], qf[c], f2, f3);
                }
                // Keys that not every row sees: behind the last one, or of the block's own tokens.
                const bool edge = g + 16 > len - p.n + 1 || g + 16 > k1;
                float top = -INFINITY;
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    float &x = s[nb][0], &y = s[nb][1];
                    x = (x + s2[nb][0]) * sl;
                    y = (y + s2[nb][1]) * sl;
                    const int key = g + nb * 8 + 2 * lq;
                    if (edge) {
                        if (key >= see) x = -INFINITY;
                        if (key + 1 >= see) y = -INFINITY;
                    }
                    if (lr < p.R) *reinterpret_cast<float2 *>(my + key) = make_float2(x, y);
                    top = fmaxf(top, fmaxf(x, y));
                }
                // The maximum moves, and O and the sum are scaled, only where it has grown by more than
                // 2^kFewLazy: weights up to 2^24 instead of 1 cost a floating sum nothing.
                if (__any_sync(0xffffffffu, top > m + kFewLazy)) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float to = fmaxf(m, top), f = to == -INFINITY ? 1.f : fast_exp2(m - to);
                    m = to;
                    l *= f;
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        o[j][0] *= f;
                        o[j][1] *= f;
                    }
                }
                // P in bf16 for the second product: off by at most 2^-8 of itself, as the output's
                // rounding; the sum is of the unrounded values.
                uint32_t a[2];
                const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    s[nb][0] = fast_exp2(s[nb][0] - mu);
                    s[nb][1] = fast_exp2(s[nb][1] - mu);
                    l += s[nb][0] + s[nb][1];
                    a[nb] = pack_bf16(s[nb][0], s[nb][1]);
                }
                if (g + 16 > k1) {
                    // Rows of V behind the last may hold anything, and 0 * NaN is NaN: zeros.
                    for (int i = lane; i < (g + 16 - k1) * HV * 8; i += 32) {
                        const int row = r0 + 15 - i / (HV * 8), c = i % (HV * 8);
                        *reinterpret_cast<uint4 *>(ring + st * STAGE + OPER + (c >> 3) * kHvHalf + swz128(row, c & 7)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                // Infinities and NaN among the V of the block's own tokens, which earlier ones must not see
                // (0 * inf is NaN), are left out of the product and added by scalars where a row sees them.
                const int last = min(16, k1 - g);
                const uint8_t *v = ring + st * STAGE + OPER;
                const bool odd = p.n > 1 && g + 16 > len - p.n + 1 && few_not_finite<HV>(v, kHvHalf, r0, last, lane);
                if (odd) {
                    for (int x = 0; x < last; ++x) {
                        const float even = x < 8 ? s[0][0] : s[1][0], next = x < 8 ? s[0][1] : s[1][1];
                        const float w = __shfl_sync(0xffffffffu, x & 1 ? next : even, (lane & ~3) | ((x & 7) >> 1));
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            uint32_t z =
                                *reinterpret_cast<const uint32_t *>(v + (j >> 3) * kHvHalf + swz128(r0 + x, j & 7) + 4 * lq);
                            z &= few_odd_bits(z);
                            if (z && g + x < see) {
                                o[j][0] = fmaf(w, __uint_as_float(z << 16), o[j][0]);
                                o[j][1] = fmaf(w, __uint_as_float(z & 0xffff0000u), o[j][1]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < NB; j += 2) {
                    uint32_t f0, f1, f2, f3;
                    ldsm_x4_trans(((vt + v_lane) ^ ((j & 7) * 16)) + (j >> 3) * kHvHalf, f0, f1, f2, f3);
                    if (odd) {
                        f0 &= ~few_odd_bits(f0);
                        f1 &= ~few_odd_bits(f1);
                        f2 &= ~few_odd_bits(f2);
                        f3 &= ~few_odd_bits(f3);
                    }
                    few_mma<1>(o[j], a, f0, f1);
                    few_mma<1>(o[j + 1], a, f2, f3);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (lq == 0) wstat[warp][lr] = make_float2(m, l);
    }
    __syncthreads();
    // The warps' maxima and sums, the CTA's, the cluster's.
    auto join = [](float2 &s, float2 x) {
        const float mx = fmaxf(s.x, x.x), mu = mx == -INFINITY ? 0.f : mx;
        s = make_float2(mx, s.y * fast_exp2(s.x - mu) + x.y * fast_exp2(x.x - mu));
    };
    if (tid < kHvRows) {
        float2 s = make_float2(-INFINITY, 0.f);
        for (int w = 0; w < kHvWarps; ++w) join(s, wstat[w][tid]);
        cstat[tid] = s;
    }
    if (C > 1) few_cluster_sync();
    if (tid < kHvRows) {
        float2 s = make_float2(-INFINITY, 0.f);
        if (C > 1)
            for (uint32_t c = 0; c < C; ++c) join(s, few_ld2(few_at(&cstat[tid], c)));
        else
            s = cstat[tid];
        // A sum of zero: a row that sees nothing.  One of NaN stays so, in every weight that it has a part in.
        all[tid] = make_float2(s.x == -INFINITY ? 0.f : s.x, s.y == 0.f ? 0.f : 1.f / s.y);
    }
    __syncthreads();
    // Every row's weight, summed over the query rows in their order; the tokens' own rows apart, over the query rows
    // that see them: an earlier token's probability there is 0, but not if its sum is NaN.
    const int own = max(k0, len - p.n), shared = min(k1, own);
    const int first_pos = p.next_pos ? ld_dep(p.next_pos + b) : 0;
    auto grown = [&](int j, int from) {
        float sum = 0.f;
        for (int r = from; r < p.R; ++r)
            sum = fmaf(fast_exp2(scores[(long long)r * p.stride + j - k0] - all[r].x), all[r].y, sum);
        return sum;
    };
    constexpr int KEYS = 8;                             // a thread's keys whose old weights are loaded together
    for (int j0 = k0 + tid; j0 < shared; j0 += KEYS * kHvThreads) {
        float old[KEYS];
#pragma unroll
        for (int x = 0; x < KEYS; ++x) {
            const int j = j0 + x * kHvThreads;
            old[x] = j < shared ? __ldcg(p.weight + row0 + j) : 0.f;
        }
#pragma unroll
        for (int x = 0; x < KEYS; ++x) {
            const int j = j0 + x * kHvThreads;
            if (j >= shared) break;
            p.weight[row0 + j] = old[x] + grown(j, 0);
        }
    }
    for (int j = own + tid; j < k1; j += kHvThreads) {
        const float old = p.next_pos ? 0.f : __ldcg(p.weight + row0 + j);
        p.weight[row0 + j] = old + grown(j, (j - (len - p.n)) * p.G);
        if (p.next_pos) p.pos[row0 + j] = first_pos + j - (len - p.n);
    }
    // O of the warps, in the softmax's own scale.
    float *osum = reinterpret_cast<float *>(ring);      // [kHvWarps][R][OROW]
    if (warp < kHvWarps && lr < p.R) {
        const float f = m == -INFINITY ? 0.f : fast_exp2(m - all[lr].x) * all[lr].y;
        float *to = osum + (warp * p.R + lr) * OROW + 2 * lq;
#pragma unroll
        for (int j = 0; j < NB; ++j) *reinterpret_cast<float2 *>(to + j * 8) = make_float2(o[j][0] * f, o[j][1] * f);
    }
    // Summed over the warps and the CTAs, each of which has a share of the channels.
    if (C > 1) few_cluster_sync();
    else __syncthreads();
    const int vecs = p.R * (D / 4), share = (vecs + (int)C - 1) / (int)C;
    for (int i = (int)rank * share + tid; i < min(vecs, (int)(rank + 1) * share); i += kHvThreads) {
        const int r = i / (D / 4), c4 = i - r * (D / 4), t = r / p.G, at = r * OROW + c4 * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t c = 0; c < C; ++c) {
            const uint32_t base = few_at(osum + at, c);
#pragma unroll
            for (int w = 0; w < kHvWarps; ++w) {
                const float4 x = C == 1 ? *reinterpret_cast<const float4 *>(osum + w * p.R * OROW + at)
                                        : few_ld4(base + (uint32_t)(w * p.R * OROW) * 4);
                s.x += x.x;
                s.y += x.y;
                s.z += x.z;
                s.w += x.w;
            }
        }
        *reinterpret_cast<uint2 *>(p.out + (((long long)b * p.n + t) * p.H_q + h * p.G + (r - t * p.G)) * D + c4 * 4) =
            make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
    if (C > 1) few_cluster_sync();                      // no CTA ends while another reads its O
}

// ----------------------------------------------------------------- host side
constexpr int kHvScores = 40 * 1024;     // scores of a CTA that stay in shared memory at most
constexpr int kHvStatic = 8 * 1024;      // room for the query rows and what else is not sized by the call

// The time of a launch by clusters of C, in us, as far as it hangs on C: CTAs come in waves, two an
// SM, the last one part full; a CTA's tiles take `each`, HBM's share of an SM, and `way` goes by
// before and after them.
double heavy_time(long long pairs, int cap, int C, int keys, double each, double way) {
    const double waves = pairs * C / (2.0 * magicdec_host::sm_count()) + 0.5;
    return (waves > 1 ? waves : 1) * ((((long long)cap + C - 1) / C + keys - 1) / keys * each + way);
}

template <int D>
static magicdec_status launch_heavy_t(const CUtensorMap (&tm)[4], const HeavyParams &p, int C, size_t smem, cudaStream_t st) {
    if (!magicdec_host::allow_smem_once<heavy_attn_kernel<D>>(magicdec_host::max_smem_optin() / 2))
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
    if (cudaLaunchKernelEx(&cfg, heavy_attn_kernel<D>, tm[0], tm[1], tm[2], tm[3], p) != cudaSuccess)
        return MAGICDEC_ERR_CUDA;
    return magicdec_host::launch_status();
}

magicdec_status launch_heavy_attn(int B, int H_q, int H_kv, int D, int cap, int n, const uint16_t *q,
                                  const uint16_t *k, const uint16_t *v, const int32_t *len, const int32_t *next_pos,
                                  float *weight, int32_t *pos, uint16_t *out, cudaStream_t st) {
    HeavyParams p{};
    p.q = q;
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
    // Clusters of 1 to 8 whose scores fit, by the time they should take.  128 sequences of 2053 rows, 8
    // heads, R = 4, clusters of 1, 2, 4 and 8: 184, 195, 216 and 331 us; 16 of up to 12,001 in
    // clusters of 8, R = 5: 90 us, and on tcgen05, in clusters of 4, 103.
    int C = 0;
    double least = 0;
    for (int c = 1; p.R <= kHvRows && c <= 8; c *= 2) {
        const long long per = (((long long)cap + c - 1) / c + 15) / 16 * 16;
        // 8 floats more than a multiple of 32: neighbouring rows' scores lie in other banks.
        const long long stride = (per + 23) / 32 * 32 + 8;
        if (stride * p.R * 4 > kHvScores) continue;
        const double t = heavy_time((long long)B * H_kv, cap, c, kHvKeys, D == 128 ? 1.4 : 0.8, 6.0);
        if (C == 0 || t < least) {
            least = t;
            C = c;
            p.stride = (int)stride;
        }
    }
    if (C == 0) return launch_heavy_tc(p, D, k, v, st);
    // The ring takes what two CTAs an SM leave beside the scores, in the end the warps' O.
    const int stage = D / 64 * 2 * kHvHalf, scores = p.stride * p.R * 4;
    const int tiles = (((cap + C - 1) / C + 15) / 16 * 16 + kHvKeys - 1) / kHvKeys;
    p.stages = (magicdec_host::max_smem_optin() / 2 - kHvStatic - scores) / stage;
    if (p.stages > kHvStages) p.stages = kHvStages;
    if (p.stages > tiles) p.stages = tiles;
    static_assert(kHvWarps * kHvRows * (64 + 8) * 4 <= 2 * kHvHalf, "a stage has room for the warps' O");
    // (channels, rows, heads, sequences), boxes of 64 channels of a stage's rows, and of 16 for its end.
    CUtensorMap tm[4];
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)cap, (uint64_t)H_kv, (uint64_t)B};
    const uint64_t row = (uint64_t)D * 2, strides[3] = {row, cap * row, (uint64_t)H_kv * cap * row};
    const uint32_t box[4] = {64, kHvKeys, 1, 1}, box16[4] = {64, 16, 1, 1};
    if (!magicdec_host::encode_tmap_bf16_4d(&tm[0], k, dims, strides, box) ||
        !magicdec_host::encode_tmap_bf16_4d(&tm[1], v, dims, strides, box) ||
        !magicdec_host::encode_tmap_bf16_4d(&tm[2], k, dims, strides, box16) ||
        !magicdec_host::encode_tmap_bf16_4d(&tm[3], v, dims, strides, box16))
        return MAGICDEC_ERR_CUDA;
    const size_t smem = (size_t)p.stages * stage + scores;
    return D == 128 ? launch_heavy_t<128>(tm, p, C, smem, st) : launch_heavy_t<64>(tm, p, C, smem, st);
}

// ------------------------------------------------------------------ eviction
// Of a (layer, sequence, KV head)'s len rows the `budget` with the largest key stay.  A row's
// key is its weight, infinity for the protected ones; equal keys: the smaller position stays, then
// the smaller row.  Seen from the other end, the E = len - budget least go.  Rows that stay behind
// the budget then fill the holes below it, in ascending order of both, so that a step that evicts E
// rows moves at most E.
// Bound: 8 bytes a row (weight, position) from HBM; in practice the chain of loads, searches and
// moves of a (layer, sequence, KV head), which only others can cover.  So one warp takes it where its
// keys are few (kEvWarpRows; keys in shared memory, reductions and lists inside the warp, no barrier of
// a CTA) and few rows can go or there are many others, else 8 warps.  A warp from which few rows go ranks the few keys that lie
// below a bound; a CTA finds the border digit by digit of 8 bits, with counts of the keys of every
// digit, until a count is met.  Positions of ties take the keys' place and are searched likewise.
// 32 layers of 16 sequences, 8 heads, up to 1029 rows of which 5 go: 15.5 us; with a CTA each 87.
constexpr int kEvThreads = 256;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvWarpRows = 2048;        // rows of a warp's own
constexpr int kEvMoves = 64;             // moves listed at a time, a warp
constexpr int kEvTake = 16;              // rows to go that are taken one after another

struct EvictParams {
    uint4 *kc, *vc;
    float *weight;
    int32_t *pos;
    const int32_t *len, *seq_len;
    int32_t *len_out;
    int *err;
    int B, H_kv, cap, vecs, budget, n_sink, n_recent;
    long long items;                     // layers * B * H_kv
    int keep;                            // rows whose keys fit shared memory, a multiple of 4
    int wide;                            // rows of weights and positions begin at 16 bytes
};

// A thread's rows: 4 neighbours of every 4 T, so that keys are written and searched 16 bytes at a time.
// Order of fp32 as unsigned integers; both zeros are one.
__device__ __forceinline__ uint32_t ev_key(float w) {
    const uint32_t x = __float_as_uint(w + 0.f);
    return x & 0x80000000u ? ~x : x | 0x80000000u;
}

// NW: warps of an item (1: a CTA has kEvWarps items).
template <int NW>
__global__ void __launch_bounds__(kEvThreads) heavy_evict_kernel(const EvictParams p) {
    constexpr int T = NW * 32, LIST = kEvMoves * NW;
    extern __shared__ __align__(16) uint32_t shared[];
    __shared__ int lists[2 * kEvMoves * kEvWarps];
    __shared__ uint2 xch[2][kEvWarps];
    __shared__ int hist[kEvThreads], digit[2];
    const int tid = threadIdx.x % T, warp = tid >> 5, lane = tid & 31, sub = threadIdx.x / T;
    const int words = (p.cap + 31) / 32;
    const int words4 = (words + 3) / 4 * 4;
    // Keys, a bit a row that goes, and, of rows whose keys are here, one a row that is alike.
    uint32_t *kept = shared + sub * (p.keep + words4 + (p.keep + 127) / 128 * 4), *gone = kept + p.keep, *ties = gone + words4;
    int *src = lists + sub * 2 * LIST, *dst = src + LIST;
    pdl_trigger();
    pdl_wait();
    const long long item = (long long)blockIdx.x * (kEvWarps / NW) + sub;
    if (item >= p.items) return;
    const int b = (int)(item / p.H_kv % p.B);
    const int len0 = checked(ld_dep(p.len + b), 0, p.cap, p.err);
    const int len = len0 < 0 ? 0 : (len0 > p.cap ? p.cap : len0);
    if (item < (long long)p.B * p.H_kv && item % p.H_kv == 0 && tid == 0) p.len_out[b] = min(len, p.budget);
    const int E = len - p.budget;                            // rows to go
    if (E <= 0) return;
    const long long row0 = item * p.cap;
    float *weight = p.weight + row0;
    int32_t *pos = p.pos + row0;
    const long long recent = (long long)ld_dep(p.seq_len + b) - p.n_recent;
    auto sync = [] {
        if (NW == 1) __syncwarp();
        else __syncthreads();
    };
    auto key_of = [&](int at, float w) { return at < p.n_sink || at >= recent ? ev_key(INFINITY) : ev_key(w); };
    auto weight_at = [&](int j) { return __uint_as_float((uint32_t)ld_dep(reinterpret_cast<const int *>(weight) + j)); };
    // Keys, those of 16 rows of a thread under way at a time; behind the last one the largest value.
    const int mine = min(len, p.keep);
    auto place_of = [](int at) { return ~((uint32_t)at ^ 0x80000000u); };
    uint32_t low = ~0u;                                      // this thread's least key
    for (int j0 = 4 * tid; j0 < mine; j0 += 16 * T) {
        int4 at[4];
        float4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * 4 * T;
            if (j + 3 < mine && p.wide) {
                const uint4 x = ld_dep_u4(reinterpret_cast<const uint4 *>(pos + j));
                at[k] = make_int4(x.x, x.y, x.z, x.w);
                w[k] = ld_dep_f4(reinterpret_cast<const float4 *>(weight + j));
            } else if (j < mine) {
                at[k] = make_int4(ld_dep(pos + j), j + 1 < mine ? ld_dep(pos + j + 1) : 0,
                                  j + 2 < mine ? ld_dep(pos + j + 2) : 0, j + 3 < mine ? ld_dep(pos + j + 3) : 0);
                w[k] = make_float4(weight_at(j), j + 1 < mine ? weight_at(j + 1) : 0.f,
                                   j + 2 < mine ? weight_at(j + 2) : 0.f, j + 3 < mine ? weight_at(j + 3) : 0.f);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * 4 * T;
            if (j < mine) {
                const uint4 x =
                    make_uint4(key_of(at[k].x, w[k].x), j + 1 < mine ? key_of(at[k].y, w[k].y) : ~0u,
                               j + 2 < mine ? key_of(at[k].z, w[k].z) : ~0u, j + 3 < mine ? key_of(at[k].w, w[k].w) : ~0u);
                *reinterpret_cast<uint4 *>(kept + j) = x;
                low = min(min(low, min(x.x, x.y)), min(x.z, x.w));
            }
        }
    }
    sync();
    auto key = [&](int j) { return j < p.keep ? kept[j] : key_of(ld_dep(pos + j), weight_at(j)); };

    // The listed rows' moves: K, V, weight and position of row src[i] to row dst[i].
    const int per = 2 * p.vecs, rows = T / per, c = tid % per;   // threads of a row of K and V
    uint4 *base = (c < p.vecs ? p.kc + c : p.vc + (c - p.vecs)) + row0 * p.vecs;
    auto move_rows = [&](int moves) {
        constexpr int AHEAD = 6;                             // rows under way
        for (int i = tid; i < moves; i += T) {
            const float w = weight_at(src[i]);
            const int at = ld_dep(pos + src[i]);
            weight[dst[i]] = w;
            pos[dst[i]] = at;
        }
        for (int i = tid / per; i < moves; i += AHEAD * rows) {
            uint4 x[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i + k * rows < moves) x[k] = ld_dep_u4(base + (long long)src[i + k * rows] * p.vecs);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i + k * rows < moves) base[(long long)dst[i + k * rows] * p.vecs] = x[k];
        }
    };
    if (NW == 1 && E <= kEvTake && len <= p.keep) {
        // Few rows to go.  The E-th least of the lanes' least keys bounds the E-th least key from above;
        // hardly more than E keys lie at or below it, and are ranked by comparing each with all.
        uint32_t rest = low, bound = 0;
        for (int k = 0; k < E; ++k) {
            bound = __reduce_min_sync(0xffffffffu, rest);
            if (lane == __ffs(__ballot_sync(0xffffffffu, rest == bound)) - 1) rest = ~0u;
        }
        const bool alike = __popc(__ballot_sync(0xffffffffu, low == bound)) > kEvTake;   // rather many rows are
        // Lists the rows whose keys lie at or below a limit, the first 32; returns how many there are.
        auto collect = [&](uint32_t limit) {
            int found = 0;
            for (int j0 = 0; j0 < len; j0 += 128) {
                const int j = j0 + 4 * lane;
                const uint4 x = j < len ? *reinterpret_cast<const uint4 *>(kept + j) : make_uint4(~0u, ~0u, ~0u, ~0u);
                if (!__any_sync(0xffffffffu, min(min(x.x, x.y), min(x.z, x.w)) <= limit)) continue;
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool in = j + k < len && y[k] <= limit;
                    const unsigned m = __ballot_sync(0xffffffffu, in);
                    const int to = found + __popc(m & ((1u << lane) - 1u));
                    if (in && to < 32) src[to] = j + k;
                    found += __popc(m);
                }
            }
            __syncwarp();
            return found;
        };
        int found = alike ? 33 : collect(bound), row = -1;
        bool go = false, known = found <= 32;
        if (known) {
            const bool in = lane < found;
            row = in ? src[lane] : -1;
            const uint32_t x = in ? kept[row] : ~0u;
            const unsigned same = __match_any_sync(0xffffffffu, x);
            uint32_t y = 0;                                  // positions only where weights are alike
            if (__any_sync(0xffffffffu, in && (same & (same - 1)))) y = in ? place_of(ld_dep(pos + row)) : 0;
            int rank = 0;
            for (int k = 0; k < found; ++k) {
                const uint32_t x2 = __shfl_sync(0xffffffffu, x, k), y2 = __shfl_sync(0xffffffffu, y, k);
                const int row2 = __shfl_sync(0xffffffffu, row, k);
                rank += x2 < x || (x2 == x && (y2 < y || (y2 == y && row2 > row)));
            }
            go = in && rank < E;
        } else if (bound > 0 && bound < ev_key(INFINITY) && (found = collect(bound - 1)) < E) {
            // Fewer than E lie below the bound, so that it is the E-th least key, which many rows have: those
            // with the largest positions go, taken one after another, of equal ones the highest row.
            // Positions take the keys' place, 0 that of other rows'; such a row is not protected, so
            // that its position is not negative.
            uint32_t best = 0;                               // of this thread's rows
            int at = -1;
            for (int j0 = 4 * lane; j0 < len; j0 += 16 * T) {
                uint4 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = j0 + k * 4 * T;
                    if (j + 3 < len && p.wide) w[k] = ld_dep_u4(reinterpret_cast<const uint4 *>(pos + j));
                    else if (j < len)
                        w[k] = make_uint4(ld_dep(pos + j), j + 1 < len ? ld_dep(pos + j + 1) : 0,
                                          j + 2 < len ? ld_dep(pos + j + 2) : 0, j + 3 < len ? ld_dep(pos + j + 3) : 0);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = j0 + k * 4 * T;
                    if (j >= len) break;
                    const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                    uint32_t y[4] = {x.x, x.y, x.z, x.w};
                    const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = y[e] == bound ? v[e] | 0x80000000u : 0u;
                        if (y[e] && y[e] >= best) {
                            best = y[e];
                            at = j + e;
                        }
                    }
                    *reinterpret_cast<uint4 *>(kept + j) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
            for (; found < E; ++found) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, best);
                const int last = __reduce_max_sync(0xffffffffu, best == top ? at : -1);
                if (lane == 0) src[found] = last;
                if (at == last) {
                    kept[last] = 0;
                    best = 0;
                    at = -1;
                    for (int j = 4 * lane; j < len; j += 4 * T) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (y[e] && y[e] >= best) {
                                best = y[e];
                                at = j + e;
                            }
                    }
                }
            }
            __syncwarp();
            known = true;
            go = lane < E;
            row = go ? src[lane] : -1;
        }
        if (known) {
            const bool hole = go && row < p.budget;
            // Of the E rows from the budget on, those that do not go, ascending, into the holes, ascending.
            bool stay = lane < E;
            int before = 0;
            for (unsigned m = __ballot_sync(0xffffffffu, go); m; m &= m - 1) {
                const int row2 = __shfl_sync(0xffffffffu, row, __ffs(m) - 1);
                stay = stay && row2 != p.budget + lane;
                before += row2 < row;
            }
            const unsigned ms = __ballot_sync(0xffffffffu, stay);
            __syncwarp();                                    // src has been read
            if (hole) dst[before] = row;
            if (stay) src[__popc(ms & ((1u << lane) - 1u))] = p.budget + lane;
            __syncwarp();
            move_rows(__popc(ms));
            return;
        }
    }

    // Sums over the item's threads.
    int turn = 0;                                            // of the two buffers, which take turns
    auto sum_all = [&](int x) {
        x = __reduce_add_sync(0xffffffffu, x);
        if (NW > 1) {
            if (lane == 0) xch[turn][warp].x = (uint32_t)x;
            sync();
            x = 0;
            for (int w = 0; w < NW; ++w) x += (int)xch[turn][w].x;
            turn ^= 1;
        }
        return x;
    };
    // The value at which the count of `part` over the rows for which `in` holds reaches `left`, which
    // becomes what is still to be taken of the rows of that value; returns how many those are.  Bit by bit,
    // for rows whose keys do not fit shared memory.
    auto border = [&](auto part, auto in, int &left, uint32_t &at) {
        at = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t top = at | (1u << bit);           // rows below it, of those that are not below `at`
            int n = 0;
            for (int j = tid; j < len; j += T) {
                if (!in(j)) continue;
                const uint32_t x = part(j);
                n += x >= at && x < top;
            }
            n = sum_all(n);
            if (n < left) {
                left -= n;
                at = top;
            }
        }
        int n = 0;
        for (int j = tid; j < len; j += T) n += in(j) && part(j) == at;
        return sum_all(n);
    };
    // The same over what shared memory holds of the rows, or of those with a bit in `mask`, 4 rows a load,
    // and no further than to where a count is met.  A warp that takes few: the least, the next, and so on;
    // one that takes many: bit by bit from the top.  A CTA: 8 bits at a time, with counts of every digit's rows.
    auto border_kept = [&](const uint32_t *mask, uint32_t least, int &left, uint32_t &at) {
        auto real = [&](int j) {                             // which of rows j .. j + 3 there are
            const uint32_t m = j + 3 < len ? 15u : (1u << (len - j)) - 1u;
            return mask ? m & mask[j >> 5] >> (j & 31) : m;
        };
        if (NW == 1 && left > kEvTake) {
            at = 0;
            for (int bit = 31;; --bit) {
                int n = 0;                                   // rows that agree so far and have no such bit
                for (int j = 4 * tid; j < len; j += 4 * T) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                    const uint32_t y[4] = {x.x, x.y, x.z, x.w}, m = real(j);
#pragma unroll
                    for (int k = 0; k < 4; ++k) n += (m >> k & 1u) && ((y[k] ^ at) >> bit) == 0;
                }
                n = sum_all(n);
                if (n == left) {                             // all of them go
                    at |= (1u << bit) - 1u;
                    return n;
                }
                if (n < left) {
                    left -= n;
                    at |= 1u << bit;
                }
                if (bit == 0) break;
            }
            int n = 0;
            for (int j = 4 * tid; j < len; j += 4 * T) {
                const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                const uint32_t y[4] = {x.x, x.y, x.z, x.w}, m = real(j);
#pragma unroll
                for (int k = 0; k < 4; ++k) n += (m >> k & 1u) && y[k] == at;
            }
            return sum_all(n);
        } else if constexpr (NW == 1) {
            for (at = __reduce_min_sync(0xffffffffu, least);;) {
                uint32_t next = ~0u;
                int n = 0;
                for (int j = 4 * tid; j < len; j += 4 * T) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                    const uint32_t y[4] = {x.x, x.y, x.z, x.w}, m = real(j);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (m >> k & 1u) {
                            n += y[k] == at;
                            if (y[k] > at) next = min(next, y[k]);
                        }
                }
                n = sum_all(n);
                if (n >= left) return n;
                left -= n;
                at = __reduce_min_sync(0xffffffffu, next);
            }
        } else {
            at = 0;
            for (int shift = 24;; shift -= 8) {
                hist[tid] = 0;
                sync();
                const uint32_t settled = shift == 24 ? 0u : ~0u << (shift + 8);
                for (int j = 4 * tid; j < len; j += 4 * T) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                    const uint32_t y[4] = {x.x, x.y, x.z, x.w}, m = real(j);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if ((m >> k & 1u) && ((y[k] ^ at) & settled) == 0) atomicAdd(&hist[y[k] >> shift & 255], 1);
                }
                sync();
                const int c = hist[tid];
                int incl = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                if (lane == 31) xch[turn][warp].x = (uint32_t)incl;
                sync();
                for (int w = 0; w < warp; ++w) incl += (int)xch[turn][w].x;
                turn ^= 1;
                if (incl >= left && incl - c < left) {
                    digit[0] = tid;
                    digit[1] = incl - c;
                }
                sync();
                at |= (uint32_t)digit[0] << shift;
                left -= digit[1];
                const int alike = hist[digit[0]];
                sync();                                      // before the counts are cleared
                if (alike == left) at |= (1u << shift) - 1u; // all that agree so far go
                if (alike == left || shift == 0) return alike;
            }
        }
    };
    // What goes first: small weights, large positions, high rows.  One bit a row, so that weights and
    // positions may move afterwards.
    const int nw = (len + 31) / 32;
    int left = E;
    uint32_t w_at = 0, p_at = 0;                             // borders: rows at them go, too, if all do
    if (len <= p.keep) {
        const int light = border_kept(nullptr, low, left, w_at);   // rows at the border, of which `left` go
        const bool tied = light != left;
        // Bits of the rows below the border, and of those at it: 4 of a thread, 8 threads a word.
        auto mark = [&](const uint32_t *mask, uint32_t at, bool all) {
            for (int w0 = warp * 4; w0 < nw; w0 += NW * 4) {
                const int j = w0 * 32 + 4 * lane, w = w0 + lane / 8;
                uint32_t m = 0, t = 0;
                if (j < len) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                    const uint32_t in = (j + 3 < len ? 15u : (1u << (len - j)) - 1u) & (mask ? mask[w] >> (j & 31) : 15u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        m |= (uint32_t)(y[k] < at) << k;
                        t |= (uint32_t)(y[k] == at) << k;
                    }
                    m = (m | (all ? t : 0u)) & in;
                    t = all ? 0u : t & in;
                }
                m <<= j & 31;
                t <<= j & 31;
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    m |= __shfl_xor_sync(0xffffffffu, m, o);
                    t |= __shfl_xor_sync(0xffffffffu, t, o);
                }
                if (lane % 8 == 0 && w < nw) {
                    gone[w] = mask ? gone[w] | m : m;
                    ties[w] = t;
                }
            }
            sync();
        };
        mark(nullptr, w_at, !tied);
        if (tied) {
            // Positions take the keys' place.
            for (int j0 = 4 * tid; j0 < len; j0 += 16 * T) {
                uint4 at[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = j0 + k * 4 * T;
                    if (j + 3 < len && p.wide) at[k] = ld_dep_u4(reinterpret_cast<const uint4 *>(pos + j));
                    else if (j < len)
                        at[k] = make_uint4(ld_dep(pos + j), j + 1 < len ? ld_dep(pos + j + 1) : 0,
                                           j + 2 < len ? ld_dep(pos + j + 2) : 0, j + 3 < len ? ld_dep(pos + j + 3) : 0);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j0 + k * 4 * T < len)
                        *reinterpret_cast<uint4 *>(kept + j0 + k * 4 * T) =
                            make_uint4(place_of(at[k].x), place_of(at[k].y), place_of(at[k].z), place_of(at[k].w));
            }
            sync();
            uint32_t least = ~0u;                            // of this thread's rows that are alike
            for (int j = 4 * tid; NW == 1 && j < len; j += 4 * T) {
                const uint4 x = *reinterpret_cast<const uint4 *>(kept + j);
                const uint32_t m = ties[j >> 5] >> (j & 31);
                least = min(least, min(min(m & 1 ? x.x : ~0u, m & 2 ? x.y : ~0u), min(m & 4 ? x.z : ~0u, m & 8 ? x.w : ~0u)));
            }
            const int alike = border_kept(ties, least, left, p_at);
            const bool twins = alike != left;
            mark(ties, p_at, !twins);
            // Of rows alike in both the last `left` go.
            int before = 0;                                  // in the words so far, alike in all threads
            for (int w0 = 0; twins && w0 < nw; w0 += T) {
                const int w = w0 + tid;
                const unsigned t = w < nw ? ties[w] : 0;
                int incl = __popc(t);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                int at = before + incl - __popc(t);
                if (NW == 1) {
                    before += __shfl_sync(0xffffffffu, incl, 31);
                } else {
                    if (lane == 31) xch[turn][warp].x = (uint32_t)incl;
                    sync();
                    for (int x = 0; x < NW; ++x) {
                        if (x < warp) at += (int)xch[turn][x].x;
                        before += (int)xch[turn][x].x;
                    }
                    turn ^= 1;
                }
                unsigned go = t;
                for (; at < alike - left && go; ++at) go &= go - 1;      // the first ones stay
                if (go) gone[w] |= go;
            }
            sync();
        }
    } else {
        auto place = [&](int j) { return place_of(ld_dep(pos + j)); };
        const int light = border(key, [](int) { return true; }, left, w_at);
        const bool tied = light != left;
        bool twins = false;
        uint32_t r_at = 0;
        if (tied) {
            const int alike = border(place, [&](int j) { return key(j) == w_at; }, left, p_at);
            twins = alike != left;
            if (twins)
                border([](int j) { return ~(uint32_t)j; }, [&](int j) { return key(j) == w_at && place(j) == p_at; }, left,
                       r_at);
        }
        for (int w = warp; w < nw; w += NW) {
            const int j = w * 32 + lane;
            bool go = false;
            if (j < len) {
                const uint32_t x = key(j);
                go = x < w_at;
                if (x == w_at) {
                    const uint32_t y = tied ? place(j) : 0;
                    go = y < p_at || (y == p_at && (!twins || ~(uint32_t)j <= r_at));
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, go);
            if (lane == 0) gone[w] = m;
        }
        sync();
    }
    // Holes below the budget and the rows to fill them, listed LIST at a time.
    for (int done = 0, holes = 1; done < holes; done += LIST) {
        holes = 0;
        int late = 0;                                        // found so far, alike in all threads
        for (int w0 = 0; w0 < nw; w0 += T) {                 // a thread has a word
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
            int ah = holes + ih - ch, as = late + is - cs;
            if (NW == 1) {
                holes += __shfl_sync(0xffffffffu, ih, 31);
                late += __shfl_sync(0xffffffffu, is, 31);
            } else {
                if (lane == 31) xch[turn][warp] = make_uint2(ih, is);
                sync();
                for (int x = 0; x < NW; ++x) {
                    const uint2 y = xch[turn][x];
                    if (x < warp) {
                        ah += (int)y.x;
                        as += (int)y.y;
                    }
                    holes += (int)y.x;
                    late += (int)y.y;
                }
                turn ^= 1;
            }
            for (; hole; hole &= hole - 1, ++ah)
                if (ah >= done && ah < done + LIST) dst[ah - done] = w * 32 + __ffs(hole) - 1;
            for (; stay; stay &= stay - 1, ++as)
                if (as >= done && as < done + LIST) src[as - done] = w * 32 + __ffs(stay) - 1;
        }
        sync();
        const int moves = min(holes - done, LIST);           // there are as many holes as rows to fill them
        move_rows(moves);
        sync();
    }
}

constexpr int kEvKeep = 24 * 1024;       // keys in shared memory at most
constexpr int kEvMaxRows = 1 << 20;

template <int NW>
static magicdec_status launch_evict_t(EvictParams &p, cudaStream_t st) {
    const int sets = kEvWarps / NW, smem = sets * (p.keep + ((p.cap + 127) / 128 + (p.keep + 127) / 128) * 4) * 4;
    if (!magicdec_host::allow_smem_once<heavy_evict_kernel<NW>>(200 * 1024)) return MAGICDEC_ERR_CUDA;
    return magicdec_host::launch_pdl(heavy_evict_kernel<NW>, dim3((unsigned)((p.items + sets - 1) / sets)),
                                     dim3(kEvThreads), (size_t)smem, st, p);
}

magicdec_status launch_heavy_evict(int layers, int B, int H_kv, int D, int cap, const int32_t *len,
                                   const int32_t *seq_len, int budget, int n_sink, int n_recent, uint16_t *kc,
                                   uint16_t *vc, float *weight, int32_t *pos, int32_t *len_out, cudaStream_t st) {
    EvictParams p{};
    p.items = (long long)layers * B * H_kv;
    if (cap > kEvMaxRows || p.items > INT_MAX) return MAGICDEC_ERR_UNSUPPORTED;
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
    p.wide = cap % 4 == 0 && magicdec_host::aligned16(weight) && magicdec_host::aligned16(pos);
    p.keep = cap < kEvKeep ? (cap + 3) / 4 * 4 : cap <= kEvMaxRows / 2 ? kEvKeep : kEvKeep / 2;
    // A warp an item where few rows can go, as it moves but a few at a time, and where there are so many items
    // that warps of other ones cover that.  Warps and CTAs, d = 128: 9728 items of 63 rows of which 17 go 40 and
    // 113 us, of 1029 of which 5 go 38 and 111, of 1200 of which 800 go 496 and 470; 2432 of 1029 19 and 36, of 2048
    // of which 1024 go 298 and 232; 1216 of 63 17 and 21, of 2048 191 and 128; 608 of 63 17 and 15.
    const long long many = (cap <= 256 ? 8 : 16) * magicdec_host::sm_count();
    return cap <= kEvWarpRows && (cap - budget <= kEvTake || p.items >= many) ? launch_evict_t<1>(p, st)
                                                                              : launch_evict_t<kEvWarps>(p, st);
}

}  // namespace magicdec
