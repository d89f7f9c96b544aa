// prefix_own.cu -- attention of up to 32 query rows of a KV head over a sequence's own slots behind
// a shared prefix, joined with the prefix's parts (sm_103a).
//
// A cluster of C CTAs takes a (sequence, KV head), each a stretch of its slots; at the end the
// CTAs exchange (max, sum), sum the warps' O in a fixed order, add the parts that
// tree_attn_kernel left of the prefix, and write the output: no parts of their own go through
// memory.  Bound: HBM, 4 d bytes a slot and KV head.  Many small CTAs, two or more an SM, so that
// one's way in and out runs beside another's keys: as entries of tree_attn_kernel's list, a CTA an
// SM with one entry after another, each took some 8 us (1024 of 1 slot 60 us, of 500 slots 131 us).
//
// All warps fill the ring, 16 bytes a thread from any rows of the pool (page sizes need no
// care, rows that hold nothing are filled with zeros), and take 16 keys of a stage of 64
// through ldmatrix and mma.sync, with more than 16 query rows two warps the same keys.
//
// The kernel before it in the stream is tree_attn_kernel, which lets it begin when all of
// its CTAs have waited for what was before them: everything but the prefixes' parts is there, and
// only these are waited for, behind the own slots (one token of 8 sequences behind 4k: 19 us, 26 with
// the wait in front; of 128 behind 32k: 127 and 149).
#include <climits>

#include "few_rows.cuh"
#include "prefix.cuh"

namespace magicdec {

constexpr int kPoKeys = 64;              // keys of a stage
constexpr int kPoHalf = kPoKeys * 128;   // bytes of 64 channels of them
constexpr int kPoMaxCluster = 8;
constexpr int kPoParts = 32;             // items' parts of a thread that are worth a CTA more

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ROWS: query rows of a warp's tile that can be real, 8 or 16; MT: row tiles (a warp has one).
template <int D, int ROWS, int MT>
struct PoShape {
    static constexpr int WARPS = 4 * MT, NT = WARPS * 32;
    static constexpr int HV = D / 64, OPER = HV * kPoHalf, STAGE = 2 * OPER;
    // CTAs an SM, and stages of a ring.  Three with 2 stages or two with 3 (128 sequences of 500 slots, 16
    // rows: 69 and 79 us; 8 rows: 66 and 67, but 8 sequences 22 and 19; 32 rows have registers for two).
    static constexpr int PER_SM = ROWS == 16 && MT == 1 ? 3 : 2;
    static constexpr int STAGES = (PER_SM == 3 ? 2 : 3) * (D == 128 ? 1 : 2);
    static constexpr int QHALF = MT * ROWS * 128;
    static constexpr int BYTES = STAGES * STAGE + HV * QHALF;
    static constexpr int OROW = D + 8;                  // floats of a row of O: rows lie in other banks
    static_assert(4 * (D / 4) <= NT, "4 rows are an item a thread, or less");
    static_assert(4 * MT * ROWS * OROW * 4 <= STAGES * STAGE, "the warps' O take the ring's place");
};

// A number that a generic lambda takes as a compile-time constant.
template <int N>
struct Items {
    static constexpr int value = N;
};

template <int D, int ROWS, int MT>
__global__ void __launch_bounds__(PoShape<D, ROWS, MT>::NT, PoShape<D, ROWS, MT>::PER_SM)
    prefix_own_kernel(const PreOwn p) {
    using L = PoShape<D, ROWS, MT>;
    constexpr int NT = L::NT, OPER = L::OPER, STAGE = L::STAGE, NST = L::STAGES, QHALF = L::QHALF, OROW = L::OROW;
    constexpr int KS = D / 16, NB = D / 8, HR = ROWS / 8, VR = D / 8;   // VR: 16-byte words of a row
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem, *qs = smem + NST * STAGE;
    __shared__ long long rows_at[8][kPoKeys];           // of a tile's keys: element of the pool, or -1
    __shared__ int par[32];
    __shared__ uint32_t sees[32];                       // of a node's slots: itself and its ancestors
    __shared__ float2 wstat[L::WARPS][16];              // of a warp's rows: (max, sum)
    __shared__ float2 cstat[32];                        // of this CTA
    __shared__ float2 both[32];                         // of this CTA and of the prefix's parts that it took
    __shared__ RowParts parts_of[32];                   // of the prefix
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lq = lane & 3, lr = lane >> 2;
    const int b = blockIdx.z, h = blockIdx.y, n = p.pre.n, G = p.pre.G, R = n * G;
    const uint32_t rank = few_rank(), C = few_ctas();
    const float sl = p.scale_log2;
    pdl_trigger();
    // Loads that wait for no others go out together: the query rows (row i * G + g: node i, head g of the
    // group), the parents, the lengths; then the pages of the first tiles, all at once.
    constexpr int QV = (MT * ROWS * VR + NT - 1) / NT;  // 16-byte words of the query rows a thread has
    uint4 qv[QV];
#pragma unroll
    for (int x = 0; x < QV; ++x) {
        const int r = (x * NT + tid) / VR, c = (x * NT + tid) % VR, i = r / G;
        const uint16_t *src = p.q + (((long long)b * n + i) * p.H_q + h * G + (r - i * G)) * D + c * 8;
        qv[x] = r < R ? __ldcg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0, 0, 0, 0);
    }
    const int parent = p.parent && tid < n ? ld_dep(p.parent + (long long)b * n + tid) : tid - 1;
    const int cap = p.page_size * p.max_pages;
    const int len_in = ld_dep(p.len + b), nodes_in = p.n_nodes ? ld_dep(p.n_nodes + b) : n;
    const int len = pre_clamp(checked(len_in, 0, cap, p.err), cap), nodes = pre_clamp(checked(nodes_in, 0, n, p.err), n);
    const int total = nodes ? (nodes > cap - len ? cap : len + nodes) : 0;
    // This CTA's keys: [k0, k1), in groups of 16.
    const int per = ((total + (int)C - 1) / (int)C + 15) & ~15;
    const int k0 = min(total, (int)rank * per), k1 = min(total, k0 + per), tiles = (k1 - k0 + kPoKeys - 1) / kPoKeys;
    // Where a key lies; one outside the pool is zeros.  A page is asked for before a tile's products and
    // its number used behind them.  (Unsigned, as keys of tiles behind the last one may pass 2^31.)
    const int32_t *table = p.table + (long long)b * p.max_pages;
    auto key_of = [&](int t, int at) { return (uint32_t)k0 + (uint32_t)t * kPoKeys + at; };
    auto ask = [&](int t, int at) {
        const uint32_t key = key_of(t, at);
        return key < (uint32_t)k1 ? ld_dep(table + key / (uint32_t)p.page_size) : -1;
    };
    auto look_up = [&](int t, int at, int page) {
        const uint32_t key = key_of(t, at);
        long long row = -1;
        if (key < (uint32_t)k1) {
            if (page < 0 || page >= p.n_pages) raise_error(p.err, kErrPage);
            else row = (((long long)page * p.page_size + key % (uint32_t)p.page_size) * p.pre.H_kv + h) * D;
        }
        rows_at[t & 7][at] = row;
    };
    auto load = [&](int t) {
        if (t < tiles) {
            const uint32_t to = smem_u32(ring + t % NST * STAGE);
#pragma unroll
            for (int x = 0; x < kPoKeys * VR; x += NT) {
                const int r = (x + tid) / VR, c = (x + tid) % VR;
                const long long at = rows_at[t & 7][r];
                const long long from = (at < 0 ? 0 : at) + c * 8;
                const uint32_t dst = to + (uint32_t)(c >> 3) * kPoHalf + swz128(r, c & 7);
                copy16(dst, p.k + from, at >= 0);
                copy16(dst + OPER, p.v + from, at >= 0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    constexpr int FIRST = (NST * kPoKeys + NT - 1) / NT;
    int pages[FIRST];
#pragma unroll
    for (int x = 0; x < FIRST; ++x) pages[x] = ask((x * NT + tid) / kPoKeys, (x * NT + tid) % kPoKeys);
#pragma unroll
    for (int x = 0; x < QV; ++x) {
        const int r = (x * NT + tid) / VR, c = (x * NT + tid) % VR;
        if (r < MT * ROWS) *reinterpret_cast<uint4 *>(qs + (c >> 3) * QHALF + swz128(r, c & 7)) = qv[x];
    }
    if (tid < n) par[tid] = checked(parent, INT_MIN, tid - 1, p.err);
#pragma unroll
    for (int x = 0; x < FIRST; ++x) look_up((x * NT + tid) / kPoKeys, (x * NT + tid) % kPoKeys, pages[x]);
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t + 1 < NST; ++t) load(t);
    if (tid < n) {
        uint32_t m = 0;
        for (int a = tid; a >= 0;) {
            m |= 1u << a;
            const int q = par[a];
            a = q < a ? q : -1;
        }
        sees[tid] = m;
    }
    __syncthreads();

    const int mt = MT == 1 ? 0 : warp % MT, kw = warp / MT;
    uint32_t qf[HR == 1 ? KS : 1][2 * HR];
    float o[NB][2 * HR], m[HR], l[HR];
    uint32_t anc[HR];
#pragma unroll
    for (int e = 0; e < HR; ++e) {
        const int r = mt * 16 + lr + 8 * e;
        anc[e] = r < R ? sees[r / G] : 0u;
        m[e] = -INFINITY;
        l[e] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 2 * HR; ++e) o[j][e] = 0.f;
    // The queries' fragments: kept with 8 rows, else from shared memory for every 16 keys (they would
    // take the registers of a second CTA on the SM).
    const uint32_t q_lane = smem_u32(qs) + (uint32_t)mt * 2048 + (HR == 2 ? swz128(lane & 15, lane >> 4) : swz128(lane & 7, lane >> 3));
    if constexpr (HR == 1)
#pragma unroll
        for (int c = 0; c < KS; c += 2)
            ldsm_x4((q_lane ^ ((c & 3) * 32)) + (c >> 2) * QHALF, qf[c][0], qf[c][1], qf[c + 1][0], qf[c + 1][1]);
    // A lane's address in a K tile, and in a V tile: 16-byte chunk c of its row is at c * 16 away from
    // chunk 0 in the sense of an exclusive or (8 chunks a half).
    const int x4 = lane >> 3, r0 = 16 * kw;
    const uint32_t k_lane = swz128(r0 + (x4 >> 1) * 8 + (lane & 7), x4 & 1);
    const uint32_t v_lane = swz128(r0 + (x4 & 1) * 8 + (lane & 7), x4 >> 1);
    for (int t = 0; t < tiles; ++t) {
        copies_wait<NST - 2>();
        __syncthreads();                                // tile t is there, and all are done with tile t - 1
        const int page = tid < kPoKeys ? ask(t + NST, tid) : -1;
        load(t + NST - 1);
        const uint32_t kt = smem_u32(ring + t % NST * STAGE), vt = kt + OPER;
        const int g = k0 + t * kPoKeys + r0;
        if (g >= k1) {                                  // nothing for this warp
            if (tid < kPoKeys) look_up(t + NST, tid, page);
            continue;
        }
        // Two chains of products a score, so that half as many wait for one another.
        float s[2][2 * HR], s2[2][2 * HR];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int e = 0; e < 2 * HR; ++e) s[nb][e] = s2[nb][e] = 0.f;
#pragma unroll
        for (int c = 0; c < KS; ++c) {
            uint32_t f0, f1, f2, f3;
            ldsm_x4(((kt + k_lane) ^ ((c & 3) * 32)) + (c >> 2) * kPoHalf, f0, f1, f2, f3);
            uint32_t(&f)[2 * HR] = qf[HR == 1 ? c : 0];
            if constexpr (HR == 2) ldsm_x4((q_lane ^ ((c & 3) * 32)) + (c >> 2) * QHALF, f[0], f[1], f[2], f[3]);
            few_mma<HR>(c & 1 ? s2[0] : s[0], f, f0, f1);
            few_mma<HR>(c & 1 ? s2[1] : s[1], f, f2, f3);
        }
        // Keys that not every row sees: behind the last one, or of the nodes.
        const bool edge = g + 16 > len || g + 16 > k1;
        auto hidden = [&](int key, uint32_t mask) {
            return key >= k1 || (key >= len && !(mask >> (key - len) & 1u));
        };
        float top[HR];
#pragma unroll
        for (int e = 0; e < HR; ++e) top[e] = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int e = 0; e < HR; ++e) {
                float &x = s[nb][2 * e], &y = s[nb][2 * e + 1];
                x = (x + s2[nb][2 * e]) * sl;
                y = (y + s2[nb][2 * e + 1]) * sl;
                if (edge) {
                    const int key = g + nb * 8 + 2 * lq;
                    if (hidden(key, anc[e])) x = -INFINITY;
                    if (hidden(key + 1, anc[e])) y = -INFINITY;
                }
                top[e] = fmaxf(top[e], fmaxf(x, y));
            }
        // The maximum moves, and O and the sum are scaled, only where it has grown by more than
        // 2^kFewLazy: weights up to 2^24 instead of 1 cost a floating sum nothing.
        bool move = false;
#pragma unroll
        for (int e = 0; e < HR; ++e) move |= top[e] > m[e] + kFewLazy;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int e = 0; e < HR; ++e) {
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                const float to = fmaxf(m[e], top[e]);
                const float f = to == -INFINITY ? 1.f : fast_exp2(m[e] - to);
                m[e] = to;
                l[e] *= f;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    o[j][2 * e] *= f;
                    o[j][2 * e + 1] *= f;
                }
            }
        }
        // P in bf16 for the second product: off by at most 2^-8 of itself, as the output's
        // rounding; the sum is of the unrounded values.
        uint32_t a[2 * HR];
#pragma unroll
        for (int e = 0; e < HR; ++e) {
            const float mu = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                const float x = fast_exp2(s[nb][2 * e] - mu), y = fast_exp2(s[nb][2 * e + 1] - mu);
                s[nb][2 * e] = x;
                s[nb][2 * e + 1] = y;
                l[e] += x + y;
                a[nb * HR + e] = pack_bf16(x, y);
            }
        }
        // Infinities and NaN among the V of nodes, which others than their descendants must not see
        // (0 * inf is NaN), are left out of the product and added by scalars where a row sees them.
        const int last = min(16, k1 - g);
        const uint8_t *v = ring + t % NST * STAGE + OPER;
        const bool odd = n > 1 && g + 16 > len && few_not_finite<L::HV>(v, kPoHalf, r0, last, lane);
        if (odd) {
            for (int x = 0; x < last; ++x) {
                const int from = (lane & ~3) | ((x & 7) >> 1);
                float w[HR];
#pragma unroll
                for (int e = 0; e < HR; ++e) {
                    const float w0 = x < 8 ? s[0][2 * e] : s[1][2 * e], w1 = x < 8 ? s[0][2 * e + 1] : s[1][2 * e + 1];
                    w[e] = __shfl_sync(0xffffffffu, x & 1 ? w1 : w0, from);
                }
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    uint32_t z = *reinterpret_cast<const uint32_t *>(v + (j >> 3) * kPoHalf + swz128(r0 + x, j & 7) + 4 * lq);
                    z &= few_odd_bits(z);
#pragma unroll
                    for (int e = 0; e < HR; ++e)
                        if (z && !hidden(g + x, anc[e])) {
                            o[j][2 * e] = fmaf(w[e], __uint_as_float(z << 16), o[j][2 * e]);
                            o[j][2 * e + 1] = fmaf(w[e], __uint_as_float(z & 0xffff0000u), o[j][2 * e + 1]);
                        }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NB; j += 2) {
            uint32_t f0, f1, f2, f3;
            ldsm_x4_trans(((vt + v_lane) ^ ((j & 7) * 16)) + (j >> 3) * kPoHalf, f0, f1, f2, f3);
            if (odd) {
                f0 &= ~few_odd_bits(f0);
                f1 &= ~few_odd_bits(f1);
                f2 &= ~few_odd_bits(f2);
                f3 &= ~few_odd_bits(f3);
            }
            few_mma<HR>(o[j], a, f0, f1);
            few_mma<HR>(o[j + 1], a, f2, f3);
        }
        if (tid < kPoKeys) look_up(t + NST, tid, page);
    }
    // The warps' maxima and sums, and the CTA's.
#pragma unroll
    for (int e = 0; e < HR; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if (lq == 0) wstat[warp][lr + 8 * e] = make_float2(m[e], l[e]);
    }
    copies_wait<0>();
    pdl_wait();
    // Where the prefix's parts lie: a chain of loads for the last warp, beside the others' sums.
    if (warp == L::WARPS - 1 && lane < R) {
        const int t = lane / G;
        parts_of[lane] = t < nodes ? pre_parts(p.pre, b, t, lane - t * G, h) : RowParts{0, 0, 1, 0};
    }
    __syncthreads();
    auto join = [](float2 &s, float2 x) {
        const float mx = fmaxf(s.x, x.x), mu = mx == -INFINITY ? 0.f : mx;
        s = make_float2(mx, s.y * fast_exp2(s.x - mu) + x.y * fast_exp2(x.x - mu));
    };
    auto of_cta = [&](int r) {
        float2 s = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int w = 0; w < L::WARPS / MT; ++w) join(s, wstat[w * MT + r / 16][r % 16]);
        return s;
    };
    if (tid < R) cstat[tid] = of_cta(tid);
    // The warps' O, at the CTA's maximum.
    float *osum = reinterpret_cast<float *>(ring);      // [WARPS / MT][R][OROW]
#pragma unroll
    for (int e = 0; e < HR; ++e) {
        const int r = mt * 16 + lr + 8 * e;
        if (r >= R) continue;
        const float f = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - of_cta(r).x);
        float *to = osum + (kw * R + r) * OROW + 2 * lq;
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *reinterpret_cast<float2 *>(to + j * 8) = make_float2(o[j][2 * e] * f, o[j][2 * e + 1] * f);
    }
    // The prefix's parts, of which the CTAs of the cluster take every C-th, then the CTA's own O, then the
    // other CTAs' sums of both.  An item is 4 channels of a row, of which a thread has ITEMS, whose loads
    // go side by side.  Neighbouring threads have up to 8 neighbouring rows of the same channels, which
    // lie together in a part.
    constexpr int ITEMS = MT * ROWS * (D / 4) / NT;
    const int lg = R > 4 ? 3 : R > 2 ? 2 : R - 1;       // log2 of such rows
    auto row_of = [&](int i) { return (i >> lg) / (D / 4) * (1 << lg) + (i & ((1 << lg) - 1)); };
    auto chan_of = [&](int i) { return (i >> lg) % (D / 4) * 4; };
    RowParts parts[ITEMS];
    float4 acc[ITEMS];
    float2 st[ITEMS];
    int most = 0;
#pragma unroll
    for (int x = 0; x < ITEMS; ++x) {
        const int r = row_of(x * NT + tid);
        parts[x] = r < R ? parts_of[r] : RowParts{0, 0, 1, 0};
        most = max(most, parts[x].count);
        acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        st[x] = make_float2(-INFINITY, 0.f);
    }
    auto add = [&](int x, float2 e, float4 y) {
        const float mx = fmaxf(st[x].x, e.x), mu = mx == -INFINITY ? 0.f : mx;
        const float f = fast_exp2(st[x].x - mu), w = fast_exp2(e.x - mu);
        st[x] = make_float2(mx, st[x].y * f + e.y * w);
        acc[x] = make_float4(acc[x].x * f + y.x * w, acc[x].y * f + y.y * w, acc[x].z * f + y.z * w, acc[x].w * f + y.w * w);
    };
    auto write = [&](int x, int r, int c) {
        const float inv = st[x].y > 0.f ? 1.f / st[x].y : 0.f;
        const int t = r / G;
        *reinterpret_cast<uint2 *>(p.out + (((long long)b * n + t) * p.H_q + h * G + (r - t * G)) * D + c) =
            make_uint2(pack_bf16(acc[x].x * inv, acc[x].y * inv), pack_bf16(acc[x].z * inv, acc[x].w * inv));
    };
    // 8 loads of a thread under way: parts of ITEMS items, or, with half the rows, more parts of one.
    auto join_parts = [&](auto of) {
        constexpr int HAS = decltype(of)::value, BATCH = 8 / HAS;
        for (int k0 = (int)rank; k0 < most; k0 += BATCH * (int)C) {
            float2 e[BATCH][HAS];
            float4 y[BATCH][HAS];
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
#pragma unroll
                for (int x = 0; x < HAS; ++x) {
                    e[k][x] = make_float2(-INFINITY, 0.f);
                    y[k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    const int j = k0 + k * (int)C;
                    if (j < parts[x].count) {
                        const long long at = parts[x].tile + (long long)j * parts[x].step;
                        e[k][x] = __ldcg(p.pre.stat + at * 128 + parts[x].row);
                        y[k][x] = __ldcg(p.pre.part + (at * (D / 4) + chan_of(x * NT + tid) / 4) * 128 + parts[x].row);
                    }
                }
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
#pragma unroll
                for (int x = 0; x < HAS; ++x) add(x, make_float2(e[k][x].x * sl, e[k][x].y), y[k][x]);
        }
    };
    if (HR == 1 && R <= 4) join_parts(Items<1>());
    else join_parts(Items<ITEMS>());
    __syncthreads();
#pragma unroll
    for (int x = 0; x < ITEMS; ++x) {
        const int r = row_of(x * NT + tid), c = chan_of(x * NT + tid);
        if (r >= R) continue;
        float4 *o4 = reinterpret_cast<float4 *>(osum + r * OROW + c);
        if (r / G < nodes) {
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < L::WARPS / MT; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(osum + (w * R + r) * OROW + c);
                sum = make_float4(sum.x + y.x, sum.y + y.y, sum.z + y.z, sum.w + y.w);
            }
            add(x, cstat[r], sum);
        }
        if (C == 1) {
            write(x, r, c);
        } else {
            *o4 = acc[x];                               // in the first warp's place, which only this thread has read
            if (c == 0) both[r] = st[x];
        }
    }
    if (C == 1) return;
    few_cluster_sync();
    for (int i = (int)rank * NT + tid; i < ITEMS * NT; i += (int)C * NT) {
        const int r = row_of(i), c = chan_of(i);
        if (r >= R) continue;
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
        st[0] = make_float2(-INFINITY, 0.f);
        for (uint32_t k = 0; k < C; ++k) add(0, few_ld2(few_at(&both[r], k)), few_ld4(few_at(osum + r * OROW + c, k)));
        write(0, r, c);
    }
    few_cluster_sync();                                 // no CTA ends while another reads its O
}

template <int D, int ROWS, int MT>
static magicdec_status launch_own_t(const PreOwn &p, cudaStream_t st) {
    using L = PoShape<D, ROWS, MT>;
    if (!magicdec_host::allow_smem_once<prefix_own_kernel<D, ROWS, MT>>(L::BYTES)) return MAGICDEC_ERR_CUDA;
    // As many CTAs a (sequence, KV head) as there are places for, with 64 slots each at least, or with parts of the
    // prefix to share: 4 turns of 8 loads (17 parts of 4 rows, 8 sequences behind 4k: a CTA 19.3 us, four 20.1; 65 of
    // 16 rows, 16 sequences of one KV head behind 16k: clusters of 2 and 8 34 and 26).
    const int slots = L::PER_SM * magicdec_host::sm_count();
    const long long cap = (long long)p.page_size * p.max_pages;
    const int items = (p.pre.n * p.pre.G * (D / 4) + L::NT - 1) / L::NT;
    int C = 1;
    while (C < kPoMaxCluster && 2ll * C * p.pre.B * p.pre.H_kv <= slots && (cap > C * kPoKeys || (long long)p.parts * items > C * kPoParts)) C *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, (unsigned)p.pre.H_kv, (unsigned)p.pre.B);
    cfg.blockDim = dim3(L::NT);
    cfg.dynamicSmemBytes = L::BYTES;
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
    if (cudaLaunchKernelEx(&cfg, prefix_own_kernel<D, ROWS, MT>, p) != cudaSuccess) return MAGICDEC_ERR_CUDA;
    return magicdec_host::launch_status();
}

magicdec_status launch_prefix_own(const PreOwn &p, int D, cudaStream_t st) {
    const int R = p.pre.n * p.pre.G;
    if (D == 128)
        return R <= 8    ? launch_own_t<128, 8, 1>(p, st)
               : R <= 16 ? launch_own_t<128, 16, 1>(p, st)
                         : launch_own_t<128, 16, 2>(p, st);
    return R <= 8 ? launch_own_t<64, 8, 1>(p, st)
           : R <= 16 ? launch_own_t<64, 16, 1>(p, st)
                     : launch_own_t<64, 16, 2>(p, st);
}

}  // namespace magicdec
