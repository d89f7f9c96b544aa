// heavy_tc.cu -- attention over a heavy-hitter draft cache on the fifth-generation tensor cores
// (tcgen05 + TMEM), by up to 32 query rows of a KV head (sm_103a).  What it computes, and the way of
// up to 8 rows whose scores fit shared memory: heavy.cu.
//
// With the keys as the 128 rows of a tile, S^T = K Q^T (128 keys x NR query rows) puts a key in a
// TMEM lane: its thread has the key's scores for all query rows, so that a row's weight is a sum
// inside one thread, and the running maxima need no shuffles (they are held at values that a score
// may exceed by 2^24 before any is moved).  O^T += V^T P^T (d channels x NR) takes V as it lies
// and P from shared memory, 64 bytes a key.  A quarter of the instructions of mma.sync tiles
// of 16 rows, which bounded 9 rows and more (16 sequences of up to 12,001, R = 25: 166 us by them, 118
// so, 3.5 TB/s).
//
// A row's weight needs the softmax's final maximum and sum.  TMEM keeps the scores of the last 6 or 14 tiles
// (32 or 16 query rows) until then; those of earlier ones are computed again, by a second pass over their
// K, out of L2.  CTAs, clusters and exchange as in heavy.cu, two CTAs an SM.  85 sequences of 1721 rows, 8
// heads, R = 12: 135 us, a tenth less than with all scores computed again.
// Roles: warp 0 issues the TMA boxes, warp 1 the products, warps 2 to 5 are the softmax.
// Every wait is bounded; after one that gave up (error 1) the roles run on without waiting.
#include <climits>

#include "few_rows.cuh"
#include "heavy.cuh"
#include "tc.cuh"

namespace magicdec {

constexpr int kHtKeys = 128;                 // keys of a tile
constexpr int kHtHalf = kHtKeys * 128;       // bytes of 64 channels of them
constexpr int kHtThreads = 192;

// NR: query rows of the products, 16 or 32.
template <int D, int NR>
struct HtShape {
    static constexpr int HV = D / 64, SLOT = HV * kHtHalf;
    // Of the ring: K and V of a tile, or of two and a half (16 sequences of 12,001 rows, d = 64, R = 25: 107 us, and 2
    // more with two), as two CTAs an SM leave room for.
    static constexpr int SLOTS = HV == 1 ? 5 : 2;
    static constexpr int P = kHtKeys * 128, Q = HV * NR * 128;   // a key's probabilities: 128 bytes, 2 NR of them used
    static constexpr int BYTES = SLOTS * SLOT + P + Q;
    // TMEM: scores of as many tiles as half of it holds beside O (two CTAs an SM).
    static constexpr int COLS = 256, S = NR == 32 ? 6 : 14;
    static_assert((S + 1) * NR <= COLS, "scores and O");
    static_assert(NR * D * 4 <= P, "O takes the probabilities' place");
};

// Whether x holds for any of the 128 softmax threads; a barrier for them, too.
__device__ __forceinline__ bool ht_any(bool x) {
    int got;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(got)
        : "r"((int)x)
        : "memory");
    return got != 0;
}

template <int NR>
__device__ __forceinline__ void ht_load(uint32_t at, uint32_t (&x)[NR]) {
    if constexpr (NR == 32) tmem_ld32u(at, x);
    else tmem_ld16(at, x);
}

// NR values of every lane, each put together over the lanes: lane r ends with value r's, by NR - 1
// exchanges (and NR more where half a warp has a value) instead of 5 NR.
template <int NR, class F>
__device__ __forceinline__ float ht_rows(const uint32_t (&x)[NR], int lane, F put) {
    float y[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        y[r] = __uint_as_float(x[r]);
        if (NR == 16) y[r] = put(y[r], __shfl_xor_sync(0xffffffffu, y[r], 16));
    }
#pragma unroll
    for (int w = NR / 2; w >= 1; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const bool up = lane & w;
            const float mine = up ? y[i + w] : y[i], give = up ? y[i] : y[i + w];
            y[i] = put(mine, __shfl_xor_sync(0xffffffffu, give, w));
        }
    return y[0];
}

template <int D, int NR>
__global__ void __launch_bounds__(kHtThreads, 2)
    heavy_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const HeavyParams p) {
    using L = HtShape<D, NR>;
    constexpr int HV = L::HV, SLOT = L::SLOT, SLOTS = L::SLOTS, KS = D / 16, QHALF = NR * 128;
    constexpr uint32_t COLS = L::COLS, NS = L::S, O_COL = NS * NR;       // TMEM columns: S of NS tiles, then O
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem, *pbuf = smem + SLOTS * SLOT, *qs = pbuf + L::P;
    __shared__ uint64_t full[SLOTS], empty[SLOTS], s_full[NS], s_free[NS], p_full, o_done;
    __shared__ __align__(16) float held[NR];             // the value that a row's scores are taken from
    __shared__ __align__(16) float moved[NR];            // what its sums are scaled by when that moves
    __shared__ float wmax[4][NR];
    __shared__ __align__(16) float2 all[NR];             // of the cluster: (max, 1 / sum)
    __shared__ float2 cstat[NR];                         // of this CTA: (held, sum)
    __shared__ float wsum[4][NR];
    __shared__ uint32_t tmem_slot;
    __shared__ int met;                                  // V of a token's own row was not finite
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.z, h = blockIdx.y;
    const uint32_t rank = few_rank(), C = few_ctas();
    const float sl = p.scale_log2;
    if (tid == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (uint32_t s = 0; s < NS; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_free[s], 4);
        }
        mbar_init(&p_full, 4);
        mbar_init(&o_done, 1);
        mbar_fence_init();
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        met = 0;
    }
    if (tid < NR) held[tid] = -INFINITY;
    __syncthreads();
    pdl_wait();
    const int len0 = checked(ld_dep(p.len + b), 0, p.cap, p.err);
    uint32_t tmem = 0;
    if (warp > 0) {
        // The query rows (row i * G + g: token i, head g of the group), K-major and swizzled, while the producer asks
        // for the first keys.  Those behind the last are the last again, which sees every key: their scores are its
        // own, and with a factor of 0 add nothing to a weight that is a number (the score of a query of zeros and an
        // infinite key is none).
        constexpr int QT = kHtThreads - 32, QV = (NR * (D / 8) + QT - 1) / QT;   // 16-byte words a thread has
        uint4 qv[QV];
#pragma unroll
        for (int x = 0; x < QV; ++x) {
            const int at = x * QT + tid - 32, r = min(at / (D / 8), p.R - 1), c = at % (D / 8), i = r / p.G;
            const uint16_t *src = p.q + (((long long)b * p.n + i) * p.H_q + h * p.G + (r - i * p.G)) * D + c * 8;
            qv[x] = ld_dep_u4(reinterpret_cast<const uint4 *>(src));
        }
        // TMEM is taken when the kernels in front are done, whoever's they are: one of them might be about to take
        // its own on this SM, and wait for this CTA, which waits for it.  The kernels behind are let go afterwards, as
        // one of them may take its own before it waits for this one.  An SM begins no second such CTA before the
        // first has its columns, so that of the first ones half come 1 us behind the wait and find other SMs than
        // side by side (taken in front of the wait, 16 sequences of up to 12,001 rows, R = 25, 113 us and now 118,
        // all of 12,001 178 and 177, 85 of 1721 with R = 12 135 both).
        if (warp == 1) {
            tmem_alloc(&tmem_slot, COLS);
            pdl_trigger();
        }
#pragma unroll
        for (int x = 0; x < QV; ++x) {
            const int at = x * QT + tid - 32, r = at / (D / 8), c = at % (D / 8);
            if (r < NR) *reinterpret_cast<uint4 *>(qs + (c >> 3) * QHALF + swz128(r, c & 7)) = qv[x];
        }
        fence_proxy_async_smem();
        tc_fence_before();
        named_bar_sync(3, QT);
        tc_fence_after();
        tmem = tmem_slot;
    }
    const int len = len0 < 0 ? 0 : (len0 > p.cap ? p.cap : len0);
    // This CTA's keys: [k0, k1), in tiles.
    const int per = ((len + (int)C - 1) / (int)C + kHtKeys - 1) / kHtKeys * kHtKeys;
    const int k0 = (int)min((long long)len, (long long)rank * per), k1 = (int)min((long long)len, (long long)k0 + per);
    const int tiles = (k1 - k0 + kHtKeys - 1) / kHtKeys;
    const int again = max(0, tiles - (int)NS);           // tiles whose scores are computed twice
    const long long row0 = ((long long)b * p.H_kv + h) * p.cap;
    const int own = len - p.n;                           // the first of the tokens' own rows
    bool ok = smem_u32(smem) % 1024 == 0;
    if (!ok && tid == 0) raise_error(p.err, kErrState);

    // A warp's role ends its first pass, all meet where the cluster exchanges, then the second.
    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        // Slots in order: K and V of every tile, then K again of the first ones.
        const uint64_t once = policy_evict_first(), keep = policy_evict_normal();
        auto produce = [&](int from, int to) {
            for (int s = from; ok && s < to; ++s) {
                const uint32_t st = (uint32_t)s % SLOTS;
                ok = mbar_poll(&empty[st], ((uint32_t)s / SLOTS & 1) ^ 1, p.err);
                if (!ok) return;
                const bool first = s < 2 * tiles, is_v = first && (s & 1);
                const int t = first ? s / 2 : s - 2 * tiles;
                mbar_arrive_expect_tx(&full[st], SLOT);
                for (int f = 0; f < HV; ++f)
                    tma_load_4d(ring + st * SLOT + f * kHtHalf, is_v ? &tmv : &tmk, f * 64, k0 + t * kHtKeys, h, b,
                                &full[st], first && !is_v ? keep : once);
            }
        };
        // What the second pass has a place for does not wait for the exchange.
        const int ahead = 2 * tiles + min(again, SLOTS), last = 2 * tiles + again;
        if (lane == 0) produce(0, ahead);
        __syncwarp();
        if (C > 1) few_cluster_sync();
        if (lane == 0) {
            produce(ahead, last);
            // No copy may be in flight when the CTA ends.
            for (int s = max(0, last - SLOTS); s < last; ++s)
                mbar_poll(&full[s % SLOTS], (uint32_t)s / SLOTS & 1, p.err);
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA issuer
        const bool one = elect_one();
        const uint32_t idesc_s = umma_idesc_bf16(kHtKeys, NR);
        const uint32_t idesc_o = umma_idesc_bf16(D, NR) | (1u << 15) | (1u << 16);   // V^T and P lie along the keys
        const uint64_t kdesc = umma_desc_sw128(smem_u32(ring)), qdesc = umma_desc_sw128(smem_u32(qs));
        const uint64_t vdesc = desc_v(smem_u32(ring), 1024, kHtHalf), pdesc = desc_v(smem_u32(pbuf), 1024, 1024);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = mbar_poll(bar, parity, p.err);
        };
        uint32_t made = 0;                               // S so far, in both passes
        auto scores = [&](int slot) {
            const uint32_t st = (uint32_t)slot % SLOTS, buf = made % NS;
            wait(&full[st], (uint32_t)slot / SLOTS & 1);
            if (made >= NS) wait(&s_free[buf], (made / NS - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                umma_bf16(tmem + buf * NR, kdesc + st * (SLOT >> 4) + (ks >> 2) * (kHtHalf >> 4) + (ks & 3) * 2,
                          qdesc + (ks >> 2) * (QHALF >> 4) + (ks & 3) * 2, idesc_s, ks > 0);
            umma_commit(&empty[st]);
            umma_commit(&s_full[buf]);
            ++made;
        };
        if (one) {
            if (tiles > 0) scores(0);
            for (int t = 0; t < tiles; ++t) {
                if (t + 1 < tiles) scores(2 * t + 2);
                const int slot = 2 * t + 1;
                const uint32_t st = (uint32_t)slot % SLOTS;
                wait(&full[st], (uint32_t)slot / SLOTS & 1);
                wait(&p_full, t & 1);
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kHtKeys / 16; ++ks)
                    umma_bf16(tmem + O_COL, vdesc + st * (SLOT >> 4) + ks * (2048 >> 4), pdesc + ks * (2048 >> 4), idesc_o,
                              t > 0 || ks > 0);
                umma_commit(&empty[st]);
                umma_commit(&o_done);
            }
        }
        __syncwarp();
        if (C > 1) few_cluster_sync();
        if (one) {
            for (int t = 0; t < again; ++t) scores(2 * tiles + t);
            // The products in flight end before the shared memory and TMEM that they use go.
            if (made) wait(&s_full[(made - 1) % NS], (made - 1) / NS & 1);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax warps
        const int quad = warp & 3, row = 32 * quad + lane;              // TMEM lanes 32 * quad ..
        const uint32_t ts = tmem + ((uint32_t)(32 * quad) << 16);
        float l[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) l[r] = 0.f;
        uint32_t used = 0;                               // S so far
        // The scores of this thread's key, and from which query row on they count: a token's own row
        // is seen by it and later ones.
        auto get = [&](uint32_t at, bool last, uint32_t (&x)[NR]) {
            tc_fence_after();
            ht_load<NR>(ts + at * NR, x);
            tc_fence_before();
            __syncwarp();
            if (last && lane == 0) mbar_arrive(&s_free[at]);
        };
        auto take = [&](bool last, uint32_t (&x)[NR]) {
            ok = few_wait(&s_full[used % NS], used / NS & 1, p.err, ok, lane);
            get(used % NS, last, x);
            ++used;
        };
        auto from_row = [&](int key) { return key >= k1 ? NR : key < own ? 0 : min((key - own) * p.G, NR); };
        for (int t = 0; t < tiles; ++t) {
            const int key = k0 + t * kHtKeys + row;
            const bool edge = k0 + (t + 1) * kHtKeys > min(own + 1, k1);     // alike in all threads
            uint32_t x[NR];
            take(t < again, x);
            const int lo = edge ? from_row(key) : 0;
            bool move = false;
#pragma unroll
            for (int r = 0; r < NR; r += 4) {
                const float4 m4 = *reinterpret_cast<const float4 *>(held + r);
                const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y = __uint_as_float(x[r + e]) * sl;
                    if (edge && r + e < lo) y = -INFINITY;
                    x[r + e] = __float_as_uint(y);
                    move |= y > m[e] + kFewLazy;
                }
            }
            if (ht_any(move)) {
                // Maxima move, and what has been summed is scaled, only where a score is above by more than
                // 2^kFewLazy: weights up to 2^24 instead of 1 cost a floating sum nothing.
                const float y = ht_rows<NR>(x, lane, [](float a, float b) { return fmaxf(a, b); });
                if (lane < NR) wmax[quad][lane] = y;
                named_bar_sync(2, 128);
                if (row < NR) {
                    const float was = held[row], y = fmaxf(fmaxf(wmax[0][row], wmax[1][row]), fmaxf(wmax[2][row], wmax[3][row]));
                    const float to = fmaxf(was, y);
                    moved[row] = to == -INFINITY ? 1.f : fast_exp2(was - to);
                    held[row] = to;
                }
                named_bar_sync(2, 128);
#pragma unroll
                for (int r = 0; r < NR; ++r) l[r] *= moved[r];
                if (t > 0) {
                    ok = few_wait(&o_done, (t - 1) & 1, p.err, ok, lane);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < NR; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(ts + O_COL + c, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * moved[c + i]);
                        tmem_st16(ts + O_COL + c, o);
                    }
                    tmem_wait_st();
                }
            }
            // P in bf16 for the second product: off by at most 2^-8 of itself, as the output's
            // rounding; the sums are of the unrounded values.
            uint32_t u[NR / 2];
#pragma unroll
            for (int r = 0; r < NR; r += 4) {
                const float4 m4 = *reinterpret_cast<const float4 *>(held + r);
                const float m[4] = {m4.x, m4.y, m4.z, m4.w};
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = fast_exp2(__uint_as_float(x[r + e]) - (m[e] == -INFINITY ? 0.f : m[e]));
                    l[r + e] += y[e];
                }
                u[r / 2] = pack_bf16(y[0], y[1]);
                u[r / 2 + 1] = pack_bf16(y[2], y[3]);
            }
            if (t > 0) ok = few_wait(&o_done, (t - 1) & 1, p.err, ok, lane);      // the last P has been used
#pragma unroll
            for (int c = 0; c < NR / 8; ++c)
                *reinterpret_cast<uint4 *>(pbuf + swz128(row, c)) = make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
            if (edge) {
                // V behind the last row may hold anything, and 0 * NaN is NaN: zeros.  Infinities and NaN in the
                // tokens' own rows, which earlier ones must not see, are taken out and added at the end.
                const uint32_t slot = 2 * t + 1, st = slot % SLOTS;
                ok = few_wait(&full[st], slot / SLOTS & 1, p.err, ok, lane);
                auto word = [&](int c) {
                    return reinterpret_cast<uint4 *>(ring + st * SLOT + (c >> 3) * kHtHalf + swz128(row, c & 7));
                };
                if (key >= k1) {
#pragma unroll
                    for (int c = 0; c < HV * 8; ++c) *word(c) = make_uint4(0, 0, 0, 0);
                } else if (p.n > 1 && key >= own) {
#pragma unroll 4
                    for (int c = 0; c < HV * 8; ++c) {
                        uint4 *at = word(c);
                        const uint4 y = *at;
                        const uint4 odd = make_uint4(few_odd_bits(y.x), few_odd_bits(y.y), few_odd_bits(y.z), few_odd_bits(y.w));
                        if (odd.x | odd.y | odd.z | odd.w) {
                            met = 1;
                            *at = make_uint4(y.x & ~odd.x, y.y & ~odd.y, y.z & ~odd.z, y.w & ~odd.w);
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full);
        }
        // The sums over the keys.
        uint32_t sums[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) sums[r] = __float_as_uint(l[r]);
        const float sum_r = ht_rows<NR>(sums, lane, [](float a, float b) { return a + b; });
        if (lane < NR) wsum[quad][lane] = sum_r;
        named_bar_sync(2, 128);
        if (row < NR) cstat[row] = make_float2(held[row], wsum[0][row] + wsum[1][row] + wsum[2][row] + wsum[3][row]);
        if (C > 1) few_cluster_sync();
        else named_bar_sync(2, 128);
        if (row < NR) {
            float2 s = make_float2(-INFINITY, 0.f);
            for (uint32_t c = 0; c < C; ++c) {
                const float2 x = few_ld2(few_at(&cstat[row], c));
                const float mx = fmaxf(s.x, x.x), mu = mx == -INFINITY ? 0.f : mx;
                s = make_float2(mx, s.y * fast_exp2(s.x - mu) + x.y * fast_exp2(x.x - mu));
            }
            // A sum of zero: a row that sees nothing.  One of NaN stays so, in the output (NaN * 0, where no score
            // of this CTA's was a number) and in every weight that it has a part in.
            all[row] = make_float2(s.x == -INFINITY ? 0.f : s.x, row >= p.R || s.y == 0.f ? 0.f : 1.f / s.y);
            moved[row] = tiles == 0 ? 0.f : (held[row] == -INFINITY ? 0.f : fast_exp2(held[row] - all[row].x)) * all[row].y;
        }
        named_bar_sync(2, 128);
        // O, in the softmax's own scale, to the probabilities' place: [R][D].
        if (tiles > 0) ok = few_wait(&o_done, (tiles - 1) & 1, p.err, ok, lane);
        tc_fence_after();
        float *osum = reinterpret_cast<float *>(pbuf);
        const int chan = D == 128 ? row : 16 * quad + lane;              // 64 rows lie in the first 16 lanes of every 32
        const bool real = D == 128 || lane < 16;
        const bool odd = met;
#pragma unroll
        for (int c = 0; c < NR; c += 16) {
            uint32_t o[16];
            tmem_ld16(ts + O_COL + c, o);
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(f + i) = *reinterpret_cast<const float4 *>(moved + c + i);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float y = f[i] == 0.f ? 0.f : __uint_as_float(o[i]) * f[i];
                if (real && c + i < p.R) osum[(c + i) * D + chan] = y;
            }
            __syncwarp();                                // TMEM is read by whole warps
        }
        if (odd && real)
            for (int j = max(own, k0); j < k1; ++j) {
                const uint32_t z = (uint32_t)__ldcg(p.v + (row0 + j) * D + chan) << 16;
                if ((z & 0x7f800000u) == 0x7f800000u)
                    for (int r = max(0, j - own) * p.G; r < p.R; ++r) osum[r * D + chan] += __uint_as_float(z);
            }
        // Every row's weight, summed over the query rows in their order: of the last tiles from the scores that
        // are there still, then of the first ones, whose scores are computed again.
        const int first_new = p.next_pos ? own : INT_MAX;
        for (int i = 0; i < tiles; ++i) {
            const bool there = i < tiles - again;
            const int t = there ? again + i : i - (tiles - again);
            const int key = k0 + t * kHtKeys + row;
            const float old = key < k1 && key < first_new ? __ldcg(p.weight + row0 + key) : 0.f;
            uint32_t x[NR];
            if (there) get((uint32_t)t % NS, true, x);
            else take(true, x);
            const int lo = from_row(key);
            float w = 0.f;
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
                const float4 a = *reinterpret_cast<const float4 *>(&all[r]);
                if (r >= lo) w = fmaf(fast_exp2(fmaf(__uint_as_float(x[r]), sl, -a.x)), a.y, w);
                if (r + 1 >= lo) w = fmaf(fast_exp2(fmaf(__uint_as_float(x[r + 1]), sl, -a.z)), a.w, w);
            }
            if (key < k1) {
                p.weight[row0 + key] = old + w;
                if (key >= first_new) p.pos[row0 + key] = ld_dep(p.next_pos + b) + (key - first_new);
            }
        }
        tc_fence_before();
    }
    // O summed over the CTAs, each of which has a share of the channels.
    if (C > 1) few_cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, COLS);
    }
    // Several words of a thread side by side.
    constexpr int WORDS = (NR * (D / 4) + kHtThreads - 1) / kHtThreads;
    const int vecs = p.R * (D / 4), share = (vecs + (int)C - 1) / (int)C;
    const int from = (int)rank * share + tid, end = min(vecs, (int)(rank + 1) * share);
    float4 s[WORDS];
#pragma unroll
    for (int x = 0; x < WORDS; ++x) s[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t c = 0; c < C; ++c) {
        const uint32_t at = few_at(pbuf, c);
#pragma unroll
        for (int x = 0; x < WORDS; ++x) {
            const int i = from + x * kHtThreads;
            if (i >= end) continue;
            const float4 y = few_ld4(at + (uint32_t)i * 16);
            s[x] = make_float4(s[x].x + y.x, s[x].y + y.y, s[x].z + y.z, s[x].w + y.w);
        }
    }
#pragma unroll
    for (int x = 0; x < WORDS; ++x) {
        const int i = from + x * kHtThreads, r = i / (D / 4), c4 = i % (D / 4), t = r / p.G;
        if (i < end)
            *reinterpret_cast<uint2 *>(p.out + (((long long)b * p.n + t) * p.H_q + h * p.G + (r - t * p.G)) * D + c4 * 4) =
                make_uint2(pack_bf16(s[x].x, s[x].y), pack_bf16(s[x].z, s[x].w));
    }
    if (C > 1) few_cluster_sync();                       // no CTA ends while another reads its O
}

template <int D, int NR>
static magicdec_status launch_ht_t(const CUtensorMap &tmk, const CUtensorMap &tmv, const HeavyParams &p, int C,
                                   cudaStream_t st) {
    using L = HtShape<D, NR>;
    if (!magicdec_host::allow_smem_once<heavy_tc_kernel<D, NR>>(L::BYTES)) return MAGICDEC_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, (unsigned)p.H_kv, (unsigned)p.B);
    cfg.blockDim = dim3(kHtThreads);
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
    if (cudaLaunchKernelEx(&cfg, heavy_tc_kernel<D, NR>, tmk, tmv, p) != cudaSuccess) return MAGICDEC_ERR_CUDA;
    return magicdec_host::launch_status();
}

magicdec_status launch_heavy_tc(const HeavyParams &p, int D, const uint16_t *k, const uint16_t *v, cudaStream_t st) {
    // Clusters of 1 to 8, by the time they should take.  16 sequences of up to 12,001 rows, 8 heads,
    // R = 25, clusters of 1, 2, 4 and 8: 254, 138, 119 and 116 us, of 12,001 each 266, 176, 178 and 187; 128 of
    // 1029: 132, 144, 210 and 338.
    int best = 1;
    double least = 0;
    for (int C = 1; C <= 8; C *= 2) {
        const double t = heavy_time((long long)p.B * p.H_kv, p.cap, C, kHtKeys, D == 128 ? 3.2 : 1.8, 12.0);
        if (C == 1 || t < least) {
            least = t;
            best = C;
        }
    }
    CUtensorMap tmk, tmv;
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.cap, (uint64_t)p.H_kv, (uint64_t)p.B};
    const uint64_t row = (uint64_t)D * 2, strides[3] = {row, p.cap * row, (uint64_t)p.H_kv * p.cap * row};
    const uint32_t box[4] = {64, kHtKeys, 1, 1};
    if (!magicdec_host::encode_tmap_bf16_4d(&tmk, k, dims, strides, box) ||
        !magicdec_host::encode_tmap_bf16_4d(&tmv, v, dims, strides, box))
        return MAGICDEC_ERR_CUDA;
    if (D == 128) return p.R <= 16 ? launch_ht_t<128, 16>(tmk, tmv, p, best, st) : launch_ht_t<128, 32>(tmk, tmv, p, best, st);
    return p.R <= 16 ? launch_ht_t<64, 16>(tmk, tmv, p, best, st) : launch_ht_t<64, 32>(tmk, tmv, p, best, st);
}

}  // namespace magicdec
