// paged.cu -- appending rotated (and normed) keys and values to a paged KV cache, and
// moving the rows of an accepted path to their final slots (sm_103a).
//
// A cache is a pool [n_pages, page_size, H_kv, d] and a block table
// [B, max_pages]: position s of sequence b is row s % page_size of page
// table[b, s / page_size].  A dense cache [B, L_cap, H_kv, d] is the pool with
// page_size = L_cap, max_pages = 1 and table[b, 0] = b.
#include <cfloat>
#include <climits>

#include "common.cuh"

namespace magicdec {

__device__ __forceinline__ int pg_clamp(int v, int hi) { return v < 0 ? 0 : (v > hi ? hi : v); }

// A 16-byte load that keeps its place after pdl_wait() and may read memory that
// the same thread overwrites later in this kernel (so not the read-only path).
__device__ __forceinline__ uint4 ld_once_u4(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Pool row (page * page_size + offset) of slot s of a sequence, or -1: past the
// capacity (error 3) or through a table entry outside the pool (error 5).
__device__ __forceinline__ long long pool_row(const int32_t *table_row, long long s, int page_size, int n_pages,
                                              int max_pages, int *err) {
    const long long pg = s / page_size;
    if (s < 0 || pg >= max_pages) {
        raise_error(err, kErrCapacity);
        return -1;
    }
    const int id = ld_dep(table_row + pg);
    if (id < 0 || id >= n_pages) {
        raise_error(err, kErrPage);
        return -1;
    }
    return (long long)id * page_size + (s - pg * page_size);
}

// ---------------------------------------------------------------------- append
constexpr int kApMaxTree = 256;      // nodes of an explicit tree

struct AppendParams {
    const uint16_t *q, *k, *v;       // token rows of H * d elements, `*_stride` elements apart
    long long q_stride, k_stride, v_stride;
    const int32_t *len, *n_new, *parent, *table;
    const float *inv_freq;
    uint16_t *q_out, *kp, *vp;
    int *err;
    int B, n, H_q, H_kv, d, rot, page_size, n_pages, max_pages;
    // of the normed form
    const uint16_t *qw, *kw;         // [d] weights of the norms, or NULL: heads not normed
    const int32_t *pos, *axis;       // [B, n, axes] positions, or NULL; [rot / 2] axis of a pair, or NULL: axis 0
    float eps;
    int axes;
};

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// One pair held in one word: (lo, hi) -> (lo cos - hi sin, lo sin + hi cos).  Products and
// sums in fp32, one rounding of each result to bf16.
__device__ __forceinline__ uint32_t turn_pair(uint32_t x, float2 c) {
    const float a = bf_lo(x), b = bf_hi(x);
    return pack_bf16(a * c.x - b * c.y, a * c.y + b * c.x);
}
// Two channels of the first half (x) and the two that they are paired with (y).
__device__ __forceinline__ void turn_halves(uint32_t &x, uint32_t &y, float2 c0, float2 c1) {
    const float a0 = bf_lo(x), a1 = bf_hi(x), b0 = bf_lo(y), b1 = bf_hi(y);
    x = pack_bf16(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
    y = pack_bf16(a0 * c0.y + b0 * c0.x, a1 * c1.y + b1 * c1.x);
}

// A lane's 16 channels in fp32, two in a register pair: lo[k] and hi[k] are what pairs 2k and 2k + 1 of
// the rotation turn, whether those are halves (two words that hold neighbours) or interleaved.
struct Head16 {
    uint64_t lo[4], hi[4];
};
template <bool INTER>
__device__ __forceinline__ Head16 unpack16(uint4 y, uint4 z) {
    const uint32_t a[4] = {y.x, y.y, y.z, y.w}, b[4] = {z.x, z.y, z.z, z.w};
    Head16 h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t v = INTER ? (k < 2 ? a[2 * k] : b[2 * k - 4]) : a[k], w = INTER ? (k < 2 ? a[2 * k + 1] : b[2 * k - 3]) : b[k];
        h.lo[k] = INTER ? pair(bf_lo(v), bf_lo(w)) : pair(bf_lo(v), bf_hi(v));
        h.hi[k] = INTER ? pair(bf_hi(v), bf_hi(w)) : pair(bf_lo(w), bf_hi(w));
    }
    return h;
}
template <bool INTER>
__device__ __forceinline__ void pack16(const Head16 &h, uint4 &y, uint4 &z) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 l = apart(h.lo[k]), e = apart(h.hi[k]);
        uint32_t &v = INTER ? (k < 2 ? a[2 * k] : b[2 * k - 4]) : a[k], &w = INTER ? (k < 2 ? a[2 * k + 1] : b[2 * k - 3]) : b[k];
        v = INTER ? pack_bf16(l.x, e.x) : pack_bf16(l.x, l.y);
        w = INTER ? pack_bf16(l.y, e.y) : pack_bf16(e.x, e.y);
    }
    y = make_uint4(a[0], a[1], a[2], a[3]);
    z = make_uint4(b[0], b[1], b[2], b[3]);
}

// Squares of a head's d channels, summed over its LR lanes of 16 channels each.
template <int LR>
__device__ __forceinline__ float squares(const Head16 &h, unsigned lanes) {
    uint64_t a = 0, b = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        a = fma2(h.lo[k], h.lo[k], a);
        b = fma2(h.hi[k], h.hi[k], b);
    }
    const float2 c = apart(add2(a, b));
    float s = c.x + c.y;
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(lanes, s, o);
    return s;
}

// x / sqrt(mean(x^2) + eps) * w over a head's channels, this lane's 16 of them, in fp32 (the one
// rounding to bf16 comes behind the rotation).  Heads whose squares leave fp32 are scaled down
// first: eps, at most 2^128, is nothing beside them.
template <int LR>
__device__ __forceinline__ void norm_head(Head16 &h, const Head16 &w, float eps, unsigned lanes) {
    float s = squares<LR>(h, lanes), e = eps;
    if (s > FLT_MAX) {
        const uint64_t down = pair(0x1p-70f, 0x1p-70f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h.lo[k] = mul2(h.lo[k], down);
            h.hi[k] = mul2(h.hi[k], down);
        }
        s = squares<LR>(h, lanes);
        e *= 0x1p-140f;
    }
    // The root first: x / rms(x) is of the order of one, while the root's inverse times the weight may leave fp32.
    const float inv = rsqrtf(fmaf(s, 1.f / (LR * 16), e));
    const uint64_t i2 = pair(inv, inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h.lo[k] = mul2(mul2(h.lo[k], i2), w.lo[k]);
        h.hi[k] = mul2(mul2(h.hi[k], i2), w.hi[k]);
    }
}

// A CTA of NT threads takes a token, LR = d / 16 lanes one of its head rows (q, k and v rows
// of d channels) at a time, two 16-byte vectors a lane: the two whose channels are rotated
// with one another, or two neighbours.  A lane keeps to its channels, so its 8 angles stay in
// registers for all rows (read from shared memory for every row, they bounded the kernel: twice
// the time for 4096 tokens of 48 rows).  The first rows' loads are under way while the lengths, the
// table, the tree and the angles (once per token) are read and computed.  Bound: HBM,
// 4 (H_q + 2 H_kv) d bytes a token.  Small CTAs, because what a token needs first is a chain of
// loads that only other CTAs' rows can cover: 4096 tokens, each in a CTA of 64, 128 or 256
// threads, take 21.5, 23.0 and 38.0 us with inputs from HBM, 17.7, 19.5 and 34.2 with inputs in
// L2, of 14.9 us at the measured copy rate.
//
// NORM: query and key heads are normed before the rotation, in the registers that hold them: a
// lane's 16 squares and log2(LR) shuffles a row.  That is twice the instructions, and a row's chain is
// longer, so what counts is how many CTAs fit: two passes under way instead of three, the next
// loaded as soon as one is taken, the weights in shared memory, fp32 arithmetic by pairs, 80 registers
// (MINB: 12 CTAs of 64 threads an SM).  128 trees of 32 with inputs from HBM: 27.8 us, with three
// passes 31, one by one and in single fp32 34; 32,000 prompt tokens of 48 rows 140, 163 and 174 us.
template <int NT, int LR, bool INTER, bool NORM, int MINB = NT == 32 ? 24 : NT == 64 ? 12 : 3>
__global__ void __launch_bounds__(NT, NORM ? MINB : 0) paged_append_kernel(const AppendParams p) {
    constexpr int ROWS = NT / LR;               // rows of a pass
    constexpr int AHEAD = NORM ? 2 : 3;         // passes under way
    __shared__ float2 cs[LR * 8];               // room for d / 2 angles
    __shared__ int par[kApMaxTree];
    __shared__ unsigned turns[kApMaxTree / 32];
    __shared__ uint4 weight[NORM ? 4 * LR : 1];  // of query heads, then of key heads
    const int b = blockIdx.y, i = blockIdx.x, tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int cap = p.page_size * p.max_pages;
    const int len = pg_clamp(checked(ld_dep(p.len + b), 0, cap, p.err), cap);
    const int cnt = p.n_new ? pg_clamp(checked(ld_dep(p.n_new + b), 0, p.n, p.err), p.n) : p.n;
    if (i >= cnt) return;
    const int nq = p.q_out ? p.H_q : 0, R = nq + 2 * p.H_kv;        // rows of the token
    const long long tok = (long long)b * p.n + i;
    const int l = tid % LR, pairs = p.rot / 16;                     // pairs: lanes of a row that rotate halves
    const bool halves = !INTER && l < pairs;
    const int v0 = halves ? l : 2 * l, v1 = halves ? l + pairs : 2 * l + 1;   // the lane's vectors
    // Row r of the token: a base, from which r is counted, for each of the three kinds.
    const int nk = nq + p.H_kv;
    const uint16_t *qb = p.q + tok * p.q_stride, *kb = p.k + tok * p.k_stride - nq * p.d,
                   *vb = p.v + tok * p.v_stride - nk * p.d;
    auto load = [&](int r, uint4 (&x)[2]) {
        const uint4 *src = reinterpret_cast<const uint4 *>((r < nq ? qb : r < nk ? kb : vb) + r * p.d);
        x[0] = ld_once_u4(src + v0);
        x[1] = ld_once_u4(src + v1);
    };
    uint4 x[AHEAD][2];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (tid / LR + k * ROWS < R) load(tid / LR + k * ROWS, x[k]);
    const unsigned lanes = (LR == 8 ? 0xffu : 0xfu) << (tid % 32 / LR * LR);     // of a row
    if (NORM && tid < 4 * LR) {                                     // seen behind the angles' barrier
        const uint16_t *w = tid < 2 * LR ? p.qw : p.kw;
        if (w) weight[tid] = ld_dep_u4(reinterpret_cast<const uint4 *>(w) + tid % (2 * LR));
    }
    const long long dst = pool_row(p.table + (long long)b * p.max_pages, (long long)len + i, p.page_size, p.n_pages,
                                   p.max_pages, tid == 0 ? p.err : nullptr);
    int at = i;                                                     // position after len
    if (p.parent) {
        // The depth, by stretches of nodes each of which follows the one before it (a bit where
        // one does not): a chain is a single one.
        for (int j = tid; j < (i / 32 + 1) * 32; j += NT) {
            const int q = j <= i ? checked(ld_dep(p.parent + (long long)b * p.n + j), INT_MIN, j - 1, p.err) : -1;
            par[j] = q;
            const unsigned m = __ballot_sync(0xffffffffu, j == 0 || q != j - 1);
            if (tid % 32 == 0) turns[j / 32] = m;
        }
        __syncthreads();
        at = 0;
        for (int j = i; j >= 0;) {
            int w = j / 32;
            unsigned m = turns[w] & (0xffffffffu >> (31 - (j & 31)));
            while (m == 0 && w > 0) m = turns[--w];
            const int z = m ? w * 32 + 31 - __clz(m) : 0;
            at += j - z + 1;
            j = par[z] < z ? par[z] : -1;
        }
        --at;
    }
    // The angle position * inv_freq reaches 1e5 radians and more, where fp32 would
    // lose the low bits of the turn: the product in turns is formed and reduced in
    // fp64, and the fraction handed to the fp32 sine and cosine.
    for (int f = tid; f < p.rot / 2; f += NT) {
        double where = (double)len + at;
        if (NORM && p.pos) {
            const int ax = p.axis ? checked(ld_dep(p.axis + f), 0, p.axes - 1, p.err) : 0;
            where = ld_dep(p.pos + tok * p.axes + (ax < 0 || ax >= p.axes ? 0 : ax));
        }
        const double turns = where * ((double)ld_dep_f(p.inv_freq + f) * 0.15915494309189535);
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[f] = make_float2(c, s);
    }
    __syncthreads();
    // Interleaved, a vector has 4 angles; the halves' vectors share 8.
    const bool turned = INTER ? v0 * 8 < p.rot : halves;            // rot is a multiple of 16: both vectors or none
    float2 a[8];
    if (turned)
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = cs[l * 8 + k];
    uint16_t *qo = p.q_out + tok * p.H_q * p.d, *ko = p.kp + dst * p.H_kv * p.d - nq * p.d,
             *vo = p.vp + dst * p.H_kv * p.d - nk * p.d;
    for (int r0 = tid / LR; r0 < R; r0 += AHEAD * ROWS) {
        if (!NORM && r0 >= AHEAD * ROWS) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (r0 + k * ROWS < R) load(r0 + k * ROWS, x[k]);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int r = r0 + k * ROWS;
            if (r >= R) break;
            uint4 y = x[k][0], z = x[k][1];
            if (NORM && r + AHEAD * ROWS < R) load(r + AHEAD * ROWS, x[k]);
            if (NORM && r < nk && (r < nq ? p.qw : p.kw)) {
                Head16 h = unpack16<INTER>(y, z);
                const uint4 *w = weight + (r < nq ? 0 : 2 * LR);
                norm_head<LR>(h, unpack16<INTER>(w[v0], w[v1]), p.eps, lanes);
                if (turned)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t c = pair(a[2 * j].x, a[2 * j + 1].x), e = pair(a[2 * j].y, a[2 * j + 1].y);
                        const uint64_t lo = h.lo[j], hi = h.hi[j];
                        h.lo[j] = fma2(lo, c, mul2(hi, pair(-a[2 * j].y, -a[2 * j + 1].y)));
                        h.hi[j] = fma2(lo, e, mul2(hi, c));
                    }
                pack16<INTER>(h, y, z);
            } else if (turned && r < nk) {
                if (INTER) {
                    y = make_uint4(turn_pair(y.x, a[0]), turn_pair(y.y, a[1]), turn_pair(y.z, a[2]), turn_pair(y.w, a[3]));
                    z = make_uint4(turn_pair(z.x, a[4]), turn_pair(z.y, a[5]), turn_pair(z.z, a[6]), turn_pair(z.w, a[7]));
                } else {
                    turn_halves(y.x, z.x, a[0], a[1]);
                    turn_halves(y.y, z.y, a[2], a[3]);
                    turn_halves(y.z, z.z, a[4], a[5]);
                    turn_halves(y.w, z.w, a[6], a[7]);
                }
            }
            if (r >= nq && dst < 0) continue;
            uint4 *out = reinterpret_cast<uint4 *>((r < nq ? qo : r < nk ? ko : vo) + r * p.d);
            out[v0] = y;
            out[v1] = z;
        }
    }
}

template <int NT, int LR>
static magicdec_status launch_append_t(const AppendParams &p, int interleaved, bool norm, cudaStream_t st) {
    auto kern = interleaved ? paged_append_kernel<NT, LR, true, true> : paged_append_kernel<NT, LR, false, true>;
    if constexpr (NT > 32)
        if (!norm) kern = interleaved ? paged_append_kernel<NT, LR, true, false> : paged_append_kernel<NT, LR, false, false>;
    return magicdec_host::launch_pdl(kern, dim3((unsigned)p.n, (unsigned)p.B), dim3(NT), 0, st, p);
}

static magicdec_status launch_append(AppendParams &p, const magicdec_paged_shape &s, int interleaved, bool norm,
                                     cudaStream_t st) {
    p.err = magicdec_host::device_error_word();
    p.B = s.B;
    p.H_q = s.H_q;
    p.H_kv = s.H_kv;
    p.d = s.d;
    p.page_size = s.page_size;
    p.n_pages = s.n_pages;
    p.max_pages = s.max_pages;
    // Larger CTAs while there are fewer tokens than SMs: then a token's own rows take longest (one
    // token of 48 rows: 2.7 us with 256 threads, 3.5 us with 64).
    const long long tokens = (long long)s.B * p.n;
    // Normed, a warp a token where there are more tokens than CTAs of 64 threads have places, and a token's rows
    // are few: with twice the tokens under way their first loads are covered better (15,000 tokens of 20 rows of
    // 128 channels 53.5 and 45.5 us, of 64 41.5 and 29.1; 3000 of 36 rows 18.2 and 16.8; 4096 of 48 29.1 and 30.1,
    // 600 of 20 7.4 and 8.8).
    if (norm && tokens > 12ll * magicdec_host::sm_count() && ((p.q_out ? s.H_q : 0) + 2 * s.H_kv) * (s.d / 16) < 384)
        return s.d == 128 ? launch_append_t<32, 8>(p, interleaved, norm, st)
                          : launch_append_t<32, 4>(p, interleaved, norm, st);
    if (tokens >= magicdec_host::sm_count())
        return s.d == 128 ? launch_append_t<64, 8>(p, interleaved, norm, st)
                          : launch_append_t<64, 4>(p, interleaved, norm, st);
    return s.d == 128 ? launch_append_t<256, 8>(p, interleaved, norm, st)
                      : launch_append_t<256, 4>(p, interleaved, norm, st);
}

static AppendParams append_params(int n, const uint16_t *q, long long q_stride, const uint16_t *k, long long k_stride,
                                  const uint16_t *v, long long v_stride, const int32_t *len, const int32_t *n_new,
                                  const int32_t *parent, const float *inv_freq, int rot_dim, const int32_t *table,
                                  uint16_t *q_out, uint16_t *kp, uint16_t *vp) {
    AppendParams p{};
    p.n = n;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.len = len;
    p.n_new = n_new;
    p.parent = parent;
    p.table = table;
    p.inv_freq = inv_freq;
    p.rot = rot_dim;
    p.q_out = q_out;
    p.kp = kp;
    p.vp = vp;
    return p;
}

magicdec_status launch_paged_append(const magicdec_paged_shape &s, int n, const uint16_t *q, long long q_stride,
                                    const uint16_t *k, long long k_stride, const uint16_t *v, long long v_stride,
                                    const int32_t *len, const int32_t *n_new, const int32_t *parent,
                                    const float *inv_freq, int rot_dim, int interleaved, const int32_t *table,
                                    uint16_t *q_out, uint16_t *kp, uint16_t *vp, cudaStream_t st) {
    AppendParams p = append_params(n, q, q_stride, k, k_stride, v, v_stride, len, n_new, parent, inv_freq, rot_dim, table,
                                   q_out, kp, vp);
    return launch_append(p, s, interleaved, false, st);
}

magicdec_status launch_norm_append(const magicdec_paged_shape &s, int n, const uint16_t *q, long long q_stride,
                                   const uint16_t *k, long long k_stride, const uint16_t *v, long long v_stride,
                                   const uint16_t *q_weight, const uint16_t *k_weight, float eps, const int32_t *len,
                                   const int32_t *n_new, const int32_t *parent, const int32_t *pos, int axes,
                                   const int32_t *axis, const float *inv_freq, int rot_dim, int interleaved,
                                   const int32_t *table, uint16_t *q_out, uint16_t *kp, uint16_t *vp, cudaStream_t st) {
    AppendParams p = append_params(n, q, q_stride, k, k_stride, v, v_stride, len, n_new, parent, inv_freq, rot_dim, table,
                                   q_out, kp, vp);
    p.qw = q_weight;
    p.kw = k_weight;
    p.eps = eps;
    p.pos = pos;
    p.axis = axis;
    p.axes = axes;
    return launch_append(p, s, interleaved, true, st);
}

// ---------------------------------------------------------------------- commit
constexpr int kCmThreads = 256;
constexpr int kCmBatch = 8;          // rows in flight per thread

struct CommitParams {
    uint4 *kp, *vp;                  // [layers, n_pages, page_size, H_kv, d] as 16-byte vectors
    const int32_t *len, *path, *n_acc, *table;
    int *err;
    int B, n, layers, row_vecs, page_size, n_pages, max_pages;
};

// Slot len + i takes the row of slot len + path[i], i = 0 .. n_acc, in every
// layer.  One thread owns a 16-byte column of all rows, so the moves of a column
// are ordered by that thread alone: a batch is read before it is written, and
// since path ascends with path[i] >= i, a slot that a batch writes is read by no
// later one (path[j] >= j > i).
__global__ void __launch_bounds__(kCmThreads) tree_commit_kernel(const CommitParams p) {
    __shared__ long long src[256], dst[256];
    __shared__ int moves;
    const int b = blockIdx.x, tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int cap = p.page_size * p.max_pages;
    const int len = pg_clamp(checked(ld_dep(p.len + b), 0, cap, p.err), cap);
    const int rows = min(max(checked(ld_dep(p.n_acc + b), -1, p.n - 1, p.err), -1), p.n - 1) + 1;
    if (tid < 32) {
        const int32_t *table = p.table + (long long)b * p.max_pages;
        int found = 0;
        for (int i0 = 0; i0 < rows; i0 += 32) {
            const int i = i0 + tid;
            long long s = -1, d = -1;
            if (i < rows) {
                const int from = checked(ld_dep(p.path + (long long)b * p.n + i), 0, p.n - 1, p.err);
                if (from >= 0 && from < p.n && from != i) {
                    s = pool_row(table, (long long)len + from, p.page_size, p.n_pages, p.max_pages, p.err);
                    d = pool_row(table, (long long)len + i, p.page_size, p.n_pages, p.max_pages, p.err);
                }
            }
            const bool move = s >= 0 && d >= 0;
            const unsigned m = __ballot_sync(0xffffffffu, move);
            if (move) {
                const int at = found + __popc(m & ((1u << tid) - 1u));
                src[at] = s * p.row_vecs;
                dst[at] = d * p.row_vecs;
            }
            found += __popc(m);
        }
        if (tid == 0) moves = found;
    }
    __syncthreads();
    const int nm = moves;
    if (nm == 0) return;
    const long long layer = (long long)p.n_pages * p.page_size * p.row_vecs;
    const int cols = 2 * p.row_vecs;
    // Columns of the layers blockIdx.y, blockIdx.y + gridDim.y, ...
    const int layers = (p.layers - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;
    for (int w = tid; w < layers * cols; w += kCmThreads) {
        const int l = w / cols, c = w - l * cols;
        uint4 *base = (c < p.row_vecs ? p.kp + c : p.vp + (c - p.row_vecs)) +
                      ((long long)blockIdx.y + (long long)l * gridDim.y) * layer;
        for (int i = 0; i < nm; i += kCmBatch) {
            uint4 x[kCmBatch];
#pragma unroll
            for (int j = 0; j < kCmBatch; ++j)
                if (i + j < nm) x[j] = ld_once_u4(base + src[i + j]);
#pragma unroll
            for (int j = 0; j < kCmBatch; ++j)
                if (i + j < nm) base[dst[i + j]] = x[j];
        }
    }
}

magicdec_status launch_tree_commit(const magicdec_paged_shape &s, int n, int layers, const int32_t *len,
                                   const int32_t *path, const int32_t *n_acc, const int32_t *table, uint16_t *kp,
                                   uint16_t *vp, cudaStream_t st) {
    CommitParams p{};
    p.kp = reinterpret_cast<uint4 *>(kp);
    p.vp = reinterpret_cast<uint4 *>(vp);
    p.len = len;
    p.path = path;
    p.n_acc = n_acc;
    p.table = table;
    p.err = magicdec_host::device_error_word();
    p.B = s.B;
    p.n = n;
    p.row_vecs = s.H_kv * s.d / 8;
    p.page_size = s.page_size;
    p.n_pages = s.n_pages;
    p.max_pages = s.max_pages;
    p.layers = layers;
    // A CTA takes several layers of a sequence, as long as there are some eight CTAs an SM, and no
    // more columns than it counts in 32 bits.
    const int want = (8 * magicdec_host::sm_count() + s.B - 1) / s.B;
    const int most = INT_MAX / 2 / (2 * p.row_vecs), least = (layers + most - 1) / most;
    const int groups = layers < want ? layers : (want < least ? least : want);
    return magicdec_host::launch_pdl(tree_commit_kernel, dim3((unsigned)s.B, (unsigned)groups), dim3(kCmThreads), 0, st,
                                     p);
}

}  // namespace magicdec
