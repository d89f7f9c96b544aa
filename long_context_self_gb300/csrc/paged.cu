// paged.cu -- appending rotated keys and values to a paged KV cache, and moving
// the rows of an accepted path to their final slots (sm_103a).
//
// A cache is a pool [n_pages, page_size, H_kv, d] and a block table
// [B, max_pages]: position s of sequence b is row s % page_size of page
// table[b, s / page_size].  A dense cache [B, L_cap, H_kv, d] is the pool with
// page_size = L_cap, max_pages = 1 and table[b, 0] = b.
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
template <int NT, int LR, bool INTER>
__global__ void __launch_bounds__(NT) paged_append_kernel(const AppendParams p) {
    constexpr int ROWS = NT / LR;               // rows of a pass
    constexpr int AHEAD = 3;                    // passes loaded together
    __shared__ float2 cs[LR * 8];               // room for d / 2 angles
    __shared__ int par[kApMaxTree];
    __shared__ unsigned turns[kApMaxTree / 32];
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
        const double turns = ((double)len + at) * ((double)ld_dep_f(p.inv_freq + f) * 0.15915494309189535);
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
        if (r0 >= AHEAD * ROWS) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (r0 + k * ROWS < R) load(r0 + k * ROWS, x[k]);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int r = r0 + k * ROWS;
            if (r >= R) break;
            uint4 y = x[k][0], z = x[k][1];
            if (turned && r < nk) {
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
static magicdec_status launch_append_t(const AppendParams &p, int interleaved, cudaStream_t st) {
    return magicdec_host::launch_pdl(interleaved ? paged_append_kernel<NT, LR, true> : paged_append_kernel<NT, LR, false>,
                                     dim3((unsigned)p.n, (unsigned)p.B), dim3(NT), 0, st, p);
}

magicdec_status launch_paged_append(const magicdec_paged_shape &s, int n, const uint16_t *q, long long q_stride,
                                    const uint16_t *k, long long k_stride, const uint16_t *v, long long v_stride,
                                    const int32_t *len, const int32_t *n_new, const int32_t *parent,
                                    const float *inv_freq, int rot_dim, int interleaved, const int32_t *table,
                                    uint16_t *q_out, uint16_t *kp, uint16_t *vp, cudaStream_t st) {
    AppendParams p{};
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
    p.q_out = q_out;
    p.kp = kp;
    p.vp = vp;
    p.err = magicdec_host::device_error_word();
    p.B = s.B;
    p.n = n;
    p.H_q = s.H_q;
    p.H_kv = s.H_kv;
    p.d = s.d;
    p.rot = rot_dim;
    p.page_size = s.page_size;
    p.n_pages = s.n_pages;
    p.max_pages = s.max_pages;
    // Larger CTAs while there are fewer tokens than SMs: then a token's own rows take longest (one
    // token of 48 rows: 2.7 us with 256 threads, 3.5 us with 64).
    if ((long long)s.B * n >= magicdec_host::sm_count())
        return s.d == 128 ? launch_append_t<64, 8>(p, interleaved, st) : launch_append_t<64, 4>(p, interleaved, st);
    return s.d == 128 ? launch_append_t<256, 8>(p, interleaved, st) : launch_append_t<256, 4>(p, interleaved, st);
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
