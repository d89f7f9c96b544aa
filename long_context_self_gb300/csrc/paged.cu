// paged.cu -- appending rotated keys and values to a paged KV cache, and moving
// the rows of an accepted path to their final slots (sm_103a).
//
// A cache is a pool [n_pages, page_size, H_kv, d] and a block table
// [B, max_pages]: position s of sequence b is row s % page_size of page
// table[b, s / page_size].  A dense cache [B, L_cap, H_kv, d] is the pool with
// page_size = L_cap, max_pages = 1 and table[b, 0] = b.
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
constexpr int kApThreads = 256;
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

// (a, b) -> (a cos - b sin, a sin + b cos) on two packed bf16 pairs; products and
// sums in fp32, one rounding of each result to bf16.
__device__ __forceinline__ void turn2(uint32_t &a, uint32_t &b, float2 c0, float2 c1) {
    const float a0 = __uint_as_float(a << 16), a1 = __uint_as_float(a & 0xffff0000u);
    const float b0 = __uint_as_float(b << 16), b1 = __uint_as_float(b & 0xffff0000u);
    a = pack_bf16(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
    b = pack_bf16(a0 * c0.y + b0 * c0.x, a1 * c1.y + b1 * c1.x);
}

// One pair held in one word: (lo, hi) -> (lo cos - hi sin, lo sin + hi cos).
__device__ __forceinline__ uint32_t turn1(uint32_t x, float2 c) {
    const float a = __uint_as_float(x << 16), b = __uint_as_float(x & 0xffff0000u);
    return pack_bf16(a * c.x - b * c.y, a * c.y + b * c.x);
}

// A CTA takes T consecutive tokens of one sequence.  First the rot / 2 angles of
// each token, once for all its heads; then its 16-byte vectors, one item of a
// thread at a time.
template <int T, bool INTER>
__global__ void __launch_bounds__(kApThreads) paged_append_kernel(const AppendParams p) {
    __shared__ float2 cs[T][64];
    __shared__ int par[kApMaxTree];
    __shared__ long long dst[T];
    __shared__ int posn[T];
    const int b = blockIdx.y, i0 = blockIdx.x * T, tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int cap = p.page_size * p.max_pages;
    const int len = pg_clamp(checked(ld_dep(p.len + b), 0, cap, p.err), cap);
    const int cnt = p.n_new ? pg_clamp(checked(ld_dep(p.n_new + b), 0, p.n, p.err), p.n) : p.n;
    if (i0 >= cnt) return;
    if (p.parent)
        for (int i = tid; i < min(i0 + T, p.n); i += kApThreads)
            par[i] = checked(ld_dep(p.parent + (long long)b * p.n + i), -1, i - 1, p.err);
    __syncthreads();
    const int nt = min(T, cnt - i0);
    if (tid < nt) {
        const int i = i0 + tid;
        int depth = i;
        if (p.parent) {
            depth = 0;
            for (int j = i; par[j] >= 0 && par[j] < j; j = par[j]) ++depth;
        }
        posn[tid] = depth;
        dst[tid] = pool_row(p.table + (long long)b * p.max_pages, (long long)len + i, p.page_size, p.n_pages,
                            p.max_pages, p.err);
    }
    __syncthreads();
    // The angle position * inv_freq reaches 1e5 radians and more, where fp32 would
    // lose the low bits of the turn: the product in turns is formed and reduced in
    // fp64, and the fraction handed to the fp32 sine and cosine.
    const int half = p.rot / 2;
    for (int w = tid; w < nt * half; w += kApThreads) {
        const int t = w / half, f = w - t * half;
        const double turns = ((double)len + posn[t]) * ((double)ld_dep_f(p.inv_freq + f) * 0.15915494309189535);
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[t][f] = make_float2(c, s);
    }
    __syncthreads();
    const int vph = p.d / 8;                                    // 16-byte vectors per head
    const int rv = p.rot / 8;                                   // of them rotated
    const int per = INTER ? vph : vph - rv / 2;                 // items per rotated head
    const int nq = p.q_out ? p.H_q : 0;
    const int rot_items = (nq + p.H_kv) * per, items = rot_items + p.H_kv * vph;
    for (int w = tid; w < nt * items; w += kApThreads) {
        const int t = w / items;
        int it = w - t * items;
        const long long tok = (long long)b * p.n + i0 + t;
        if (it >= rot_items) {                                  // a value vector: copied
            it -= rot_items;
            if (dst[t] < 0) continue;
            const uint4 x = ld_once_u4(reinterpret_cast<const uint4 *>(p.v + tok * p.v_stride) + it);
            reinterpret_cast<uint4 *>(p.vp + dst[t] * p.H_kv * p.d)[it] = x;
            continue;
        }
        int h = it / per;
        const int c = it - h * per;
        const bool is_q = h < nq;
        const uint4 *src;
        uint4 *out;
        if (is_q) {
            src = reinterpret_cast<const uint4 *>(p.q + tok * p.q_stride) + h * vph;
            out = reinterpret_cast<uint4 *>(p.q_out + tok * p.H_q * p.d) + h * vph;
        } else {
            if (dst[t] < 0) continue;
            h -= nq;
            src = reinterpret_cast<const uint4 *>(p.k + tok * p.k_stride) + h * vph;
            out = reinterpret_cast<uint4 *>(p.kp + dst[t] * p.H_kv * p.d) + h * vph;
        }
        if (INTER) {
            uint4 x = ld_once_u4(src + c);
            if (c < rv) {
                const float2 *a = &cs[t][c * 4];
                x = make_uint4(turn1(x.x, a[0]), turn1(x.y, a[1]), turn1(x.z, a[2]), turn1(x.w, a[3]));
            }
            out[c] = x;
        } else if (c < rv / 2) {
            uint4 x = ld_once_u4(src + c), y = ld_once_u4(src + c + rv / 2);
            const float2 *a = &cs[t][c * 8];
            turn2(x.x, y.x, a[0], a[1]);
            turn2(x.y, y.y, a[2], a[3]);
            turn2(x.z, y.z, a[4], a[5]);
            turn2(x.w, y.w, a[6], a[7]);
            out[c] = x;
            out[c + rv / 2] = y;
        } else {
            out[c + rv / 2] = ld_once_u4(src + c + rv / 2);
        }
    }
}

template <int T>
static magicdec_status launch_append_t(const AppendParams &p, int interleaved, cudaStream_t st) {
    const dim3 grid((unsigned)((p.n + T - 1) / T), (unsigned)p.B);
    if (interleaved)
        return magicdec_host::launch_pdl(paged_append_kernel<T, true>, grid, dim3(kApThreads), 0, st, p);
    return magicdec_host::launch_pdl(paged_append_kernel<T, false>, grid, dim3(kApThreads), 0, st, p);
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
    return launch_append_t<1>(p, interleaved, st);
}

// ---------------------------------------------------------------------- commit
constexpr int kCmThreads = 256;
constexpr int kCmBatch = 8;          // rows in flight per thread

struct CommitParams {
    uint4 *kp, *vp;                  // [layers, n_pages, page_size, H_kv, d] as 16-byte vectors
    const int32_t *len, *path, *n_acc, *table;
    int *err;
    int B, n, row_vecs, page_size, n_pages, max_pages;
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
    const int rows = min(max(ld_dep(p.n_acc + b), -1), p.n - 1) + 1;
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
    const long long layer = (long long)blockIdx.y * p.n_pages * p.page_size * p.row_vecs;
    for (int c = blockIdx.z * kCmThreads + tid; c < 2 * p.row_vecs; c += gridDim.z * kCmThreads) {
        uint4 *base = (c < p.row_vecs ? p.kp + c : p.vp + (c - p.row_vecs)) + layer;
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
    const int splits = (2 * p.row_vecs + kCmThreads - 1) / kCmThreads;
    return magicdec_host::launch_pdl(tree_commit_kernel,
                                     dim3((unsigned)s.B, (unsigned)layers, (unsigned)(splits < 8 ? splits : 8)),
                                     dim3(kCmThreads), 0, st, p);
}

}  // namespace magicdec
