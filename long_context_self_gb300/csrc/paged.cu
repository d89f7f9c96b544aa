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

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// One pair held in one word: (lo, hi) -> (lo cos - hi sin, lo sin + hi cos).  Products and
// sums in fp32, one rounding of each result to bf16.
__device__ __forceinline__ uint32_t turn_pair(uint32_t x, float2 c) {
    const float a = bf_lo(x), b = bf_hi(x);
    return pack_bf16(a * c.x - b * c.y, a * c.y + b * c.x);
}
// Two channels and, `sign` times, the two that they are paired with: x cos + sign * y sin.
__device__ __forceinline__ uint32_t turn_with(uint32_t x, uint32_t y, float4 c, float sign) {
    return pack_bf16(bf_lo(x) * c.x + sign * (bf_lo(y) * c.y), bf_hi(x) * c.z + sign * (bf_hi(y) * c.w));
}

// A CTA takes T consecutive tokens of one sequence and goes over their head rows (q, k and v
// rows of d channels), VPH = d / 8 lanes a row, one 16-byte vector a lane: a row is read and
// written whole, and the channels rotated with one another come from another lane of the row.
// The first rows' loads are under way while the lengths, the table and the angles (once per
// token, for all its heads) are read and computed.  Bound: HBM, 4 (H_q + 2 H_kv) d bytes a
// token.
template <int T, int VPH, bool INTER>
__global__ void __launch_bounds__(kApThreads) paged_append_kernel(const AppendParams p) {
    constexpr int ROWS = kApThreads / VPH;      // rows of a pass
    constexpr int AHEAD = 4;                    // passes loaded together
    __shared__ __align__(16) float2 cs[T][VPH * 4];
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
    const int nt = min(T, cnt - i0);
    const int nq = p.q_out ? p.H_q : 0, R = nq + 2 * p.H_kv;         // rows of a token
    const int c = tid % VPH, total = nt * R;
    const long long tok0 = (long long)b * p.n + i0;
    auto load = [&](int w) {                                        // vector c of row w % R of token w / R
        const int t = T == 1 ? 0 : w / R, r = w - t * R;
        const uint16_t *src = r < nq ? p.q + (tok0 + t) * p.q_stride + r * p.d
                              : r < nq + p.H_kv ? p.k + (tok0 + t) * p.k_stride + (r - nq) * p.d
                                                : p.v + (tok0 + t) * p.v_stride + (r - nq - p.H_kv) * p.d;
        return ld_once_u4(reinterpret_cast<const uint4 *>(src) + c);
    };
    uint4 x[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
        const int w = tid / VPH + k * ROWS;
        if (w < total) x[k] = load(w);
    }
    if (p.parent)
        for (int i = tid; i < min(i0 + T, p.n); i += kApThreads)
            par[i] = checked(ld_dep(p.parent + (long long)b * p.n + i), -1, i - 1, p.err);
    if (tid < nt)
        dst[tid] = pool_row(p.table + (long long)b * p.max_pages, (long long)len + i0 + tid, p.page_size, p.n_pages,
                            p.max_pages, p.err);
    if (p.parent) {
        __syncthreads();
        if (tid < nt) {
            int depth = 0;
            for (int j = i0 + tid; par[j] >= 0 && par[j] < j; j = par[j]) ++depth;
            posn[tid] = depth;
        }
        __syncthreads();
    }
    // The angle position * inv_freq reaches 1e5 radians and more, where fp32 would
    // lose the low bits of the turn: the product in turns is formed and reduced in
    // fp64, and the fraction handed to the fp32 sine and cosine.
    const int half = p.rot / 2;
    for (int w = tid; w < nt * half; w += kApThreads) {
        const int t = w / half, f = w - t * half;
        const int at = p.parent ? posn[t] : i0 + t;
        const double turns = ((double)len + at) * ((double)ld_dep_f(p.inv_freq + f) * 0.15915494309189535);
        float s, co;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &co);
        cs[t][f] = make_float2(co, s);
    }
    __syncthreads();
    const int rv = p.rot / 8;                                       // rotated vectors of a row
    const int lane = tid & 31, other = c < rv / 2 ? lane + rv / 2 : lane - rv / 2;
    const float sign = c < rv / 2 ? -1.f : 1.f;
    const int f0 = INTER ? c * 4 : (c < rv / 2 ? c : c - rv / 2) * 8;
    // Every lane of a warp takes part in a pass's exchange; a row that is not there is not stored.
    for (int w0 = tid / VPH; w0 - tid / VPH < total; w0 += AHEAD * ROWS) {
        if (w0 != tid / VPH) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (w0 + k * ROWS < total) x[k] = load(w0 + k * ROWS);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int w = w0 + k * ROWS;
            if (w - tid / VPH >= total) break;                      // the same for the whole block
            const int t = T == 1 ? 0 : min(w / R, nt - 1), r = w - t * R;
            uint4 o = x[k];
            const bool turned = c < rv && r < nq + p.H_kv;
            if (INTER) {
                if (turned) {
                    const float2 *a = &cs[t][f0];
                    o = make_uint4(turn_pair(o.x, a[0]), turn_pair(o.y, a[1]), turn_pair(o.z, a[2]), turn_pair(o.w, a[3]));
                }
            } else {
                uint4 y;
                y.x = __shfl_sync(0xffffffffu, x[k].x, other & 31);
                y.y = __shfl_sync(0xffffffffu, x[k].y, other & 31);
                y.z = __shfl_sync(0xffffffffu, x[k].z, other & 31);
                y.w = __shfl_sync(0xffffffffu, x[k].w, other & 31);
                if (turned) {
                    const float4 *a = reinterpret_cast<const float4 *>(&cs[t][f0]);
                    o = make_uint4(turn_with(o.x, y.x, a[0], sign), turn_with(o.y, y.y, a[1], sign),
                                   turn_with(o.z, y.z, a[2], sign), turn_with(o.w, y.w, a[3], sign));
                }
            }
            if (w >= total) continue;
            if (r < nq) {
                reinterpret_cast<uint4 *>(p.q_out + ((tok0 + t) * p.H_q + r) * p.d)[c] = o;
            } else if (dst[t] >= 0) {
                const int h = r - nq;
                uint16_t *out = h < p.H_kv ? p.kp + (dst[t] * p.H_kv + h) * p.d : p.vp + (dst[t] * p.H_kv + h - p.H_kv) * p.d;
                reinterpret_cast<uint4 *>(out)[c] = o;
            }
        }
    }
}

template <int T, int VPH>
static magicdec_status launch_append_t(const AppendParams &p, int interleaved, cudaStream_t st) {
    const dim3 grid((unsigned)((p.n + T - 1) / T), (unsigned)p.B);
    return magicdec_host::launch_pdl(interleaved ? paged_append_kernel<T, VPH, true> : paged_append_kernel<T, VPH, false>,
                                     grid, dim3(kApThreads), 0, st, p);
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
    // Four tokens a CTA pay for its way in (angles, table, tree) once the GPU has CTAs enough
    // without splitting further.
    if ((long long)s.B * n >= 8ll * magicdec_host::sm_count())
        return s.d == 128 ? launch_append_t<4, 16>(p, interleaved, st) : launch_append_t<4, 8>(p, interleaved, st);
    return s.d == 128 ? launch_append_t<1, 16>(p, interleaved, st) : launch_append_t<1, 8>(p, interleaved, st);
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
    // A CTA takes several layers of a sequence, as long as there are some eight CTAs an SM.
    const int want = (8 * magicdec_host::sm_count() + s.B - 1) / s.B;
    const int groups = layers < want ? layers : want;
    return magicdec_host::launch_pdl(tree_commit_kernel, dim3((unsigned)s.B, (unsigned)groups), dim3(kCmThreads), 0, st,
                                     p);
}

}  // namespace magicdec
