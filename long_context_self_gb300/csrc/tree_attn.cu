// tree_attn.cu -- attention of a tree of drafted tokens over a paged KV cache,
// on the fifth-generation tensor cores (tcgen05 + TMEM), sm_103a.
//
//   out_i = sum_j p_ij v_j,  p_i = softmax_j(q_i . k_j / sqrt(d))
//
// over j in the committed positions [0, len) and the slots len + a of node i's
// ancestors a and itself.  The n nodes and the G query heads of a KV head give
// R = n * G query rows that read the same K and V, so one tile of 128 keys is
// the product S = Q K^T (128 rows x 128 keys) and O += P V (128 rows x d).
// Floors: K and V once, 4 (len + n) H_kv d bytes; 4 n len H_q d flops.  They
// meet at R of about 270, so one kernel serves both ends: below, it has to keep
// HBM busy while the tensor cores idle, above, the other way round.
//
// A row tile is 128 rows: NB = 128 / G whole nodes.  A CTA holds two streams,
// each with its own S, O (TMEM) and two softmax warpgroups, one per half of the
// keys of a tile (a thread: one row, 64 keys):
//   one row tile  (n <= NB): the streams take the even and odd key tiles, so one
//     softmax runs while the other's products do; their O are merged at the end;
//   two row tiles (n > NB):  each stream owns a row tile and sees every key tile;
//     K and V are read once for both (further pairs of tiles: other work items).
// P overwrites S's columns as bf16 (the A operand of the second product comes
// from TMEM).  P in bf16 costs a relative 2^-9 per probability, as much as the
// rounding of the output; sums, maxima and O are fp32.
//
// Work: the key tiles of all (sequence, KV head, row block), as one list, cut
// into equal runs of tiles, one per CTA; what a CTA has of a list entry that it
// does not own whole goes to the workspace as (O, max, sum) and is joined by a
// second kernel in a fixed order.  No atomics: results do not change from run to run.
//
// Roles (640 threads): warps 0, 2 and 3 issue the TMA boxes, warp 1 the MMAs, warps 4-11
// and 12-19 are the softmax of the two streams, which take over registers that the
// first warpgroup gives up.  Every wait is bounded; after one that
// gave up (error 1) the roles run on without waiting, so that all of them end.
#include "common.cuh"

namespace magicdec {

constexpr int kTrThreads = 640;
constexpr int kTrKeys = 128;                  // keys per tile
constexpr int kTrBox = kTrKeys * 128;         // 128 rows x 64 channels (16 KB)
constexpr int kTrMaxNodes = 256;
constexpr int kTrOut = 256;                   // first TMEM column of O (S: 0 and 128)
constexpr float kTrLazy = 8.0f;               // log2 growth of a row's maximum that is put up with

// What the joining kernel has to know of a sequence: its first entry in the list
// of work, the number of its key tiles and its nodes.  Entry B holds the run length.
struct TreeSeq {
    long long first;
    int tiles, nodes;
};

struct TreeAttnParams {
    const int32_t *len, *n_nodes, *parent, *table;
    uint16_t *out;
    TreeSeq *seq;          // workspace: [B + 1]
    float2 *stat;          // workspace: [2 * grid][RT * 128] (max, sum)
    float4 *part;          // workspace: [2 * grid][RT][d / 4][128]
    int *err;
    int B, H_q, H_kv, G, n, page_size, n_pages, max_pages;
    int NB;                // nodes per row tile
    int ppt;               // pages per key tile (pages of at most 128 rows), else 0
    int tpp;               // key tiles per page (larger pages)
    int grid;
    int br;                // rows of a box
    int by8;               // pages of a multiple of 8 rows: copied by 5-D boxes
    uint32_t sbo, hoff;    // bytes between groups of 8 rows, and between 64-channel halves, of a K or V tile
    float scale_log2;      // log2(e) / sqrt(d)
};

__device__ __forceinline__ int tr_clamp(int v, int hi) { return v < 0 ? 0 : (v > hi ? hi : v); }

// ---------------------------------------------------------------- tcgen05 forms
// A K or V tile in shared memory: rows of 64 channels (128 bytes, swizzled), groups of
// 8 rows `sbo` apart, the two halves of 128 channels `hoff` apart.  Pages of a multiple of
// 8 rows are copied whole, [group][half][8 rows], by one box; other pages half by half,
// [half][rows].
// K is K-major: a row is a key's channels, the reduction runs along it.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr, uint32_t sbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)1u << 16;                   // leading byte offset (unused for swizzled K-major)
    d |= (uint64_t)(sbo >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
// V is MN-major: the reduction runs over the rows, 64 channels of a row lie together,
// the next 64 the leading byte offset further.
__device__ __forceinline__ uint64_t desc_v(uint32_t saddr, uint32_t sbo, uint32_t hoff) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(hoff >> 4) << 16;
    d |= (uint64_t)(sbo >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// D[tmem] (+)= A[tmem] * B[smem], B transposed (MN-major) by the instruction descriptor.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

#define TR_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
    "=r"(r[i + 6]), "=r"(r[i + 7])
#define TR_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
    "r"(r[i + 6]), "r"(r[i + 7])

// 64 columns of S: two loads and their completion in one statement, so that no use
// of a register can be moved before the wait.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,"
        "%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : TR_R8(r, 0), TR_R8(r, 8), TR_R8(r, 16), TR_R8(r, 24), TR_R8(r, 32), TR_R8(r, 40), TR_R8(r, 48), TR_R8(r, 56)
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : TR_R8(r, 0), TR_R8(r, 8)
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        TR_W8(r, 0), TR_W8(r, 8)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One thread of a converged warp, the same each time.  The compiler knows a branch on it
// for uniform, and keeps descriptors in uniform registers: with a branch on the lane
// number it moved them there one by one, 150 cycles a product instead of the 64 that it
// takes (8 products: 1250 -> 560 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(x));
    return x != 0;
}

// Registers per thread from here on, for the whole warpgroup.  640 threads start with
// 96 each; 64 + 4 * 104 is 5 * 96.
__device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }
__device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 104;"); }

// Whether x holds for any of the 64 threads of two warps; a barrier for them, too.
__device__ __forceinline__ bool pair_any(int id, bool x) {
    int got;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 64, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(got)
        : "r"(id), "r"((int)x)
        : "memory");
    return got != 0;
}

// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 apart(uint64_t d) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(d));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// ------------------------------------------------------------------ work list
// Key tile tj of a sequence: its first position and its rows that hold positions.
struct Tile {
    int p0, rows;
};
__device__ __forceinline__ Tile tile_at(const TreeAttnParams &p, int tj, int total) {
    Tile t;
    int span;
    if (p.ppt) {
        span = p.ppt * p.page_size;
        t.p0 = tj * span;
    } else {
        const int pg = tj / p.tpp, r0 = (tj - pg * p.tpp) * kTrKeys;
        t.p0 = pg * p.page_size + r0;
        span = min(kTrKeys, p.page_size - r0);
    }
    t.rows = min(span, total - t.p0);
    return t;
}
__device__ __forceinline__ int tiles_of(const TreeAttnParams &p, int total) {
    if (p.ppt) {
        const int span = p.ppt * p.page_size;
        return (total + span - 1) / span;
    }
    const int full = total / p.page_size;
    return full * p.tpp + (total - full * p.page_size + kTrKeys - 1) / kTrKeys;
}

// A sequence as the roles see it.
struct Seq {
    int len, nodes, total, tiles, blocks;   // blocks: pairs of row tiles (one: a single tile)
};
template <int RT>
__device__ __forceinline__ Seq seq_at(const TreeAttnParams &p, int b) {
    Seq s;
    const int cap = p.page_size * p.max_pages;
    s.len = tr_clamp(checked(ld_dep(p.len + b), 0, cap, p.err), cap);
    s.nodes = p.n_nodes ? tr_clamp(checked(ld_dep(p.n_nodes + b), 0, p.n, p.err), p.n) : p.n;
    s.total = s.nodes ? (s.nodes > cap - s.len ? cap : s.len + s.nodes) : 0;
    s.tiles = tiles_of(p, s.total);
    s.blocks = (s.nodes + RT * p.NB - 1) / (RT * p.NB);
    return s;
}

// A run of tiles of one (sequence, KV head, row block).
struct Run {
    int b, h, rb, t0, cnt;
    Seq s;
};

// Walks a CTA's part of the list; every role has its own.
template <int RT>
struct Walk {
    int b, off;             // off: tiles of sequence b already passed, over its heads and blocks
    long long left;
    Seq s;
    __device__ __forceinline__ void start(const TreeAttnParams &p, int b0, int off0, long long n) {
        b = b0;
        off = off0;
        left = n;
        if (left > 0) s = seq_at<RT>(p, b);
    }
    __device__ __forceinline__ bool next(const TreeAttnParams &p, Run &r) {
        if (left <= 0) return false;
        while (off >= s.tiles * s.blocks * p.H_kv) {
            if (++b >= p.B) return false;
            off = 0;
            s = seq_at<RT>(p, b);
        }
        const int item = off / s.tiles;
        r.b = b;
        r.s = s;
        r.h = item / s.blocks;
        r.rb = item - r.h * s.blocks;
        r.t0 = off - item * s.tiles;
        r.cnt = (int)min((long long)(s.tiles - r.t0), left);
        off += r.cnt;
        left -= r.cnt;
        return true;
    }
};

template <int D, int RT>
struct TrSmem {
    static constexpr int HALVES = D / 64;
    static constexpr int OPER = HALVES * kTrBox;                         // a K or V tile, or a row tile of Q
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr int XCH = 2 * 2 * 128 * 4 + (RT == 1 ? 2 * 128 * 4 : 0);
    static constexpr int BYTES = RT * OPER + STAGES * OPER + 2 * kTrMaxNodes + XCH + (2 * STAGES + 9) * 8 + 16;
};

// Position in the ring of the K and V tile j of a run of cnt.  With one row tile the
// products are issued K0 K1 | V0 K2 | V1 K3 | ..., with two K0 | V0 K1 | V1 K2 ...
template <int RT>
__device__ __forceinline__ int ring_k(int j, int) { return RT == 1 ? (j < 2 ? j : 2 * j - 1) : 2 * j; }
template <int RT>
__device__ __forceinline__ int ring_v(int j, int cnt) { return RT == 1 ? min(2 * j + 2, cnt + j) : 2 * j + 1; }

// Bounded wait.  The clock is read only now and then: a read takes as long as the whole
// wait does on the path from one product to the next (both sides measured: 32 trees of 64
// nodes over 32k).
__device__ __forceinline__ bool tr_poll(uint64_t *bar, uint32_t parity, int *err) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; i < kMaxPolls; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 1023u) == 0) {
            const uint64_t t = globaltimer();
            if (t0 == 0) t0 = t;
            else if (t - t0 > kMaxWaitNs) break;
        }
    }
    raise_error(err, kErrTimeout);
    return false;
}

// Lane 0 waits and the warp agrees on the outcome; once a wait has given up, the later
// ones return at once.
__device__ __forceinline__ bool tr_wait(uint64_t *bar, uint32_t parity, int *err, bool ok, int lane) {
    int got = ok ? 1 : 0;
    if (ok && lane == 0) got = tr_poll(bar, parity, err) ? 1 : 0;
    return __shfl_sync(0xffffffffu, got, 0) != 0;
}

template <int D, int RT>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const TreeAttnParams p) {
    using L = TrSmem<D, RT>;
    constexpr int HALVES = L::HALVES, OPER = L::OPER, NST = L::STAGES, KS = D / 16;
    extern __shared__ __align__(1024) uint8_t smem[];      // swizzled tiles start at multiples of 1024
    uint8_t *qbuf = smem, *ring = smem + RT * OPER;
    uint8_t *par = ring + NST * OPER;                                    // [2][kTrMaxNodes]
    float *xch = reinterpret_cast<float *>(par + 2 * kTrMaxNodes);       // [stream][half][128]
    float *xmax = xch + 2 * 2 * 128;                                     // [stream][128], one row tile only
    uint64_t *full = reinterpret_cast<uint64_t *>(par + 2 * kTrMaxNodes + L::XCH);
    uint64_t *empty = full + NST;
    uint64_t *q_full = empty + NST, *q_empty = q_full + 1;
    uint64_t *s_full = q_empty + 1, *p_full = s_full + 2, *o_full = p_full + 2;   // [2] each
    uint64_t *mma_done = o_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    int *found = reinterpret_cast<int *>(tmem_slot + 1);                 // b0, off0, run length
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(smem) & 1023u) {
        if (tid == 0) raise_error(p.err, kErrState);
        pdl_wait();
        return;
    }

    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(mma_done, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 8);
            mbar_init(&o_full[s], 1);
        }
        mbar_fence_init();
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        found[2] = 0;
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    pdl_trigger();
    pdl_wait();

    // The list of work: prefix sums over the sequences, this CTA's run of tiles, and the
    // sequence that it begins in.
    {
        long long *wsum = reinterpret_cast<long long *>(par);
        const int per = (p.B + kTrThreads - 1) / kTrThreads;
        const int ba = min(p.B, tid * per), bz = min(p.B, ba + per);
        long long mine = 0;
        for (int b = ba; b < bz; ++b) {
            const Seq s = seq_at<RT>(p, b);
            mine += (long long)s.tiles * s.blocks * p.H_kv;
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        long long before = incl - mine, all = 0;
        for (int w = 0; w < kTrThreads / 32; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        const long long run = max(1ll, (all + p.grid - 1) / p.grid);
        const long long t0 = blockIdx.x * run;
        for (int b = ba; b < bz; ++b) {
            const Seq s = seq_at<RT>(p, b);
            const long long w = (long long)s.tiles * s.blocks * p.H_kv;
            if (blockIdx.x == 0) p.seq[b] = TreeSeq{before, s.tiles, s.nodes};
            if (t0 >= before && t0 < before + w) {
                found[0] = b;
                found[1] = (int)(t0 - before);
                found[2] = (int)min(run, all - t0);
            }
            before += w;
        }
        if (blockIdx.x == 0 && tid == 0) p.seq[p.B] = TreeSeq{run, 0, 0};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk<RT> walk;
    walk.start(p, found[0], found[1], found[2]);
    Run r;
    bool ok = true;

    if (warp < 4 && warp != 1) {
        regs_give();
        // ------------------------------------------------------------ TMA producers
        // Three warps, every third slot of the ring each: a box of the lanes' loop takes 60
        // cycles to issue, which with small pages is as long as its data need.
        const uint32_t pw = warp == 0 ? 0 : warp - 1;
        const uint64_t pol = p.n > RT * p.NB ? policy_evict_normal() : policy_evict_first();
        uint32_t slot = 0, runs = 0;                 // ring slots issued, runs begun
        while (walk.next(p, r)) {
            const int tiles_q = RT == 2 && r.rb * 2 * p.NB + p.NB < r.s.nodes ? 2 : 1;
            if (pw == 0) ok = tr_wait(q_empty, (runs & 1) ^ 1, p.err, ok, lane);
            if (!ok) break;
            if (pw == 0 && lane == 0) {
                mbar_arrive_expect_tx(q_full, (uint32_t)(tiles_q * HALVES * p.NB * p.G * 128));
                for (int t = 0; t < tiles_q; ++t)
                    for (int hf = 0; hf < HALVES; ++hf)
                        tma_load_4d(qbuf + t * OPER + hf * kTrBox, &tmq, hf * 64, r.h * p.G, (r.rb * RT + t) * p.NB, r.b,
                                    q_full, policy_evict_normal());
            }
            ++runs;
            const int32_t *table = p.table + (long long)r.b * p.max_pages;
            // K and V boxes in the order of the products.
            for (int i = 0; i < 2 * r.cnt; ++i, ++slot) {
                if (slot % 3 != pw) continue;
                int j, is_v;
                if (RT == 1) {
                    if (i < 2 && i < r.cnt) { j = i; is_v = 0; }
                    else if (r.cnt == 1) { j = 0; is_v = 1; }
                    else if (i >= 2 * r.cnt - 2) { j = i - r.cnt; is_v = 1; }
                    else { is_v = (i & 1) == 0; j = is_v ? (i - 2) / 2 : (i + 1) / 2; }
                } else {
                    j = i >> 1;
                    is_v = i & 1;
                }
                const Tile t = tile_at(p, r.t0 + j, r.s.total);
                const uint32_t st = slot % NST, ph = (slot / NST) & 1;
                uint8_t *dst = ring + st * OPER;
                const int pg0 = t.p0 / p.page_size;
                // Boxes of br rows: a page each, or parts of one page.  The lane's page number is
                // on its way while the warp waits for the ring.
                const int boxes = (t.rows + p.br - 1) / p.br, r0 = t.p0 - pg0 * p.page_size;
                const bool pages = p.br == p.page_size;
                int id = lane < boxes ? ld_dep(table + pg0 + (pages ? lane : 0)) : 0;
                ok = tr_wait(&empty[st], ph ^ 1, p.err, ok, lane);
                if (!ok) break;
                const CUtensorMap *tm = is_v ? &tmv : &tmk;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(boxes * p.br * HALVES * 128));
                __syncwarp();
                for (int g = lane; g < boxes; g += 32) {
                    if (g >= 32) id = ld_dep(table + pg0 + (pages ? g : 0));
                    if (id < 0 || id >= p.n_pages) {       // such a page is filled with zeros
                        raise_error(p.err, kErrPage);
                        id = p.n_pages;
                    }
                    const int at = g * p.br, pr = pages ? 0 : r0 + at;      // row in the tile, in the page
                    if (p.by8)
                        tma_load_5d(dst + at / 8 * (HALVES * 1024), tm, 0, 0, r.h * HALVES, pr / 8, id, &full[st], pol);
                    else
                        for (int hf = 0; hf < HALVES; ++hf)
                            tma_load_4d(dst + hf * kTrBox + at * 128, tm, hf * 64, r.h, pr, id, &full[st], pol);
                }
            }
            if (!ok) break;
        }
        // No copy may be in flight when the CTA ends.
        __syncwarp();
        if (lane == 0) {
            if (pw == 0 && runs) mbar_wait(q_full, (runs - 1) & 1, p.err);
            const uint32_t last = min(slot, (uint32_t)NST);
            for (uint32_t i = slot - last; i < slot; ++i)
                if (i % 3 == pw) mbar_wait(&full[i % NST], (i / NST) & 1, p.err);
        }
    } else if (warp == 1) {
        regs_give();
        // -------------------------------------------------------------- MMA issuer
        const uint32_t idesc_s = umma_idesc_bf16(128, kTrKeys);
        const uint32_t idesc_o = umma_idesc_bf16(128, D) | (1u << 16);   // B (V) is MN-major
        const uint32_t qb = smem_u32(qbuf), rb0 = smem_u32(ring);
        uint32_t slot0 = 0, runs = 0, done[2] = {0, 0};                  // done: tiles of each stream

        const uint64_t kdesc = desc_k(rb0, p.sbo), vdesc = desc_v(rb0, p.sbo, p.hoff), qdesc = umma_desc_sw128(qb);
        const uint32_t khalf = p.hoff >> 4, vstep = 2 * p.sbo >> 4;      // descriptor units of 16 bytes
        auto stage = [&](uint32_t slot) {                                // of a ring slot, in the same units
            return (uint64_t)__shfl_sync(0xffffffffu, (slot % NST) * (OPER >> 4), 0);
        };
        auto scores = [&](int s, uint32_t slot) {                        // S_s = Q K^T
            const uint64_t k = kdesc + stage(slot), q = qdesc + (RT == 2 ? s : 0) * (OPER >> 4);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    umma_bf16(tmem + s * 128, q + (ks >> 2) * (kTrBox >> 4) + (ks & 3) * 2,
                              k + (ks >> 2) * khalf + (ks & 3) * 2, idesc_s, ks > 0);
                umma_commit(&s_full[s]);
            }
            __syncwarp();
        };
        auto values = [&](int s, uint32_t slot, int rows, bool first) {  // O_s (+)= P V
            const uint64_t v = vdesc + stage(slot);
            const uint32_t o = tmem + kTrOut + s * D, a = tmem + s * 128;
            if (elect_one()) {
                if (rows > kTrKeys - 16) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_bf16_ts(o, a + ks * 8, v + ks * vstep, idesc_o, ks > 0 || !first);
                } else {
                    for (int ks = 0; ks * 16 < rows; ++ks)
                        umma_bf16_ts(o, a + ks * 8, v + ks * vstep, idesc_o, ks > 0 || !first);
                }
                umma_commit(&o_full[s]);
            }
            __syncwarp();
        };
        auto release = [&](uint32_t slot) {
            const uint32_t st = __shfl_sync(0xffffffffu, slot % NST, 0);
            if (elect_one()) umma_commit(&empty[st]);
            __syncwarp();
        };
        auto arrived = [&](uint32_t slot) {
            ok = tr_wait(&full[slot % NST], (slot / NST) & 1, p.err, ok, lane);
            tc_fence_after();
        };
        // Rows of V behind the sequence's last position may hold anything, and 0 * NaN is
        // NaN: those that the last step of 16 keys still reads are set to zero.
        auto clear_tail = [&](uint32_t slot, int rows) {
            const int end = (rows + 15) & ~15;
            if (rows == end) return;
            uint8_t *v = ring + (slot % NST) * OPER;
            for (int i = lane; i < HALVES * (end - rows) * 8; i += 32) {
                const int hf = i / ((end - rows) * 8), e = i - hf * (end - rows) * 8;
                const int row = rows + e / 8;
                *reinterpret_cast<uint4 *>(v + hf * p.hoff + (row >> 3) * p.sbo + (row & 7) * 128 + (e & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        while (ok && walk.next(p, r)) {
            ok = tr_wait(q_full, runs & 1, p.err, ok, lane);
            tc_fence_after();
            ++runs;
            const bool second = RT == 2 && r.rb * 2 * p.NB + p.NB < r.s.nodes;
            const int cnt = r.cnt;
            if (RT == 1) {
                for (int j = 0; j < 2 && j < cnt && ok; ++j) {
                    arrived(slot0 + ring_k<RT>(j, cnt));
                    if (!ok) break;
                    scores(j, slot0 + ring_k<RT>(j, cnt));
                    release(slot0 + ring_k<RT>(j, cnt));
                }
                if (cnt <= 2 && elect_one()) umma_commit(q_empty);
                for (int j = 0; j < cnt && ok; ++j) {
                    const int s = j & 1;
                    const uint32_t vs = slot0 + ring_v<RT>(j, cnt);
                    const int rows = tile_at(p, r.t0 + j, r.s.total).rows;
                    arrived(vs);
                    if (ok) clear_tail(vs, rows);
                    ok = tr_wait(&p_full[s], done[s] & 1, p.err, ok, lane);
                    tc_fence_after();
                    if (!ok) break;
                    values(s, vs, rows, j < 2);
                    ++done[s];
                    release(vs);
                    if (j + 2 < cnt) {
                        const uint32_t ks = slot0 + ring_k<RT>(j + 2, cnt);
                        arrived(ks);
                        if (!ok) break;
                        scores(s, ks);
                        release(ks);
                        if (j + 3 == cnt && elect_one()) umma_commit(q_empty);
                    }
                }
            } else {
                arrived(slot0);
                if (!ok) break;
                scores(0, slot0);
                if (second) scores(1, slot0);
                release(slot0);
                if (cnt == 1 && elect_one()) umma_commit(q_empty);
                for (int j = 0; j < cnt && ok; ++j) {
                    const uint32_t vs = slot0 + ring_v<RT>(j, cnt), ks = slot0 + ring_k<RT>(j + 1, cnt);
                    const int rows = tile_at(p, r.t0 + j, r.s.total).rows;
                    arrived(vs);
                    if (ok) clear_tail(vs, rows);
                    for (int s = 0; s < (second ? 2 : 1) && ok; ++s) {
                        ok = tr_wait(&p_full[s], done[s] & 1, p.err, ok, lane);
                        tc_fence_after();
                        if (!ok) break;
                        values(s, vs, rows, j == 0);
                        ++done[s];
                        if (j + 1 < cnt) {
                            if (s == 0) arrived(ks);
                            if (!ok) break;
                            scores(s, ks);
                        }
                    }
                    if (!ok) break;
                    release(vs);
                    if (j + 1 < cnt) {
                        release(ks);
                        if (j + 2 == cnt && elect_one()) umma_commit(q_empty);
                    }
                }
            }
            slot0 += 2 * cnt;
        }
        // The products in flight end before the shared memory and TMEM that they use go.
        __syncwarp();
        if (elect_one()) {
            umma_commit(mma_done);
            mbar_wait(mma_done, 0, p.err);
        }
    } else {
        regs_take();
        // -------------------------------------------------------- softmax warpgroups
        const int s = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;    // stream, half of a tile's keys
        const int quad = warp & 3;                                      // TMEM lanes 32 * quad ..
        const int row = 32 * quad + lane;
        const int pair_bar = 1 + s * 4 + quad;                          // the two warps of 32 rows
        const uint32_t lane_addr = (uint32_t)(32 * quad) << 16;
        const uint32_t ts = tmem + lane_addr + s * 128, to = tmem + lane_addr + kTrOut + s * D;
        const int wt = tid - 128 - s * 256;                             // thread of the stream
        const int node_r = row / p.G;                                   // node within the row tile
        const float sl = p.scale_log2;
        uint8_t *mypar = par + s * kTrMaxNodes;
        float *mine_x = xch + (s * 2 + half) * 128 + row, *other_x = xch + (s * 2 + 1 - half) * 128 + row;
        uint32_t tiles_done = 0;
        int par_b = -1;
        bool first_run = true;
        while (walk.next(p, r)) {
            const int base = (r.rb * RT + (RT == 2 ? s : 0)) * p.NB;      // first node of the row tile
            const int node = node_r < p.NB && base + node_r < r.s.nodes ? base + node_r : -1;
            const bool active = RT == 1 || base < r.s.nodes;
            const bool live = __any_sync(0xffffffffu, node >= 0);         // the warp has rows
            if (p.parent && par_b != r.b) {
                // parent + 1 of every node in a byte (0: none); a parent that is not before its
                // node counts as none.
                named_bar_sync(9 + s, 256);
                if (wt < r.s.nodes) {
                    const int pi = checked(ld_dep(p.parent + (long long)r.b * p.n + wt), -1, wt - 1, p.err);
                    mypar[wt] = (uint8_t)(pi >= 0 && pi < wt ? pi + 1 : 0);
                }
                named_bar_sync(9 + s, 256);
                par_b = r.b;
            }
            float m = -INFINITY, l = 0.f;                    // m: of the row, l: of this half's keys
            int mine = 0;                                    // tiles of this run that this stream had
            for (int j = RT == 1 ? s : 0; active && j < r.cnt; j += RT == 1 ? 2 : 1) {
                const Tile t = tile_at(p, r.t0 + j, r.s.total);
                ok = tr_wait(&s_full[s], tiles_done & 1, p.err, ok, lane);
                tc_fence_after();
                if (live) {
                    uint32_t v[64];
                    tmem_ld64(ts + half * 64, v);
                    if (t.rows < kTrKeys || t.p0 + t.rows > r.s.len) {
                        const int k0 = t.p0 + half * 64;                  // position of this half's first key
                        const int rows = t.rows - half * 64;
                        uint32_t see[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int c = min(r.s.len - k0, rows) - 32 * k;
                            see[k] = node < 0 || c <= 0 ? 0u : c >= 32 ? 0xffffffffu : (1u << c) - 1u;
                        }
                        if (node >= 0 && k0 + rows > r.s.len) {
                            for (int a = node; a >= 0; a = p.parent ? (int)mypar[a] - 1 : a - 1) {
                                const int off = r.s.len + a - k0;
                                if (off < 0) break;                       // ancestors come before their nodes
                                if (off < rows && off < 64) {
                                    if (off < 32) see[0] |= 1u << off;
                                    else see[1] |= 1u << (off - 32);
                                }
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (__all_sync(0xffffffffu, see[k] == 0xffffffffu)) continue;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!((see[k] >> c) & 1u)) v[32 * k + c] = 0xff800000u;
                        }
                    }
                    // Four chains, so that one maximum does not wait for the last.
                    float t4[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) t4[c] = __uint_as_float(v[c]);
#pragma unroll
                    for (int c = 4; c < 60; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            t4[i] = fmaxf(t4[i], fmaxf(__uint_as_float(v[c + i]), __uint_as_float(v[c + 4 + i])));
#pragma unroll
                    for (int i = 0; i < 4; ++i) t4[i] = fmaxf(t4[i], __uint_as_float(v[60 + i]));
                    float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                    // The maximum is moved, and O scaled, only where it has grown by more than
                    // 2^kTrLazy: sums then stay below 2^kTrLazy * keys, far inside fp32.  Both
                    // halves of a row have to agree; the barrier also puts the loads of S by
                    // both before the stores of P over it.
                    float f = 1.f;
                    if (pair_any(pair_bar, top > m && (top - m) * sl > kTrLazy)) {
                        *mine_x = top;
                        named_bar_sync(pair_bar, 64);
                        top = fmaxf(top, *other_x);
                        if (top > m && (top - m) * sl > kTrLazy) {
                            f = m == -INFINITY ? 1.f : fast_exp2((m - top) * sl);   // from -inf: O and l are zero
                            m = top;
                        }
                        if (mine > 0) {
                            ok = tr_wait(&o_full[s], (tiles_done - 1) & 1, p.err, ok, lane);
                            tc_fence_after();
#pragma unroll 1
                            for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 16) {
                                uint32_t o[16];
                                tmem_ld16(to + c0, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st16(to + c0, o);
                            }
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m * sl;
                    const uint64_t sl2 = pair(sl, sl), ms2 = pair(-ms, -ms);
                    uint64_t sum2[2] = {0, 0};
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = apart(fma2(pair(v[c0 + 2 * i], v[c0 + 2 * i + 1]), sl2, ms2));
                            const float a = fast_exp2(x.x), b = fast_exp2(x.y);
                            sum2[i & 1] = add2(sum2[i & 1], pair(a, b));
                            u[i] = pack_bf16(a, b);
                        }
                        tmem_st16(ts + half * 32 + c0 / 2, u);
                    }
                    const float2 sum = apart(add2(sum2[0], sum2[1]));
                    l = l * f + (sum.x + sum.y);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
                ++tiles_done;
                ++mine;
            }
            // The end of the run: O / l if the run is the whole list entry, else a partial.
            if (mine > 0) ok = tr_wait(&o_full[s], (tiles_done - 1) & 1, p.err, ok, lane);
            const int part = 2 * blockIdx.x + (first_run ? 0 : 1);
            first_run = false;
            // The halves' sums, and with one row tile both streams' maxima: each warp then
            // joins what it needs for its share of the channels.
            if (RT == 1) {
                named_bar_sync(11, 512);
                *mine_x = l;
                if (half == 0) xmax[s * 128 + row] = m;
                tc_fence_before();
                named_bar_sync(11, 512);
            } else {
                named_bar_sync(pair_bar, 64);
                *mine_x = l;
                named_bar_sync(pair_bar, 64);
            }
            tc_fence_after();
            float w0 = 1.f, w1 = 0.f, mm = m, ll;
            if (RT == 1) {
                const float m0 = xmax[row], m1 = r.cnt > 1 ? xmax[128 + row] : -INFINITY;
                mm = fmaxf(m0, m1);
                const float mu = mm == -INFINITY ? 0.f : mm;
                w0 = fast_exp2((m0 - mu) * sl);
                w1 = fast_exp2((m1 - mu) * sl);
                ll = w0 * (xch[row] + xch[128 + row]);
                if (r.cnt > 1) ll += w1 * (xch[256 + row] + xch[384 + row]);
            } else {
                ll = xch[s * 256 + row] + xch[s * 256 + 128 + row];
            }
            const bool whole = r.cnt == r.s.tiles;
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
            uint16_t *dst = p.out + (((long long)r.b * p.n + node) * p.H_q + r.h * p.G + (row - node_r * p.G)) * D;
            const int rt = RT == 2 ? s : 0;
            float4 *pd = p.part + ((long long)part * RT + rt) * (D / 4) * 128 + row;
            constexpr int SHARE = RT == 1 ? D / 4 : D / 2;               // channels of a warp
            const int c_lo = RT == 1 ? (s * 2 + half) * SHARE : half * SHARE;
#pragma unroll 1
            for (int c0 = c_lo; live && c0 < c_lo + SHARE; c0 += 16) {
                uint32_t o[16];
                float x[16];
                tmem_ld16((RT == 1 ? tmem + lane_addr + kTrOut : to) + c0, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = w0 * __uint_as_float(o[i]);
                if (RT == 1 && r.cnt > 1) {
                    tmem_ld16(tmem + lane_addr + kTrOut + D + c0, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] += w1 * __uint_as_float(o[i]);
                }
                if (node < 0) continue;
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        uint4 y;
                        y.x = pack_bf16(x[i] * inv, x[i + 1] * inv);
                        y.y = pack_bf16(x[i + 2] * inv, x[i + 3] * inv);
                        y.z = pack_bf16(x[i + 4] * inv, x[i + 5] * inv);
                        y.w = pack_bf16(x[i + 6] * inv, x[i + 7] * inv);
                        *reinterpret_cast<uint4 *>(dst + c0 + i) = y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        pd[(c0 + i) / 4 * 128] = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                }
            }
            if (!whole && node >= 0 && c_lo == 0)
                p.stat[(long long)part * RT * 128 + rt * 128 + row] = make_float2(mm, ll);
            tc_fence_before();
            // O is free for the next run, whose first P says so: with one row tile, once all
            // warps have read both.
            if (RT == 1) named_bar_sync(11, 512);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ the joining
// One thread: four channels of one row, over the CTAs that had a run of its list
// entry, in the order of the list.  Rows that belong to no entry (nodes past the
// sequence's count) are set to zero.
constexpr int kTjThreads = 256;

template <int RT>
__global__ void __launch_bounds__(kTjThreads) tree_attn_join_kernel(const TreeAttnParams p, int D) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, h = blockIdx.y;
    const int R = p.n * p.G;
    const int it = blockIdx.x * kTjThreads + threadIdx.x;
    if (it >= R * (D / 4)) return;
    const int c4 = it / R, gr = it - c4 * R;
    const int node = gr / p.G, g = gr - node * p.G;
    const TreeSeq s = p.seq[b];
    uint2 *dst = reinterpret_cast<uint2 *>(p.out + (((long long)b * p.n + node) * p.H_q + h * p.G + g) * D) + c4;
    if (node >= s.nodes || s.tiles == 0) {
        *dst = make_uint2(0, 0);
        return;
    }
    const long long run = p.seq[p.B].first;
    const int blocks = (s.nodes + RT * p.NB - 1) / (RT * p.NB);
    const int tile = node / p.NB, rb = tile / RT, rt = tile - rb * RT;
    const long long t0 = s.first + (long long)(h * blocks + rb) * s.tiles, t1 = t0 + s.tiles - 1;
    const int c0 = (int)(t0 / run), c1 = (int)(t1 / run);
    if (c0 == c1) return;                              // one CTA had it whole and wrote it
    const int row = (node - tile * p.NB) * p.G + g;
    const int first = 2 * c0 + (t0 == c0 * run ? 0 : 1);
    const float sl = p.scale_log2;
    const long long srow = rt * 128 + row;
    float top = p.stat[(long long)first * RT * 128 + srow].x;
    for (int c = c0 + 1; c <= c1; ++c) top = fmaxf(top, p.stat[(long long)2 * c * RT * 128 + srow].x);
    const float mu = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
        const long long slot = c == c0 ? first : 2 * c;
        const float2 e = p.stat[slot * RT * 128 + srow];
        const float4 o = p.part[((slot * RT + rt) * (D / 4) + c4) * 128 + row];
        const float w = fast_exp2((e.x - mu) * sl);
        sum += w * e.y;
        acc.x += w * o.x;
        acc.y += w * o.y;
        acc.z += w * o.z;
        acc.w += w * o.w;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    *dst = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// ------------------------------------------------------------------- host side
static size_t tr_align(size_t x) { return (x + 255) & ~(size_t)255; }

static int tr_row_tiles(int n, int G) { return n <= 128 / G ? 1 : 2; }

size_t tree_attn_workspace_bytes(const magicdec_paged_shape &s, int n) {
    const int RT = tr_row_tiles(n, s.H_q / s.H_kv);
    const size_t slots = 2 * (size_t)magicdec_host::sm_count();
    return tr_align(((size_t)s.B + 1) * sizeof(TreeSeq)) + tr_align(slots * RT * 128 * sizeof(float2)) +
           slots * RT * 128 * s.d * 4;
}

template <int D, int RT>
static magicdec_status launch_tree_t(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                     const TreeAttnParams &p, cudaStream_t st) {
    auto kern = tree_attn_kernel<D, RT>;
    constexpr int smem = TrSmem<D, RT>::BYTES;
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return MAGICDEC_ERR_CUDA;
    magicdec_status s =
        magicdec_host::launch_pdl(kern, dim3((unsigned)p.grid), dim3(kTrThreads), smem, st, tmq, tmk, tmv, p);
    if (s != MAGICDEC_OK) return s;
    const int items = p.n * p.G * (D / 4);
    return magicdec_host::launch_pdl(tree_attn_join_kernel<RT>,
                                     dim3((unsigned)((items + kTjThreads - 1) / kTjThreads), (unsigned)p.H_kv,
                                          (unsigned)p.B),
                                     dim3(kTjThreads), 0, st, p, D);
}

magicdec_status launch_tree_attn(const magicdec_paged_shape &s, int n, const uint16_t *q, const uint16_t *kp,
                                 const uint16_t *vp, const int32_t *table, const int32_t *len, const int32_t *n_nodes,
                                 const int32_t *parent, uint16_t *out, void *ws, cudaStream_t st) {
    TreeAttnParams p{};
    p.len = len;
    p.n_nodes = n_nodes;
    p.parent = parent;
    p.table = table;
    p.out = out;
    p.err = magicdec_host::device_error_word();
    p.B = s.B;
    p.H_q = s.H_q;
    p.H_kv = s.H_kv;
    p.G = s.H_q / s.H_kv;
    p.n = n;
    p.page_size = s.page_size;
    p.n_pages = s.n_pages;
    p.max_pages = s.max_pages;
    p.NB = 128 / p.G;
    p.ppt = s.page_size <= kTrKeys ? kTrKeys / s.page_size : 0;
    p.tpp = (s.page_size + kTrKeys - 1) / kTrKeys;
    p.scale_log2 = kLog2e / sqrtf((float)s.d);
    p.grid = magicdec_host::sm_count();
    const int RT = tr_row_tiles(n, p.G);
    const size_t slots = 2 * (size_t)p.grid;
    uint8_t *w = static_cast<uint8_t *>(ws);
    p.seq = reinterpret_cast<TreeSeq *>(w);
    w += tr_align(((size_t)s.B + 1) * sizeof(TreeSeq));
    p.stat = reinterpret_cast<float2 *>(w);
    w += tr_align(slots * RT * 128 * sizeof(float2));
    p.part = reinterpret_cast<float4 *>(w);

    // Queries as (d, H_q, n, B), one box = NB nodes of a KV head's group.  The pool with
    // pages of a multiple of 8 rows as (64 channels, 8 rows, halves of all heads, groups of 8
    // rows, pages): one box is a page (or 128 rows of it) of one KV head, its channels read
    // together and its rows laid out for the tensor cores.  Other pages as (d, H_kv,
    // page_size, n_pages), boxes of 64 channels x a page (or 128 rows).
    CUtensorMap tmq, tmk, tmv;
    const int D = s.d, HV = D / 64;
    p.by8 = s.page_size % 8 == 0;
    p.sbo = p.by8 ? HV * 1024 : 1024;
    p.hoff = p.by8 ? 1024 : kTrBox;
    const uint64_t row = (uint64_t)s.H_kv * D * 2;
    p.br = s.page_size < kTrKeys ? s.page_size : kTrKeys;
    const uint32_t span = (uint32_t)p.br;
    const uint64_t kd4[4] = {(uint64_t)D, (uint64_t)s.H_kv, (uint64_t)s.page_size, (uint64_t)s.n_pages};
    const uint64_t ks4[3] = {(uint64_t)D * 2, row, s.page_size * row};
    const uint32_t kb4[4] = {64, 1, span, 1};
    const uint64_t kd5[5] = {64, 8, (uint64_t)s.H_kv * HV, (uint64_t)s.page_size / 8, (uint64_t)s.n_pages};
    const uint64_t ks5[4] = {row, 128, 8 * row, s.page_size * row};
    const uint32_t kb5[5] = {64, 8, (uint32_t)HV, span / 8, 1};
    const uint64_t qd[4] = {(uint64_t)D, (uint64_t)s.H_q, (uint64_t)n, (uint64_t)s.B};
    const uint64_t qs[3] = {(uint64_t)D * 2, (uint64_t)s.H_q * D * 2, (uint64_t)n * s.H_q * D * 2};
    const uint32_t qbx[4] = {64, (uint32_t)p.G, (uint32_t)p.NB, 1};
    auto pool = [&](CUtensorMap *m, const uint16_t *x) {
        return p.by8 ? magicdec_host::encode_tmap_bf16(m, x, 5, kd5, ks5, kb5)
                     : magicdec_host::encode_tmap_bf16(m, x, 4, kd4, ks4, kb4);
    };
    if (!pool(&tmk, kp) || !pool(&tmv, vp) || !magicdec_host::encode_tmap_bf16_4d(&tmq, q, qd, qs, qbx))
        return MAGICDEC_ERR_CUDA;
    if (D == 128)
        return RT == 1 ? launch_tree_t<128, 1>(tmq, tmk, tmv, p, st) : launch_tree_t<128, 2>(tmq, tmk, tmv, p, st);
    return RT == 1 ? launch_tree_t<64, 1>(tmq, tmk, tmv, p, st) : launch_tree_t<64, 2>(tmq, tmk, tmv, p, st);
}

}  // namespace magicdec
