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
// keys (a thread: one row, 32 keys at a time):
//   one row tile  (n <= NB): the streams take the even and odd key tiles, so one
//     softmax runs while the other's products do; their O are merged at the end;
//   two row tiles (n > NB):  each stream owns a row tile and sees every key tile;
//     K and V are read once for both (further pairs of tiles: other work items).
// A stream's S is in two parts of 64 keys, so that the scores of one are computed
// while the softmax is at the other.  P overwrites S's columns as bf16 (the A operand
// of the second product comes from TMEM).  P in bf16 is off by at most 2^-8 relative, as the
// rounding of the output; sums, maxima and O are fp32.
//
// Work: the key tiles of all (sequence, KV head, row block), as one list, cut
// into equal runs of tiles, one per CTA; what a CTA has of a list entry that it
// does not own whole goes to the workspace as (O, max, sum) and is joined by a
// second kernel in a fixed order.  No atomics: results do not change from run to run.
//
// Behind shared prefixes (template parameter PRE) the list begins with the prefixes: an entry
// "sequence" of which the rows of all sequences of a group are the nodes, B n G rows a KV
// head, so that a prefix's K and V are read once for a row block of any of them.  Every entry's
// part goes to the workspace.  Own slots of up to 32 query rows are the work of another kernel, which
// joins a row's parts (prefix_own.cu); those of more follow in the list, and a joining kernel here
// puts the parts together.
//
// Roles (640 threads): warps 0 and 3 issue the TMA boxes, warps 1 and 2 the MMAs, warps
// 4-11 and 12-19 are the softmax of the two streams.  Every wait is bounded; after one that
// gave up (error 1) the roles run on without waiting, so that all of them end.
#include <climits>

#include "prefix.cuh"
#include "tc.cuh"

namespace magicdec {

constexpr int kTrThreads = 640;
constexpr int kTrKeys = 128;                  // keys per tile
constexpr int kTrBox = kTrKeys * 128;         // 128 rows x 64 channels (16 KB)
constexpr int kTrMaxNodes = 256;
constexpr int kTrOut = 256;                   // first TMEM column of O (S: 0 and 128)
constexpr float kTrLazy = 24.0f;              // log2 growth of a row's maximum that is put up with

// Where a CTA's part of the list begins, for the joining kernel: a list entry, its first
// tile there, its tiles and its sequence's nodes, and the length of a run.
struct TreeStart {
    int b, h, rb, t0, tiles, nodes, run, pad;
};

struct TreeAttnParams {
    const int32_t *len, *n_nodes, *parent, *table;
    const uint16_t *vp;    // the pool of V, for add_back
    uint16_t *out;
    TreeStart *start;      // workspace: [grid]
    float2 *stat;          // workspace: [2 * grid][RT * rr] (max, sum)
    float4 *part;          // workspace: [2 * grid][RT][d / 4][rr]
    int rr;                // rows of a row tile in the workspace
    int *err;
    int B, H_q, H_kv, G, n, page_size, n_pages, max_pages;
    int NB;                // nodes per row tile
    int span;              // keys of a tile, where tiles run on over the pages, else 0
    int tpp;               // key tiles per page, where each page begins with one
    int grid;
    int br;                // rows of a box
    int by4;               // pages of fewer than 4 rows: 4 rows of any pages at a time
    int by8;               // pages of a multiple of 8 rows: copied by 5-D boxes
    uint32_t sbo, hoff;    // bytes between groups of 8 rows, and between 64-channel halves, of a K or V tile
    float scale_log2;      // log2(e) / sqrt(d)
    // PRE only
    PreParts pre;          // the parts of prefixes, in the workspace
    const int32_t *plen, *ptable;
    int pmax;              // pages of a row of ptable
    int own;               // sequences in the list: B, or none where another kernel takes their own slots
    int own_rt, own_blocks;   // of a sequence's own slots: row tiles of a part, blocks at most
};

__device__ __forceinline__ int tr_clamp(int v, int hi) { return v < 0 ? 0 : (v > hi ? hi : v); }

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

__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}

// ------------------------------------------------------------------ work list
// A key tile of a sequence: its first position and its rows that hold positions.
struct Tile {
    int p0, rows;
};
// Walks over key tiles; a division only where it begins.
struct TileWalk {
    int tj, pg, part;       // the tile; with pages of several tiles, its page and its place there
    __device__ __forceinline__ TileWalk(const TreeAttnParams &p, int tj_) : tj(tj_), pg(0), part(0) {
        if (!p.span) {
            pg = tj / p.tpp;
            part = tj - pg * p.tpp;
        }
    }
    __device__ __forceinline__ void step(const TreeAttnParams &p, int n) {
        tj += n;
        if (!p.span)
            for (part += n; part >= p.tpp; part -= p.tpp) ++pg;
    }
    __device__ __forceinline__ Tile at(const TreeAttnParams &p, int total) const {
        Tile t;
        int span;
        if (p.span) {
            span = p.span;
            t.p0 = tj * span;
        } else {
            t.p0 = pg * p.page_size + part * kTrKeys;
            span = min(kTrKeys, p.page_size - part * kTrKeys);
        }
        t.rows = min(span, total - t.p0);
        return t;
    }
};
__device__ __forceinline__ int tiles_of(const TreeAttnParams &p, int total) {
    if (p.span) return (total + p.span - 1) / p.span;
    const int full = total / p.page_size;
    return full * p.tpp + (total - full * p.page_size + kTrKeys - 1) / kTrKeys;
}

// A sequence as the roles see it.
struct Seq {
    int len, nodes, total, tiles, blocks;   // blocks: pairs of row tiles (one: a single tile)
    int row0;                               // PRE: its first row of queries, over all sequences
};
template <int RT, bool PRE>
__device__ __forceinline__ Seq seq_at(const TreeAttnParams &p, int b) {
    Seq s;
    if (PRE) {
        if (b < p.pre.P) {
            const Group g = group_at(p.pre.first, p.B, b, p.err);
            const int most = p.page_size * p.pmax;
            s.row0 = g.lo * p.n;
            s.nodes = max(g.hi - g.lo, 0) * p.n;
            s.len = s.total = s.nodes ? tr_clamp(checked(ld_dep(p.plen + b), 0, most, p.err), most) : 0;
            s.tiles = tiles_of(p, s.total);
            s.blocks = (s.nodes + RT * p.NB - 1) / (RT * p.NB);
            return s;
        }
        b -= p.pre.P;
        s.row0 = b * p.n;
    }
    const int cap = p.page_size * p.max_pages;
    s.len = tr_clamp(checked(ld_dep(p.len + b), 0, cap, p.err), cap);
    s.nodes = p.n_nodes ? tr_clamp(checked(ld_dep(p.n_nodes + b), 0, p.n, p.err), p.n) : p.n;
    s.total = s.nodes ? (s.nodes > cap - s.len ? cap : s.len + s.nodes) : 0;
    s.tiles = tiles_of(p, s.total);
    s.blocks = (s.nodes + RT * p.NB - 1) / (RT * p.NB);
    return s;
}

// The first node of the stretch that ends at node a and in which each one's parent is the
// node before it: the last bit up to a, of which the first node has one.
__device__ __forceinline__ int stretch(const uint32_t *turns, int a) {
    int w = a >> 5;
    uint32_t m = turns[w] & (0xffffffffu >> (31 - (a & 31)));
    while (m == 0 && w > 0) m = turns[--w];
    return m ? w * 32 + 31 - __clz(m) : 0;
}

// The 32 keys that a node sees, as bits: `prefix` of them (or more, or none) lie before the
// nodes' slots, `rows` hold anything; of the nodes' it sees its ancestors and itself.  A
// function of its own, so that its registers are not taken from the tiles that do not call it
// (32 trees of 64 over 32k: 800 us inline, 770 us so).
__device__ __noinline__ uint32_t seen(int prefix, int rows, int node, const uint8_t *par, const uint32_t *turns) {
    const int c = min(prefix, rows);
    uint32_t see = node < 0 || c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
    // A node's ancestors in stretches of neighbours: a chain is a single one.
    const int last = min(rows, 32) - 1;
    for (int a = node; a >= 0;) {
        const int z = par ? stretch(turns, a) : 0;
        const int lo = max(prefix + z, 0), hi = min(prefix + a, last);
        if (lo <= hi) see |= (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
        if (prefix + z <= 0) break;                        // what is further up lies before these keys
        a = par ? (int)par[z] - 1 : -1;
    }
    return see;
}

// A node's V may hold infinities and NaN, of which the nodes that do not see it must have
// nothing; but a masked probability is a product with zero, and 0 * inf is NaN.  So in the tiles
// that hold nodes' slots those values are taken out of shared memory before the product
// (take_out), and a run whose CTA met any adds them, of the nodes that a row does see, to the
// row's sums at its end, from the pool (add_back): a product with a probability above zero is
// the same infinity, or NaN.  What it costs the tiles that are looked through (ragged d = 64,
// 24 sequences of up to 9k: 65.9 -> 67.4 us; chain of 200 over 8k: 225.1 -> 227.6; others nothing) is
// mostly behind the softmax of their first half, while their V arrives.

// Whether either bf16 of a word is not finite: 0x8000 in its place, else 0.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// All bits of the bf16 whose top bit is set in `m`.
__device__ __forceinline__ uint32_t whole_halves(uint32_t m) { return (m >> 15) * 0xffffu; }

// Rows [lo, hi) of a V tile, by the 256 threads of a stream; `met` is set if there were any, before
// they are taken out, so that the other stream, which then does not find them, knows.
template <int HALVES>
__device__ __forceinline__ void take_out(uint8_t *v, int lo, int hi, uint32_t sbo, uint32_t hoff, int thread,
                                         volatile int *met) {
    bool any = false;
#pragma unroll 1
    for (int i = thread; i < (hi - lo) * HALVES * 8; i += 256) {
        const int row = lo + i / (HALVES * 8), c = i % (HALVES * 8);
        uint4 *at = reinterpret_cast<uint4 *>(v + (c >> 3) * hoff + (row >> 3) * sbo + (row & 7) * 128 + (c & 7) * 16);
        uint4 x = *at;
        const uint4 m = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
        if (m.x | m.y | m.z | m.w) {
            *met = 1;
            __threadfence_block();
            x.x &= ~whole_halves(m.x);
            x.y &= ~whole_halves(m.y);
            x.z &= ~whole_halves(m.z);
            x.w &= ~whole_halves(m.w);
            *at = x;
            any = true;
        }
    }
    if (any) fence_proxy_async_smem();
}

// 16 channels, as pairs of bf16: the sum of the values that are not finite over the nodes that
// `node` sees and whose slots lie in [from, to).  A function of its own, as it is hardly ever called.
struct Channels16 {
    uint32_t x[8];
};
__device__ __noinline__ Channels16 add_back(const uint16_t *v, long long stride, const int32_t *table, int page_size,
                                            int n_pages, int len, int from, int to, int node, const uint8_t *par) {
    Channels16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.x[i] = 0;
    for (int a = node; a >= 0; a = par ? (int)par[a] - 1 : a - 1) {
        const int slot = len + a;
        if (slot < from || slot >= to) continue;
        const int pg = slot / page_size, id = table[pg];
        if (id < 0 || id >= n_pages) continue;                 // zeros
        const uint32_t *x =
            reinterpret_cast<const uint32_t *>(v + ((long long)id * page_size + slot - pg * page_size) * stride);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t y = x[i] & whole_halves(not_finite(x[i]));
            r.x[i] = pack_bf16(__uint_as_float(r.x[i] << 16) + __uint_as_float(y << 16),
                               __uint_as_float(r.x[i] & 0xffff0000u) + __uint_as_float(y & 0xffff0000u));
        }
    }
    return r;
}

// What an entry's row block takes of the list.
template <bool PRE>
__device__ __forceinline__ int list_tiles(const Seq &s) {
    return PRE && s.tiles ? s.tiles + kTrEntry : s.tiles;
}

// A run of tiles of one (sequence, KV head, row block).
struct Run {
    int b, h, rb, t0, cnt;
    Seq s;
};

// Walks a CTA's part of the list; every role has its own.
template <int RT, bool PRE>
struct Walk {
    int b, off;             // off: tiles of sequence b already passed, over its heads and blocks
    int left;               // tiles of the run
    Seq s;
    const int *end;         // PRE: the run's part of an entry that it does not finish, which comes first
    __device__ __forceinline__ bool next(const TreeAttnParams &p, Run &r) {
        if (PRE && end) {
            const int n = end[2];
            if (n > kTrEntry) {
                r.b = end[0];
                r.s = Seq{end[3], end[4], end[5], end[6], end[7], end[8]};
                r.h = end[1] / r.s.blocks;
                r.rb = end[1] - r.h * r.s.blocks;
                r.t0 = 0;
                r.cnt = n - kTrEntry;
            }
            end = nullptr;
            if (n > kTrEntry) return true;
        }
        if (left <= 0) return false;
        for (;;) {
            while (off >= list_tiles<PRE>(s) * s.blocks * p.H_kv) {
                if (++b >= (PRE ? p.pre.P + p.own : p.B)) return false;
                off = 0;
                s = seq_at<RT, PRE>(p, b);
            }
            const int tiles = list_tiles<PRE>(s), item = off / tiles;
            r.b = b;
            r.s = s;
            r.h = s.blocks == 1 ? item : item / s.blocks;
            r.rb = item - r.h * s.blocks;
            const int at = off - item * tiles, n = min(tiles - at, left);
            off += n;
            left -= n;
            if (!PRE) {
                r.t0 = at;
                r.cnt = n;
                return true;
            }
            r.t0 = max(at - kTrEntry, 0);
            r.cnt = max(at + n - kTrEntry, 0) - r.t0;
            if (r.cnt > 0) return true;
            if (left <= 0) return false;
        }
    }
};

// Number of an entry's parts: see pre_slot; a sequence's by its own blocks at most.
template <int RT>
__device__ __forceinline__ long long part_slot(const TreeAttnParams &p, int e, int h, int rb, int blocks, int row0) {
    if (e < p.pre.P) return pre_slot(row0, e, h, rb, blocks, p.H_kv, RT * p.NB);
    return ((long long)(e - p.pre.P) * p.H_kv + h) * p.own_blocks + rb;
}

template <int D, int RT>
struct TrSmem {
    static constexpr int HALVES = D / 64;
    static constexpr int OPER = HALVES * kTrBox;                         // a K or V tile, or a row tile of Q
    // Stages of a ring.  With one row tile a ring for each stream, so that a ring has one
    // reader, and stays in order, whichever stream is ahead; else one ring for both, which
    // frees a stage when both have read it.
    static constexpr int RINGS = RT == 1 ? 2 : 1;
    static constexpr int STAGES = (RT == 1 ? 3 : 5) * (D == 128 ? 1 : 2);
    static constexpr int XCH = 2 * 2 * 128 * 4;
    static constexpr int BYTES =
        RT * OPER + RINGS * STAGES * OPER + 2 * kTrMaxNodes + 2 * kTrMaxNodes / 8 + XCH +
        (2 * RINGS * STAGES + 16) * 8 + 80;
};

// A number that a generic lambda takes as a compile-time constant.
template <int N>
struct Const {
    __device__ constexpr operator int() const { return N; }
};

// A warp's wait, with one outcome for all lanes; once a wait has given up, the later ones
// return at once.
__device__ __forceinline__ bool tr_wait(uint64_t *bar, uint32_t parity, int *err, bool ok, int lane) {
    if (__all_sync(0xffffffffu, ok && mbar_try_sleep(bar, parity))) return true;
    int got = ok ? 1 : 0;
    if (ok && lane == 0) got = mbar_poll_on(bar, parity, err) ? 1 : 0;
    return __shfl_sync(0xffffffffu, got, 0) != 0;
}

template <int D, int RT, bool PRE>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmg,
                     const TreeAttnParams p) {
    using L = TrSmem<D, RT>;
    constexpr int HALVES = L::HALVES, OPER = L::OPER, NST = L::STAGES, ALL = L::RINGS * NST, KS = D / 16;
    constexpr int STEP = RT == 1 ? 2 : 1;                  // tiles from one of a stream to its next
    extern __shared__ __align__(1024) uint8_t smem[];      // swizzled tiles start at multiples of 1024
    uint8_t *qbuf = smem, *ring = smem + RT * OPER;
    uint8_t *par = ring + ALL * OPER;                                    // [2][kTrMaxNodes]
    uint32_t *turns = reinterpret_cast<uint32_t *>(par + 2 * kTrMaxNodes);   // [2][kTrMaxNodes / 32]
    float *xch = reinterpret_cast<float *>(turns + 2 * kTrMaxNodes / 32);       // [stream][half][128]
    uint64_t *full = reinterpret_cast<uint64_t *>(xch) + L::XCH / 8;
    uint64_t *empty = full + ALL;
    uint64_t *q_full = empty + ALL, *q_empty = q_full + 1;
    uint64_t *s_full = q_empty + 1, *p_full = s_full + 4, *o_full = p_full + 4;   // [stream][half tile]
    uint64_t *mma_done = o_full + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 2);
    int *found = reinterpret_cast<int *>(tmem_slot + 1);                 // where this CTA begins: see the list of work
    volatile int *met = found + 18;                                      // a node's V was not finite: see take_out
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(smem) & 1023u) {
        if (tid == 0) raise_error(p.err, kErrState);
        pdl_wait();
        return;
    }

    if (tid == 0) {
        for (int s = 0; s < ALL; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], RT);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        mbar_init(&mma_done[0], 1);
        mbar_init(&mma_done[1], 1);
        for (int s = 0; s < 4; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 8);
            mbar_init(&o_full[s], 1);
        }
        mbar_fence_init();
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        found[2] = found[11] = 0;
        *met = 0;
    }
    // TMEM is taken when the kernels in front are done, which may be about to take their own, and the kernels behind are
    // let go when it is there, as they may take theirs before they wait (in front of the wait: times as these).  The one
    // behind PRE reads what was there before this kernel without waiting for its end.
    pdl_wait();
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        pdl_trigger();
    }

    // The list of work: prefix sums over the sequences (a thread has one of them, or with more
    // than kTrThreads several in a row), this CTA's run of tiles, and the sequence that it
    // begins in.
    Walk<RT, PRE> walk;
    const int first_own = PRE ? p.pre.P : 0;                                 // list entries of the prefixes
    {
        long long *wsum = reinterpret_cast<long long *>(par);
        PreEntry *entry = const_cast<PreEntry *>(p.pre.entry);
        const int entries = PRE ? first_own + p.own : p.B, per = entries <= kTrThreads ? 1 : (entries + kTrThreads - 1) / kTrThreads;
        const int ba = min(entries, tid * per), bz = min(entries, ba + per);
        Seq sq{};
        long long mine = 0;
        for (int b = ba; b < bz; ++b) {
            sq = seq_at<RT, PRE>(p, b);
            mine += (long long)(list_tiles<PRE>(sq) * sq.blocks) * p.H_kv;
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
#pragma unroll
        for (int w = 0; w < kTrThreads / 32; ++w) {
            const long long x = wsum[w];
            if (w < warp) before += x;
            all += x;
        }
        const long long run = max(PRE ? (long long)kTrLeast : 1ll, quotient(all + p.grid - 1, p.grid));
        const long long t0 = blockIdx.x * run;
        for (int b = ba; b < bz; ++b) {
            if (per > 1) sq = seq_at<RT, PRE>(p, b);
            const long long w = (long long)(list_tiles<PRE>(sq) * sq.blocks) * p.H_kv;
            if (PRE && blockIdx.x == 0) entry[b] = PreEntry{before, sq.tiles, sq.blocks};
            if (t0 >= before && t0 < before + w) {
                found[0] = b;
                found[1] = (int)(t0 - before);
                found[2] = (int)min(run, all - t0);
                found[3] = sq.len;
                found[4] = sq.nodes;
                found[5] = sq.total;
                found[6] = sq.tiles;
                found[7] = sq.blocks;
                if (PRE) found[8] = sq.row0;
                if (!PRE) {
                    const int item = found[1] / sq.tiles, h = item / sq.blocks;
                    p.start[blockIdx.x] = TreeStart{b, h, item - h * sq.blocks, found[1] - item * sq.tiles, sq.tiles,
                                                    sq.nodes, (int)run, 0};
                }
            }
            // Behind shared prefixes a CTA begins with the end of its run, where that is the beginning of an
            // entry, and goes on with the run's own beginning, the end of one: then all CTAs of a prefix
            // sweep over it side by side, and find in L2 what others have read.  Trees of 8 for 128
            // sequences behind 32k: 0.15 GB from HBM, some 420 us a call; in the list's order 1.25 GB, 14 us more.
            const long long last = min(t0 + run, all) - 1;
            if (PRE && last >= before && last < before + w) {
                const int item = (int)((last - before) / list_tiles<PRE>(sq));
                const long long begin = before + (long long)item * list_tiles<PRE>(sq);
                if (begin > t0) {
                    found[9] = b;
                    found[10] = item;
                    found[11] = (int)(last + 1 - begin);
                    found[12] = sq.len;
                    found[13] = sq.nodes;
                    found[14] = sq.total;
                    found[15] = sq.tiles;
                    found[16] = sq.blocks;
                    found[17] = sq.row0;
                }
            }
            before += w;
        }
        if (PRE) {
            if (blockIdx.x == 0 && tid == 0) *const_cast<PreEntry *>(p.pre.run) = PreEntry{run, 0, 0};
        } else if (t0 >= all && tid == 0) {
            p.start[blockIdx.x] = TreeStart{};
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    walk.b = found[0];
    walk.off = found[1];
    walk.left = PRE ? found[2] - found[11] : found[2];
    walk.end = PRE && found[11] > 0 ? found + 9 : nullptr;
    walk.s = Seq{found[3], found[4], found[5], found[6], found[7], PRE ? found[8] : 0};
    Run r;
    bool ok = true;

    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------------ TMA producers
        // A warp for each stream's ring, or every other slot of the one ring: a box of the
        // lanes' loop takes 60 cycles to issue, which with small pages is as long as its data
        // need.  (Waits on a parity are right only for a reader at most one phase away: of two
        // warps on one ring, a slot two turns back is read by both streams before the other
        // warp, which has seen the release of a later one, can be here.)
        const uint32_t pw = warp == 0 ? 0 : 1;
        const uint64_t keep = policy_evict_normal(), once = policy_evict_first();
        uint8_t *buf = ring + (RT == 1 ? pw : 0) * (NST * OPER);
        uint64_t *full_r = full + (RT == 1 ? pw : 0) * NST, *empty_r = empty + (RT == 1 ? pw : 0) * NST;
        uint32_t slot = 0, runs = 0;                 // ring slots passed, runs begun
        while (walk.next(p, r)) {
            const int tiles_q = RT == 2 && r.rb * 2 * p.NB + p.NB < r.s.nodes ? 2 : 1;
            if (pw == 0) ok = tr_wait(q_empty, (runs & 1) ^ 1, p.err, ok, lane);
            if (!ok) break;
            const bool pre = PRE && r.b < first_own;
            const uint64_t pol = (PRE ? r.s.blocks > 1 : p.n > RT * p.NB) ? keep : once;
            if (pw == 0 && lane == 0) {
                mbar_arrive_expect_tx(q_full, (uint32_t)(tiles_q * HALVES * p.NB * p.G * 128));
                for (int t = 0; t < tiles_q; ++t)
                    for (int hf = 0; hf < HALVES; ++hf)
                        tma_load_4d(qbuf + t * OPER + hf * kTrBox, pre ? &tmg : &tmq, hf * 64, r.h * p.G,
                                    (r.rb * RT + t) * p.NB + (pre ? r.s.row0 : 0), pre ? 0 : r.b - first_own, q_full,
                                    policy_evict_normal());
            }
            ++runs;
            const int32_t *table = pre ? p.ptable + (long long)r.b * p.pmax
                                       : p.table + (long long)(r.b - first_own) * p.max_pages;
            // K and V in turn, as the products need them.
            const int j0 = RT == 1 ? pw : 0, mine = (r.cnt - j0 + STEP - 1) / STEP;
            int id = 0, pr = 0;                          // of the lane's box: its page, and its first row there
            TileWalk tile(p, r.t0 + j0);
            for (int i = 0; i < 2 * mine; ++i, ++slot) {
                if (i && (i & 1) == 0) tile.step(p, STEP);
                if (RT == 2 && (slot & 1) != pw) continue;
                const int is_v = i & 1;
                const Tile t = tile.at(p, r.s.total);
                const uint32_t st = slot % NST, ph = (slot / NST) & 1;
                uint8_t *dst = buf + st * OPER;
                if (p.by4) {
                    // A lane's 4 rows; one behind the tile or outside the pool is past the pool's last.
                    int rows[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = lane * 4 + k, pg = (t.p0 + at) / p.page_size;
                        rows[k] = p.n_pages * p.page_size;
                        if (at < t.rows) {
                            const int q = ld_dep(table + pg);
                            if (q < 0 || q >= p.n_pages) raise_error(p.err, kErrPage);
                            else rows[k] = q * p.page_size + t.p0 + at - pg * p.page_size;
                        }
                    }
                    ok = tr_wait(&empty_r[st], ph ^ 1, p.err, ok, lane);
                    if (!ok) break;
                    const int fours = (t.rows + 3) / 4;
                    if (lane == 0) mbar_arrive_expect_tx(&full_r[st], (uint32_t)(fours * HALVES * 512));
                    __syncwarp();
                    if (lane < fours)
                        for (int hf = 0; hf < HALVES; ++hf)
                            tma_gather4(dst + hf * kTrBox + lane * 512, is_v ? &tmv : &tmk, (r.h * HALVES + hf) * 64, rows,
                                        &full_r[st], pol);
                    continue;
                }
                // Boxes of br rows, each inside a page, at most one a lane (pages of fewer than 4 rows go
                // the way above).  The lane's page number is on its way while the warp waits for the ring.
                const int boxes = (t.rows + p.br - 1) / p.br, at = lane * p.br;      // row in the tile
                if ((RT == 2 || !is_v) && lane < boxes) {
                    const int pos = t.p0 + at, pg = pos / p.page_size;
                    id = ld_dep(table + pg);
                    pr = pos - pg * p.page_size;
                }
                ok = tr_wait(&empty_r[st], ph ^ 1, p.err, ok, lane);
                if (!ok) break;
                const CUtensorMap *tm = is_v ? &tmv : &tmk;
                if (lane == 0) mbar_arrive_expect_tx(&full_r[st], (uint32_t)(boxes * p.br * HALVES * 128));
                __syncwarp();
                if (lane < boxes) {
                    if (id < 0 || id >= p.n_pages) {       // such a page is filled with zeros
                        raise_error(p.err, kErrPage);
                        id = p.n_pages;
                    }
                    if (p.by8)
                        tma_load_5d(dst + at / 8 * (HALVES * 1024), tm, 0, 0, r.h * HALVES, pr / 8, id, &full_r[st], pol);
                    else
                        for (int hf = 0; hf < HALVES; ++hf)
                            tma_load_4d(dst + hf * kTrBox + at * 128, tm, hf * 64, r.h, pr, id, &full_r[st], pol);
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
                if (RT == 1 || (i & 1) == pw) mbar_wait(&full_r[i % NST], (i / NST) & 1, p.err);
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------- MMA issuers
        // A warp, and of it one thread, per stream.  A stream's S has two halves of 64 keys,
        // each with its own barriers: while the softmax is at one, the scores of the other's
        // next tile are computed.  The queue of products is short, and what a thread does
        // between two products takes as long as several of them; so the streams have a thread
        // each, and one's products run while the other waits for its next P.
        const int s = warp - 1;
        if (elect_one()) {
            const uint32_t idesc_s = umma_idesc_bf16(128, kTrKeys / 2);
            const uint32_t idesc_o = umma_idesc_bf16(128, D) | (1u << 16);      // B (V) is MN-major
            uint8_t *buf = ring + (RT == 1 ? s : 0) * (NST * OPER);
            uint64_t *full_r = full + (RT == 1 ? s : 0) * NST, *empty_r = empty + (RT == 1 ? s : 0) * NST;
            const uint32_t rb0 = smem_u32(buf), ts = tmem + s * 128, to = tmem + kTrOut + s * D;
            const uint64_t kdesc = desc_k(rb0, p.sbo), vdesc = desc_v(rb0, p.sbo, p.hoff);
            const uint64_t qdesc = umma_desc_sw128(smem_u32(qbuf)) + (RT == 2 ? s : 0) * (OPER >> 4);
            // in descriptor units of 16 bytes: between halves of a key, 16 keys, 64 keys
            const uint32_t khalf = p.hoff >> 4, step16 = 2 * p.sbo >> 4, step64 = 8 * p.sbo >> 4;
            uint32_t slot = 0, runs = 0, done0 = 0, done1 = 0;                 // done: uses of a P

            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok) ok = mbar_poll(bar, parity, p.err);
                return ok;
            };
            auto arrived = [&](uint32_t slot) { return wait(&full_r[slot % NST], (slot / NST) & 1); };
            // S = Q K^T of 64 keys
            auto scores = [&](auto h, uint32_t st) {
                const uint64_t k = kdesc + st * (OPER >> 4) + h * step64;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    umma_bf16(ts + h * 64, qdesc + (ks >> 2) * (kTrBox >> 4) + (ks & 3) * 2,
                              k + (ks >> 2) * khalf + (ks & 3) * 2, idesc_s, ks > 0);
                umma_commit(&s_full[s * 2 + h]);
            };
            // O (+)= P V of 64 keys, as soon as P is there
            auto weigh = [&](auto h, uint32_t st, int rows, bool first) {
                if (!wait(&p_full[s * 2 + h], (h ? done1 : done0) & 1)) return false;
                tc_fence_after();
                if (h) ++done1;
                else ++done0;
                const uint64_t v = vdesc + st * (OPER >> 4) + h * step64;
                if (rows - h * 64 > 48) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        umma_bf16_ts(to, ts + h * 64 + ks * 8, v + ks * step16, idesc_o, ks > 0 || !first);
                } else {
                    for (int ks = 0; ks * 16 < rows - h * 64; ++ks)
                        umma_bf16_ts(to, ts + h * 64 + ks * 8, v + ks * step16, idesc_o, ks > 0 || !first);
                }
                umma_commit(&o_full[s * 2 + h]);
                return true;
            };
            // Rows of V behind the sequence's last position may hold anything, and 0 * NaN is
            // NaN: those that the last step of 16 keys still reads are set to zero (by either
            // stream's thread before its own products: the same zeros).
            auto clear_tail = [&](uint32_t st, int rows) {
                const int end = (rows + 15) & ~15;
                if (rows == end) return;
                uint8_t *v = buf + st * OPER;
                for (int row = rows; row < end; ++row)
                    for (int i = 0; i < HALVES * 8; ++i)
                        *reinterpret_cast<uint4 *>(v + (i >> 3) * p.hoff + (row >> 3) * p.sbo + (row & 7) * 128 +
                                                   (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            };
            const Const<0> c0{};
            const Const<1> c1{};
            while (ok && walk.next(p, r)) {
                if (!wait(q_full, runs & 1)) break;
                ++runs;
                const int cnt = r.cnt, j0 = RT == 1 ? s : 0;
                TileWalk tile(p, r.t0 + j0);
                int tj = j0;
                auto next_rows = [&]() {                       // of this stream's next tile, 0 behind the last
                    const int rows = tj < cnt ? tile.at(p, r.s.total).rows : 0;
                    tj += STEP;
                    tile.step(p, STEP);
                    return rows;
                };
                if (RT == 2 && s == 1 && r.rb * 2 * p.NB + p.NB >= r.s.nodes) {
                    // No node in this stream's row tile: its part of every release, in step with the ring.
                    for (int i = 0; i < 2 * cnt; ++i) {
                        if (!arrived(slot)) break;
                        mbar_arrive(&empty_r[slot % NST]);
                        ++slot;
                    }
                    mbar_arrive(q_empty);
                    continue;
                }
                int rows = next_rows(), next = next_rows();    // of the tile at hand and the one after it
                if (rows > 0) {
                    const uint32_t st = slot % NST;
                    if (!arrived(slot)) break;
                    scores(c0, st);
                    if (rows > 64) scores(c1, st);
                    umma_commit(&empty_r[st]);
                    ++slot;
                }
                if (j0 + STEP >= cnt) {
                    if (rows > 0) umma_commit(q_empty);
                    else mbar_arrive(q_empty);
                }
                uint32_t vst = slot % NST, kst = (slot + 1) % NST;
                bool in = false;                               // the tile's V is known to be there
                for (int j = j0; j < cnt; j += STEP) {
                    if (!in && !arrived(slot)) break;
                    clear_tail(vst, rows);
                    if (!weigh(c0, vst, rows, j == j0)) break;
                    if (rows <= 64) umma_commit(&empty_r[vst]);
                    if (next > 0) {
                        if (!arrived(slot + 1)) break;
                        scores(c0, kst);
                    }
                    // While the tensor cores have these: what the next tile needs.
                    const int after = next_rows();
                    const uint32_t slot1 = slot + (next > 0 ? 2 : 1), vst1 = slot1 % NST, kst1 = (slot1 + 1) % NST;
                    in = next > 0 && mbar_try_wait(&full_r[vst1], (slot1 / NST) & 1);
                    if (rows > 64) {
                        if (!weigh(c1, vst, rows, false)) break;
                        umma_commit(&empty_r[vst]);
                    }
                    if (next > 64) scores(c1, kst);
                    if (next > 0) {
                        umma_commit(&empty_r[kst]);
                        if (after == 0) umma_commit(q_empty);
                    }
                    rows = next;
                    next = after;
                    slot = slot1;
                    vst = vst1;
                    kst = kst1;
                }
            }
            // The products in flight end before the shared memory and TMEM that they use go.
            umma_commit(&mma_done[s]);
            mbar_wait(&mma_done[s], 0, p.err);
        }
        __syncwarp();
    } else {
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
        uint32_t *myturns = turns + s * (kTrMaxNodes / 32);
        float *mine_x = xch + (s * 2 + half) * 128 + row, *other_x = xch + (s * 2 + 1 - half) * 128 + row;
        uint32_t used[2] = {0, 0};                                      // of this stream's two S
        uint32_t idle = 0;                                              // tiles that this stream passed by
        int par_b = -1;
        bool first_run = true;
        while (walk.next(p, r)) {
            const int base = (r.rb * RT + (RT == 2 ? s : 0)) * p.NB;      // first node of the row tile
            const int node = node_r < p.NB && base + node_r < r.s.nodes ? base + node_r : -1;
            const bool active = RT == 1 || base < r.s.nodes;
            const bool live = __any_sync(0xffffffffu, node >= 0);         // the warp has rows
            if (p.parent && par_b != r.b && (!PRE || r.b >= first_own)) {
                // parent + 1 of every node in a byte (0: none; a parent that is not before its
                // node counts as none), and a bit where it is not the node just before.
                named_bar_sync(9 + s, 256);
                const int pi = wt < r.s.nodes
                                   ? checked(ld_dep(p.parent + (long long)(r.b - first_own) * p.n + wt), INT_MIN, wt - 1, p.err)
                                   : -1;
                mypar[wt] = (uint8_t)(pi >= 0 && pi < wt ? pi + 1 : 0);
                const uint32_t turn = __ballot_sync(0xffffffffu, wt == 0 || pi != wt - 1);
                if (lane == 0) myturns[wt >> 5] = turn;
                named_bar_sync(9 + s, 256);
                par_b = r.b;
            }
            // m: the maximum that O and l are held at, ms: m * sl, grown: a score above it moves m.
            float m = -INFINITY, ms = 0.f, grown = -INFINITY, l = 0.f;
            const uint32_t before[2] = {used[0], used[1]};   // uses of the two S before this run
            // One half of a tile; `edge`: not every row sees all of its keys (compiled apart, as
            // what it does to S costs the other tiles 30 instructions).
            auto half_tile = [&](const Tile &t, auto h, auto edge) {
                ok = tr_wait(&s_full[s * 2 + h], used[h] & 1, p.err, ok, lane);
                tc_fence_after();
                if (live) {
                    uint32_t v[32];
                    tmem_ld32u(ts + h * 64 + half * 32, v);
                    if (edge) {
                        const int first = h * 64 + half * 32;             // this thread's first key of the tile
                        // Before the nodes' slots only the tile's end counts.  (A row without a node may
                        // see anything: it is not used.)
                        const int prefix = r.s.len - (t.p0 + first), rows = t.rows - first;
                        uint32_t see = node < 0 || rows >= 32 ? 0xffffffffu : rows <= 0 ? 0u : (1u << rows) - 1u;
                        if (rows > prefix)
                            see = seen(prefix, rows, node, p.parent ? par + s * kTrMaxNodes : nullptr,
                                       turns + s * (kTrMaxNodes / 32));
                        if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((see >> i) & 1u)) v[i] = 0xff800000u;
                        }
                    }
                    // Four chains, so that one maximum does not wait for the last.
                    float t4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) t4[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[4 + k]));
#pragma unroll
                    for (int i = 8; i < 32; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) t4[k] = max3(t4[k], v[i + k], v[i + 4 + k]);
                    float top = fmaxf(max3(t4[0], __float_as_uint(t4[1]), __float_as_uint(t4[2])), t4[3]);
                    // The maximum is moved, and O scaled, only where it has grown by more than
                    // 2^kTrLazy: probabilities are then up to 2^24 instead of 1, which costs a
                    // floating sum nothing (its relative errors stay, and 2^24 * keys * |v| is
                    // inside fp32 for every |v| below 2^80), and a scaling takes as long as the
                    // half tile itself.  Both halves of a row have to agree; the barrier also puts
                    // the loads of S by both before the stores of P over it.
                    if (pair_any(pair_bar, top > grown)) {
                        *mine_x = top;
                        named_bar_sync(pair_bar, 64);
                        top = fmaxf(top, *other_x);
                        float f = 1.f;
                        if (top > grown) {
                            f = m == -INFINITY ? 1.f : fast_exp2((m - top) * sl);   // from -inf: O and l are zero
                            m = top;
                            ms = m * sl;
                            grown = m + kTrLazy / sl;
                            l *= f;
                        }
                        __syncwarp();                        // TMEM is read and written by whole warps
                        // This S being there, the product over the last P in its place is done;
                        // the one over the other's may be under way.
                        if (used[1 - h] != before[1 - h])
                            ok = tr_wait(&o_full[s * 2 + 1 - h], (used[1 - h] - 1) & 1, p.err, ok, lane);
                        tc_fence_after();
                        if (used[0] != before[0]) {
#pragma unroll 1
                            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                                uint32_t o[16];
                                tmem_ld16(to + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st16(to + c, o);
                            }
                        }
                    }
                    const uint64_t sl2 = pair(sl, sl), ms2 = pair(-ms, -ms);
                    uint64_t sum2[2] = {0, 0};
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 x = apart(fma2(pair(v[2 * i], v[2 * i + 1]), sl2, ms2));
                        const float a = fast_exp2(x.x), b = fast_exp2(x.y);
                        sum2[i & 1] = add2(sum2[i & 1], pair(a, b));
                        u[i] = pack_bf16(a, b);
                    }
                    tmem_st16(ts + h * 64 + half * 16, u);
                    const float2 sum = apart(add2(sum2[0], sum2[1]));
                    l += sum.x + sum.y;
                    tmem_wait_st();
                }
                if (edge && h == 0 && r.s.nodes > 1 && t.p0 + t.rows > r.s.len) {   // a node sees itself
                    const uint32_t slot = 2 * (used[0] + idle) + 1, at = (RT == 1 ? s : 0) * NST + slot % NST;
                    ok = tr_wait(&full[at], (slot / NST) & 1, p.err, ok, lane);    // the tile's V
                    if (ok) take_out<HALVES>(ring + at * OPER, max(r.s.len - t.p0, 0), t.rows, p.sbo, p.hoff, wt, met);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s * 2 + h]);
                ++used[h];
            };
            const Const<0> c0{};
            const Const<1> c1{};
            TileWalk tile(p, r.t0 + (RT == 1 ? s : 0));
            for (int j = RT == 1 ? s : 0; active && j < r.cnt; j += STEP, tile.step(p, STEP)) {
                const Tile t = tile.at(p, r.s.total);
                if (t.rows == kTrKeys && t.p0 + t.rows <= r.s.len) {
                    half_tile(t, c0, c0);
                    half_tile(t, c1, c0);
                } else {
                    half_tile(t, c0, c1);
                    if (t.rows > 64) half_tile(t, c1, c1);
                }
            }
            if (!active) idle += r.cnt;
            // The end of the run: O / l if the run is the whole list entry, else a partial.
            for (int h = 0; h < 2; ++h)
                if (used[h] != before[h]) ok = tr_wait(&o_full[s * 2 + h], (used[h] - 1) & 1, p.err, ok, lane);
            const int part = 2 * blockIdx.x + (first_run ? 0 : 1);
            first_run = false;
            // The halves' sums, and with one row tile both streams' maxima: each warp then
            // joins what it needs for its share of the channels.
            if (RT == 1) {
                named_bar_sync(pair_bar, 64);
                if (half == 1) *mine_x = l;
                named_bar_sync(pair_bar, 64);
                if (half == 0) {                             // a row's sum, and its maximum
                    *mine_x = l + *other_x;
                    *other_x = m;
                }
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
                const float m0 = xch[128 + row], m1 = r.cnt > 1 ? xch[384 + row] : -INFINITY;
                mm = fmaxf(m0, m1);
                const float mu = mm == -INFINITY ? 0.f : mm;
                w0 = fast_exp2((m0 - mu) * sl);
                w1 = fast_exp2((m1 - mu) * sl);
                ll = w0 * xch[row];
                if (r.cnt > 1) ll += w1 * xch[256 + row];
            } else {
                ll = xch[s * 256 + row] + xch[s * 256 + 128 + row];
            }
            const bool whole = !PRE && r.cnt == r.s.tiles, pre = PRE && r.b < first_own;
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
            uint16_t *dst = p.out + (((long long)r.b * p.n + node) * p.H_q + r.h * p.G + (row - node_r * p.G)) * D;
            const int rt = RT == 2 ? s : 0;
            const int rr = pre ? 128 : p.rr;
            const long long tile_at = PRE ? (part_slot<RT>(p, r.b, r.h, r.rb, r.s.blocks, r.s.row0) + blockIdx.x) *
                                                    (pre ? RT : p.own_rt) + rt
                                          : (long long)part * RT + rt;
            float4 *pd = (pre ? const_cast<float4 *>(p.pre.part) : p.part) + tile_at * (D / 4) * rr + row;
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
                if (node >= 0) {
                    if (*met && !pre) {
                        const Tile e = TileWalk(p, r.t0 + r.cnt - 1).at(p, r.s.total);
                        const Channels16 z =
                            add_back(p.vp + r.h * D + c0, (long long)p.H_kv * D, p.table + (long long)(r.b - first_own) * p.max_pages,
                                     p.page_size, p.n_pages, r.s.len, TileWalk(p, r.t0).at(p, r.s.total).p0,
                                     e.p0 + e.rows, node, p.parent ? mypar : nullptr);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] += __uint_as_float(i & 1 ? z.x[i / 2] & 0xffff0000u : z.x[i / 2] << 16);
                    }
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
                            pd[(c0 + i) / 4 * rr] = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                    }
                }
                __syncwarp();                                // TMEM is read by whole warps
            }
            if (!whole && node >= 0 && c_lo == 0)
                (pre ? const_cast<float2 *>(p.pre.stat) : p.stat)[tile_at * rr + row] = make_float2(mm, ll);
            __syncwarp();
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
// `per` blocks for every border between two CTAs' runs: where it is the first inside a list
// entry, they join that entry's partials, in the order of the list.  PL neighbouring warps
// share the partials of 32 * (8 / PL) items, channels of a row.  With few entries, each
// in many parts, and few items, PL = 8 keeps the chain of loads short (one token over 2k, 16
// parts: 4 us less); with many items it would be blocks without number (64 nodes, 8 sequences
// of 8k: 38,656 blocks, 32 us more), and PL = 1 keeps them few.  A block for every
// sequence then sets the rows of the nodes that it does not have to zero.
constexpr int kTjThreads = 256;

// A thread has W * 4 channels of a row: 8 for PL = 1, so that its stores are 16 bytes (4 channels,
// 8 and 16: 32 trees of 64 over 8k 221, 216 and 215 us, chain of 200 over 8k 217, 211 and 214).
template <int RT, int PL, int W>
__global__ void __launch_bounds__(kTjThreads) tree_attn_join_kernel(const TreeAttnParams p, int D, int per) {
    static_assert(PL == 1 || W == 1, "partials are shared out for 4 channels a thread");
    __shared__ float4 xo[PL > 1 ? kTjThreads : 1];
    __shared__ float2 xs[PL > 1 ? kTjThreads : 1];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, borders = (p.grid - 1) * per;
    if ((int)blockIdx.x >= borders) {
        const int b = blockIdx.x - borders;
        const int nodes = tr_clamp(ld_dep(p.n_nodes + b), p.n);
        const long long row = (long long)p.H_q * D / 8;
        uint4 *o = reinterpret_cast<uint4 *>(p.out) + (long long)b * p.n * row;
        for (long long i = nodes * row + tid; i < p.n * row; i += kTjThreads) o[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int c1 = 1 + blockIdx.x / per;
    const TreeStart s = p.start[c1];
    if (s.t0 == 0 || s.t0 > s.run) return;             // no entry is cut here, or not for the first time
    constexpr int ITEMS = kTjThreads / PL;
    const int it = (blockIdx.x % per) * ITEMS + tid % ITEMS, pl = tid / ITEMS;
    const int base = s.rb * RT * p.NB;                 // first node of the entry
    const int rows = min(s.nodes - base, RT * p.NB) * p.G;
    const bool real = it < rows * (D / (4 * W));
    if (PL == 1 && !real) return;
    const int cw = real ? it / rows : 0, c4 = cw * W, gr = real ? it - cw * rows : 0;
    const int rt = RT == 2 && gr >= p.NB * p.G ? 1 : 0, row = gr - rt * p.NB * p.G;
    const int first = 2 * (c1 - 1) + (s.t0 == s.run ? 0 : 1);      // the partial before the border
    const int parts = 1 + (s.tiles - s.t0 + s.run - 1) / s.run;
    const float sl = p.scale_log2;
    float4 acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -INFINITY, sum = 0.f;
    auto add = [&](float2 e, const float4 *o) {
        const float m = fmaxf(top, e.x), mu = m == -INFINITY ? 0.f : m;
        const float f = fast_exp2((top - mu) * sl), w = fast_exp2((e.x - mu) * sl);
        top = m;
        sum = sum * f + w * e.y;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            acc[i].x = acc[i].x * f + w * o[i].x;
            acc[i].y = acc[i].y * f + w * o[i].y;
            acc[i].z = acc[i].z * f + w * o[i].z;
            acc[i].w = acc[i].w * f + w * o[i].w;
        }
    };
#pragma unroll(W > 1 ? 2 : 4)
    for (int k = pl; k < parts; k += PL) {
        const long long slot = k == 0 ? first : 2 * (c1 + k - 1);
        const float4 *src = p.part + ((slot * RT + rt) * (D / 4) + c4) * p.rr + row;
        float4 o[W];
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = src[i * p.rr];
        add(p.stat[(slot * RT + rt) * p.rr + row], o);
    }
    if (PL > 1) {
        xs[tid] = make_float2(top, sum);
        xo[tid] = acc[0];
        __syncthreads();
        if (pl > 0 || !real) return;
        for (int k = 1; k < PL; ++k) add(xs[k * ITEMS + tid], &xo[k * ITEMS + tid]);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int local = gr / p.G;
    uint16_t *dst = p.out + (((long long)s.b * p.n + base + local) * p.H_q + s.h * p.G + (gr - local * p.G)) * D + c4 * 4;
    uint2 y[W];
#pragma unroll
    for (int i = 0; i < W; ++i)
        y[i] = make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
    if (W == 1) *reinterpret_cast<uint2 *>(dst) = y[0];
#pragma unroll
    for (int i = 0; i + 1 < W; i += 2)
        reinterpret_cast<uint4 *>(dst)[i / 2] = make_uint4(y[i].x, y[i].y, y[i + 1].x, y[i + 1].y);
}

// ------------------------------------------- the joining behind shared prefixes
// A block joins 32 neighbouring query rows (b, i, g) of a KV head, of each the parts of its group's
// prefix and of its own slots, in the order of the list.  PL = 1: its 8 warps share the channels, 8
// of a row a thread at a time; PL = 8: a block has 8 channels of the rows, and its warps share the
// parts (few rows, each in many parts, as one warp's chain of loads would be all that runs).
template <int RT, int PL>
__global__ void __launch_bounds__(kTjThreads) tree_attn_pre_join_kernel(const TreeAttnParams p, int D) {
    __shared__ float4 xo[PL > 1 ? 2 * kTjThreads : 1];
    __shared__ float2 xs[PL > 1 ? kTjThreads : 1];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
    const int rows = p.B * p.n * p.G, at = blockIdx.x * 32 + lane;
    const bool real = at < rows;
    const int flat = real ? at / p.G : 0, g = real ? at - flat * p.G : 0, b = flat / p.n, i = flat - b * p.n;
    const int nodes = !real ? 0 : p.n_nodes ? tr_clamp(ld_dep(p.n_nodes + b), p.n) : p.n;
    // The parts of the row: in the entry of a prefix, and in that of the sequence.
    RowParts piece[2] = {RowParts{0, 0, 1, 0}, RowParts{0, 0, 1, 0}};
    if (i < nodes) {
        piece[0] = pre_parts(p.pre, b, i, g, h);
        const PreEntry x = entry_at(p.pre.entry + p.pre.P + b);
        if (x.tiles) {
            const int rb = i / (RT * p.NB), local = i - rb * RT * p.NB, rt = local / p.NB, run = (int)entry_at(p.pre.run).start;
            const long long t0 = x.start + (long long)(h * x.blocks + rb) * (x.tiles + kTrEntry) + kTrEntry;
            const long long c0 = quotient(t0, run), c1 = quotient(t0 + x.tiles - 1, run);
            piece[1] = RowParts{(part_slot<RT>(p, p.pre.P + b, h, rb, x.blocks, 0) + c0) * p.own_rt + rt, (int)(c1 - c0) + 1,
                              p.own_rt, (local - rt * p.NB) * p.G + g};
        }
    }
    const float sl = p.scale_log2;
    uint16_t *dst = p.out + ((long long)flat * p.H_q + h * p.G + g) * D;
    for (int c = PL > 1 ? blockIdx.z : warp; c < D / 8; c += PL > 1 ? D : kTjThreads / 32) {
        float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        float top = -INFINITY, sum = 0.f;
        auto add = [&](float2 e, float4 x, float4 y) {
            const float m = fmaxf(top, e.x), mu = m == -INFINITY ? 0.f : m;
            const float f = fast_exp2((top - mu) * sl), w = fast_exp2((e.x - mu) * sl);
            top = m;
            sum = sum * f + w * e.y;
            acc[0] = make_float4(acc[0].x * f + w * x.x, acc[0].y * f + w * x.y, acc[0].z * f + w * x.z, acc[0].w * f + w * x.w);
            acc[1] = make_float4(acc[1].x * f + w * y.x, acc[1].y * f + w * y.y, acc[1].z * f + w * y.z, acc[1].w * f + w * y.w);
        };
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int rr = k ? p.rr : 128;
            const float2 *stat = k ? p.stat : p.pre.stat;
            const float4 *part = k ? p.part : p.pre.part;
#pragma unroll 4
            for (int j = PL > 1 ? warp : 0; j < piece[k].count; j += PL) {
                const long long s = piece[k].tile + (long long)j * piece[k].step;
                const float4 *src = part + (s * (D / 4) + 2 * c) * rr + piece[k].row;
                add(__ldcg(stat + s * rr + piece[k].row), __ldcg(src), __ldcg(src + rr));
            }
        }
        if (PL > 1) {
            xs[tid] = make_float2(top, sum);
            xo[2 * tid] = acc[0];
            xo[2 * tid + 1] = acc[1];
            __syncthreads();
            if (warp > 0) return;
            for (int w = 1; w < PL; ++w) add(xs[w * 32 + lane], xo[2 * (w * 32 + lane)], xo[2 * (w * 32 + lane) + 1]);
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        if (real)
            *reinterpret_cast<uint4 *>(dst + c * 8) =
                make_uint4(pack_bf16(acc[0].x * inv, acc[0].y * inv), pack_bf16(acc[0].z * inv, acc[0].w * inv),
                           pack_bf16(acc[1].x * inv, acc[1].y * inv), pack_bf16(acc[1].z * inv, acc[1].w * inv));
    }
}

// ------------------------------------------------------------------- host side
static size_t tr_align(size_t x) { return (x + 255) & ~(size_t)255; }

static int tr_row_tiles(int n, int G) { return n <= 128 / G ? 1 : 2; }

// Rows of a row tile in the workspace: those of one short tile, in pairs of 64-byte segments.
static int tr_part_rows(int n, int G) { return n <= 128 / G ? (n * G + 7) / 8 * 8 : 128; }

size_t tree_attn_workspace_bytes(const magicdec_paged_shape &s, int n) {
    const int G = s.H_q / s.H_kv;
    const size_t rows = 2 * (size_t)magicdec_host::sm_count() * tr_row_tiles(n, G) * tr_part_rows(n, G);
    return tr_align(magicdec_host::sm_count() * sizeof(TreeStart)) + tr_align(rows * sizeof(float2)) + rows * s.d * 4;
}

// The list of work is counted in 32 bits within a sequence and within a CTA's run.
static bool tr_counts(const TreeAttnParams &p) {
    const long long cap = (long long)p.page_size * p.max_pages;
    const long long tiles = p.span ? (cap + p.span - 1) / p.span : (long long)p.max_pages * p.tpp;
    const long long work = tiles * p.H_kv * ((p.n + p.NB - 1) / p.NB);
    return work <= INT_MAX && work * p.B / p.grid < INT_MAX;
}

template <int D, int RT>
static magicdec_status launch_tree_t(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                     const TreeAttnParams &p, cudaStream_t st) {
    auto kern = tree_attn_kernel<D, RT, false>;
    constexpr int smem = TrSmem<D, RT>::BYTES;
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    if (!magicdec_host::allow_smem_once<tree_attn_kernel<D, RT, false>>(smem)) return MAGICDEC_ERR_CUDA;
    magicdec_status s =
        magicdec_host::launch_pdl(kern, dim3((unsigned)p.grid), dim3(kTrThreads), smem, st, tmq, tmk, tmv, tmq, p);
    if (s != MAGICDEC_OK) return s;
    const int items = (p.n < RT * p.NB ? p.n : RT * p.NB) * p.G * (D / 4);
    const bool few = items <= 512 && 2 * (long long)p.B * p.H_kv <= p.grid;
    const int block = few ? kTjThreads / 8 : kTjThreads * 2;
    const int per = (items + block - 1) / block;
    return magicdec_host::launch_pdl(few ? tree_attn_join_kernel<RT, 8, 1> : tree_attn_join_kernel<RT, 1, 2>,
                                     dim3((unsigned)((p.grid - 1) * per + (p.n_nodes ? p.B : 0))), dim3(kTjThreads), 0,
                                     st, p, D, per);
}

// What follows from the shape of the pool and the heads.
static void set_tiles(TreeAttnParams &p, const magicdec_paged_shape &s) {
    p.err = magicdec_host::device_error_word();
    p.B = s.B;
    p.H_q = s.H_q;
    p.H_kv = s.H_kv;
    p.G = s.H_q / s.H_kv;
    p.page_size = s.page_size;
    p.n_pages = s.n_pages;
    p.max_pages = s.max_pages;
    p.NB = 128 / p.G;
    // Tiles and boxes.  A tile is of whole pages, or a part of one page, copied by boxes of a page
    // or of 64 rows (boxes of 128 rows, 16 trees of 8 over 30k at d = 128: 327 us, of 64: 299).
    // Where that leaves too much of the tiles empty, and pages are of a multiple of 8 rows, tiles
    // run on over the pages, in boxes of the largest power of 2 rows that divides a page; how
    // much is too much hangs on the bytes of such a box, as the copy engine takes 70 cycles for
    // even the smallest (24 ragged sequences of up to 36k, 13 nodes, d = 64: boxes of 8 rows 242
    // us whatever the page, of 16 rows 198, of 64 rows 172; pages of 48 rows in twos 228).
    p.by8 = s.page_size % 8 == 0;
    p.tpp = (s.page_size + kTrKeys - 1) / kTrKeys;
    p.span = s.page_size <= kTrKeys ? kTrKeys / s.page_size * s.page_size : 0;
    p.br = s.page_size < kTrKeys / 2 ? s.page_size : kTrKeys / 2;
    const int even = s.page_size & -s.page_size, bytes = even * s.d * 2;
    const long long used = p.span ? p.span : s.page_size, room = p.span ? kTrKeys : (long long)p.tpp * kTrKeys;
    if (p.by8 && used * 16 < room * (bytes >= 4096 ? 15 : bytes >= 2048 ? 14 : 12)) {
        p.span = kTrKeys;
        p.br = even < p.br ? even : p.br;
    }
    p.scale_log2 = kLog2e / sqrtf((float)s.d);
    p.grid = magicdec_host::sm_count();
    p.by4 = s.page_size < 4;
    p.sbo = p.by8 ? s.d / 64 * 1024 : 1024;
    p.hoff = p.by8 ? 1024 : kTrBox;
}

static bool set_maps(const TreeAttnParams &p, const magicdec_paged_shape &s, const uint16_t *q, const uint16_t *kp,
                     const uint16_t *vp, CUtensorMap *tmq, CUtensorMap *tmk, CUtensorMap *tmv, CUtensorMap *tmg) {
    // Queries as (d, H_q, n, B), one box = NB nodes of a KV head's group; tmg, if
    // given, takes the rows of all sequences for those of one.  The pool with
    // pages of a multiple of 8 rows as (64 channels, 8 rows, halves of all heads, groups of 8
    // rows, pages): one box is a page (or a part of it) of one KV head, its channels read
    // together and its rows laid out for the tensor cores.  Other pages as (d, H_kv,
    // page_size, n_pages), boxes of 64 channels x a page (or 64 rows); pages of 1 to 3 rows as
    // one list of rows, 4 of them a copy (32 sequences of 32k, 8 nodes, pages of 1, 2 and 3 rows:
    // 4.2, 2.2 and 1.8 ms with a box a page, 1.6 ms so; of 4 rows: 1.15 ms with boxes).
    const int D = s.d, HV = D / 64;
    const uint64_t row = (uint64_t)s.H_kv * D * 2;
    const uint32_t br = (uint32_t)p.br;
    const uint64_t kd4[4] = {(uint64_t)D, (uint64_t)s.H_kv, (uint64_t)s.page_size, (uint64_t)s.n_pages};
    const uint64_t ks4[3] = {(uint64_t)D * 2, row, s.page_size * row};
    const uint32_t kb4[4] = {64, 1, br, 1};
    const uint64_t kd2[2] = {(uint64_t)s.H_kv * D, (uint64_t)s.n_pages * s.page_size};
    const uint32_t kb2[2] = {64, 1};
    const uint64_t kd5[5] = {64, 8, (uint64_t)s.H_kv * HV, (uint64_t)s.page_size / 8, (uint64_t)s.n_pages};
    const uint64_t ks5[4] = {row, 128, 8 * row, s.page_size * row};
    const uint32_t kb5[5] = {64, 8, (uint32_t)HV, br / 8, 1};
    const uint64_t qd[4] = {(uint64_t)D, (uint64_t)s.H_q, (uint64_t)p.n, (uint64_t)s.B};
    const uint64_t qs[3] = {(uint64_t)D * 2, (uint64_t)s.H_q * D * 2, (uint64_t)p.n * s.H_q * D * 2};
    const uint32_t qbx[4] = {64, (uint32_t)p.G, (uint32_t)p.NB, 1};
    auto pool = [&](CUtensorMap *m, const uint16_t *x) {
        return p.by4   ? magicdec_host::encode_tmap_bf16(m, x, 2, kd2, &row, kb2, D * 2)
               : p.by8 ? magicdec_host::encode_tmap_bf16(m, x, 5, kd5, ks5, kb5, D * 2)
                       : magicdec_host::encode_tmap_bf16(m, x, 4, kd4, ks4, kb4, D * 2);
    };
    const uint64_t gd[4] = {(uint64_t)D, (uint64_t)s.H_q, (uint64_t)s.B * p.n, 1};
    return pool(tmk, kp) && pool(tmv, vp) && magicdec_host::encode_tmap_bf16_4d(tmq, q, qd, qs, qbx) &&
           (!tmg || magicdec_host::encode_tmap_bf16_4d(tmg, q, gd, qs, qbx));
}

magicdec_status launch_tree_attn(const magicdec_paged_shape &s, int n, const uint16_t *q, const uint16_t *kp,
                                 const uint16_t *vp, const int32_t *table, const int32_t *len, const int32_t *n_nodes,
                                 const int32_t *parent, uint16_t *out, void *ws, cudaStream_t st) {
    TreeAttnParams p{};
    p.len = len;
    p.n_nodes = n_nodes;
    p.parent = parent;
    p.table = table;
    p.vp = vp;
    p.out = out;
    p.n = n;
    set_tiles(p, s);
    if (!tr_counts(p)) return MAGICDEC_ERR_UNSUPPORTED;
    const int RT = tr_row_tiles(n, p.G);
    const size_t slots = 2 * (size_t)p.grid;
    uint8_t *w = static_cast<uint8_t *>(ws);
    p.start = reinterpret_cast<TreeStart *>(w);
    w += tr_align(p.grid * sizeof(TreeStart));
    p.stat = reinterpret_cast<float2 *>(w);
    p.rr = tr_part_rows(n, p.G);
    w += tr_align(slots * RT * p.rr * sizeof(float2));
    p.part = reinterpret_cast<float4 *>(w);

    CUtensorMap tmq, tmk, tmv;
    if (!set_maps(p, s, q, kp, vp, &tmq, &tmk, &tmv, nullptr)) return MAGICDEC_ERR_CUDA;
    if (s.d == 128)
        return RT == 1 ? launch_tree_t<128, 1>(tmq, tmk, tmv, p, st) : launch_tree_t<128, 2>(tmq, tmk, tmv, p, st);
    return RT == 1 ? launch_tree_t<64, 1>(tmq, tmk, tmv, p, st) : launch_tree_t<64, 2>(tmq, tmk, tmv, p, st);
}

// ------------------------------------------------- behind shared prefixes: host side
// One row tile a CTA while a group's rows fit one on average and a sequence's do; else two, which
// read K and V once for 256 rows.
static int pre_row_tiles(int B, int P, int n, int G) {
    const int NB = 128 / G;
    return n <= NB && (long long)((B + P - 1) / P) * n <= NB ? 1 : 2;
}

// Up to this many query rows of a sequence's KV head, its own slots are another kernel's (prefix_own.cu).
constexpr int kTrOwnRows = 32;

struct PreSizes {
    int RT, own, own_rt, own_blocks, rr;       // own: sequences in the list
    long long pslots, slots;
};
static PreSizes pre_sizes(const magicdec_paged_shape &s, int P, int n) {
    PreSizes z;
    const int G = s.H_q / s.H_kv, NB = 128 / G;
    z.RT = pre_row_tiles(s.B, P, n, G);
    z.own = n * G > kTrOwnRows ? s.B : 0;
    z.own_rt = tr_row_tiles(n, G);
    z.own_blocks = (n + z.RT * NB - 1) / (z.RT * NB);
    z.rr = tr_part_rows(n, G);
    z.pslots = ((long long)s.B * n / (z.RT * NB) + P) * s.H_kv + magicdec_host::sm_count();
    z.slots = z.own ? (long long)s.B * s.H_kv * z.own_blocks + magicdec_host::sm_count() : 0;
    return z;
}

size_t prefix_attn_workspace_bytes(const magicdec_paged_shape &s, int P, int n) {
    const PreSizes z = pre_sizes(s, P, n);
    const size_t prows = (size_t)z.pslots * z.RT * 128, rows = (size_t)z.slots * z.own_rt * z.rr;
    return tr_align(((size_t)P + s.B + 1) * sizeof(PreEntry)) + tr_align(prows * sizeof(float2)) +
           tr_align(rows * sizeof(float2)) + (prows + rows) * s.d * 4;
}

template <int D, int RT>
static magicdec_status launch_prefix_t(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                       const CUtensorMap &tmg, const TreeAttnParams &p, const uint16_t *q,
                                       const uint16_t *k, int parts, cudaStream_t st) {
    auto kern = tree_attn_kernel<D, RT, true>;
    constexpr int smem = TrSmem<D, RT>::BYTES;
    if (!magicdec_host::allow_smem_once<tree_attn_kernel<D, RT, true>>(smem)) return MAGICDEC_ERR_CUDA;
    magicdec_status s =
        magicdec_host::launch_pdl(kern, dim3((unsigned)p.grid), dim3(kTrThreads), smem, st, tmq, tmk, tmv, tmg, p);
    if (s != MAGICDEC_OK) return s;
    if (!p.own) {
        PreOwn x{};
        x.pre = p.pre;
        x.q = q;
        x.k = k;
        x.v = p.vp;
        x.out = p.out;
        x.len = p.len;
        x.n_nodes = p.n_nodes;
        x.parent = p.parent;
        x.table = p.table;
        x.err = p.err;
        x.H_q = p.H_q;
        x.page_size = p.page_size;
        x.n_pages = p.n_pages;
        x.max_pages = p.max_pages;
        x.parts = parts;
        x.scale_log2 = p.scale_log2;
        return launch_prefix_own(x, D, st);
    }
    const unsigned blocks = (unsigned)(((long long)p.B * p.n * p.G + 31) / 32);
    // Parts shared out while the blocks of whole rows are few, each of the 16 or 8 blocks of a row finding its
    // parts anew (trees of 16 behind 4k, 8 KV heads, shared out and not: 1 sequence 18.2 and 31.0 us, 4 31.2 and
    // 33.6; behind 1268, 4 28.6 and 25.9, 8 36.8 and 27.2).
    const long long whole = (long long)blocks * p.H_kv;
    if (4 * whole <= p.grid || (2 * whole <= p.grid && parts >= 8))
        return magicdec_host::launch_pdl(tree_attn_pre_join_kernel<RT, 8>, dim3(blocks, (unsigned)p.H_kv, D / 8),
                                         dim3(kTjThreads), 0, st, p, D);
    return magicdec_host::launch_pdl(tree_attn_pre_join_kernel<RT, 1>, dim3(blocks, (unsigned)p.H_kv), dim3(kTjThreads), 0,
                                     st, p, D);
}

magicdec_status launch_prefix_attn(const magicdec_paged_shape &s, int P, int pmax, int n, const uint16_t *q,
                                   const uint16_t *kp, const uint16_t *vp, const int32_t *ptable, const int32_t *plen,
                                   const int32_t *first, const int32_t *table, const int32_t *len,
                                   const int32_t *n_nodes, const int32_t *parent, uint16_t *out, void *ws,
                                   cudaStream_t st) {
    TreeAttnParams p{};
    p.len = len;
    p.n_nodes = n_nodes;
    p.parent = parent;
    p.table = table;
    p.vp = vp;
    p.out = out;
    p.n = n;
    set_tiles(p, s);
    p.plen = plen;
    p.ptable = ptable;
    p.pmax = pmax;
    // The list is counted in 32 bits within an entry and within a CTA's run.
    auto tiles = [&](long long pages) {
        return p.span ? (pages * p.page_size + p.span - 1) / p.span : pages * p.tpp;
    };
    const PreSizes z = pre_sizes(s, P, n);
    const long long rows = (long long)s.B * n;
    const double work = (double)(tiles(pmax) + kTrEntry) * s.H_kv * (double)((rows + p.NB - 1) / p.NB);
    const double own = (double)(tiles(s.max_pages) + kTrEntry) * s.H_kv * ((n + p.NB - 1) / p.NB);
    if (work > INT_MAX || own > INT_MAX || (work * P + own * s.B) / p.grid >= INT_MAX / 2) return MAGICDEC_ERR_UNSUPPORTED;
    uint8_t *w = static_cast<uint8_t *>(ws);
    const size_t prows = (size_t)z.pslots * z.RT * 128, orows = (size_t)z.slots * z.own_rt * z.rr;
    p.own = z.own;
    p.pre.entry = reinterpret_cast<PreEntry *>(w);
    p.pre.run = p.pre.entry + P + s.B;
    w += tr_align(((size_t)P + s.B + 1) * sizeof(PreEntry));
    p.pre.stat = reinterpret_cast<float2 *>(w);
    w += tr_align(prows * sizeof(float2));
    p.stat = reinterpret_cast<float2 *>(w);
    w += tr_align(orows * sizeof(float2));
    p.pre.part = reinterpret_cast<float4 *>(w);
    p.pre.first = first;
    p.pre.P = P;
    p.pre.B = s.B;
    p.pre.n = n;
    p.pre.G = p.G;
    p.pre.H_kv = s.H_kv;
    p.pre.NB = p.NB;
    p.pre.RT = z.RT;
    p.part = reinterpret_cast<float4 *>(w + prows * s.d * 4);
    p.rr = z.rr;
    p.own_rt = z.own_rt;
    p.own_blocks = z.own_blocks;
    // A row's parts of its prefix, about: where prefixes and own slots are as long as they can be.
    const long long blocks = (rows + z.RT * p.NB - 1) / (z.RT * p.NB), list = ((tiles(pmax) + kTrEntry) * (blocks > P ? blocks : P) +
                             (tiles(s.max_pages) + kTrEntry) * z.own_blocks * z.own) * s.H_kv, run = (list + p.grid - 1) / p.grid;
    const long long parts = tiles(pmax) / (run > kTrLeast ? run : kTrLeast) + 1;
    CUtensorMap tmq, tmk, tmv, tmg;
    if (!set_maps(p, s, q, kp, vp, &tmq, &tmk, &tmv, &tmg)) return MAGICDEC_ERR_CUDA;
    if (s.d == 128)
        return z.RT == 1 ? launch_prefix_t<128, 1>(tmq, tmk, tmv, tmg, p, q, kp, (int)parts, st)
                         : launch_prefix_t<128, 2>(tmq, tmk, tmv, tmg, p, q, kp, (int)parts, st);
    return z.RT == 1 ? launch_prefix_t<64, 1>(tmq, tmk, tmv, tmg, p, q, kp, (int)parts, st)
                     : launch_prefix_t<64, 2>(tmq, tmk, tmv, tmg, p, q, kp, (int)parts, st);
}

}  // namespace magicdec
