// prefix.cuh -- where the parts of attention over shared prefixes lie in the workspace: written by
// tree_attn_kernel (tree_attn.cu), put together there or in prefix_own.cu (sm_103a).
#pragma once

#include "common.cuh"

namespace magicdec {

// List tiles that an entry counts for, in front of its own, for the way in and out of it: CTAs' runs
// are equal in list tiles.  Without, 1024 entries of one tile behind 32,000 tiles of prefixes all fell
// to a few CTAs, and the call took 890 us instead of some 500.
constexpr int kTrEntry = 2;

// Tiles of a CTA's run at least: a tile more is soon done, a part more has to be written and joined.
constexpr int kTrLeast = 2;

// Where an entry of the list of work begins, its tiles and blocks; one more behind the last
// holds the length of a CTA's run of tiles.
struct __align__(16) PreEntry {
    long long start;
    int tiles, blocks;
};

// The sequences [lo, hi) behind prefix g.
struct Group {
    int lo, hi;
};

// What a kernel needs to find a row's parts of its prefix.
struct PreParts {
    const PreEntry *entry;       // of the prefixes first
    const PreEntry *run;         // the length of a run
    const float2 *stat;          // [slots][RT * 128] (max, sum)
    const float4 *part;          // [slots][RT][d / 4][128]
    const int32_t *first;        // [P + 1], or NULL: one prefix for all
    int P, B, n, G, H_kv;
    int NB, RT;                  // nodes of a row tile, row tiles of a block
};

__device__ __forceinline__ int pre_clamp(int v, int hi) { return v < 0 ? 0 : (v > hi ? hi : v); }

__device__ __forceinline__ Group group_at(const int32_t *first, int B, int g, int *err) {
    if (!first) return Group{0, B};
    return Group{pre_clamp(checked(ld_dep(first + g), 0, B, err), B),
                 pre_clamp(checked(ld_dep(first + g + 1), 0, B, err), B)};
}

// An entry's parts lie at this number and the CTA's added, one for each CTA that has some of it, and no
// two entries' meet: along the list either grows.  Prefixes are numbered by their first rows, of
// which RT * NB make a block.
__device__ __forceinline__ long long pre_slot(int row0, int e, int h, int rb, int blocks, int H_kv, int block_rows) {
    return (long long)(row0 / block_rows + e) * H_kv + h * blocks + rb;
}

// What another kernel has just written is read from L2: no line of L1 can then be older.
__device__ __forceinline__ PreEntry entry_at(const PreEntry *e) {
    const int4 x = __ldcg(reinterpret_cast<const int4 *>(e));
    return PreEntry{(long long)(uint32_t)x.x | (long long)x.y << 32, x.z, x.w};
}

// x / d, in 32 bits where they suffice (a 64-bit division is a hundred instructions).
__device__ __forceinline__ long long quotient(long long x, int d) {
    return x <= 0xffffffffll ? (long long)((uint32_t)x / (uint32_t)d) : x / d;
}

// The parts of one query row: `count` row tiles, `step` apart from `tile` on, in each its row.
struct RowParts {
    long long tile;
    int count, step, row;
};
// Of node i, head g of the group, of sequence b: what KV head h's prefix gave it.
__device__ __forceinline__ RowParts pre_parts(const PreParts &p, int b, int i, int g, int h) {
    RowParts r{0, 0, p.RT, 0};
    // The last group that begins at b or before; an empty one begins where the next does.
    int lo = 0, hi = p.first ? p.P : 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pre_clamp(ld_dep(p.first + mid), p.B) <= b) lo = mid;
        else hi = mid;
    }
    const Group q = group_at(p.first, p.B, lo, nullptr);
    const PreEntry x = entry_at(p.entry + lo), runs = entry_at(p.run);
    if (b < q.lo || b >= q.hi || x.tiles == 0) return r;
    const int node = (b - q.lo) * p.n + i, rb = node / (p.RT * p.NB), local = node - rb * p.RT * p.NB, rt = local / p.NB;
    const int run = (int)runs.start;
    const long long t0 = x.start + (long long)(h * x.blocks + rb) * (x.tiles + kTrEntry) + kTrEntry;
    const long long c0 = quotient(t0, run), c1 = quotient(t0 + x.tiles - 1, run);
    r.count = (int)(c1 - c0) + 1;
    r.tile = (pre_slot(q.lo * p.n, lo, h, rb, x.blocks, p.H_kv, p.RT * p.NB) + c0) * p.RT + rt;
    r.row = (local - rt * p.NB) * p.G + g;
    return r;
}

// What the kernel of prefix_own.cu takes beside.
struct PreOwn {
    PreParts pre;
    const uint16_t *q, *k, *v;   // [B, n, H_q, d]; the pool
    uint16_t *out;
    const int32_t *len, *n_nodes, *parent, *table;
    int *err;
    int H_q, page_size, n_pages, max_pages;
    int parts;                   // of a row's prefix, about
    float scale_log2;            // log2(e) / sqrt(d)
};
magicdec_status launch_prefix_own(const PreOwn &p, int D, cudaStream_t st);

}  // namespace magicdec
