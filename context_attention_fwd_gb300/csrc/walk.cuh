// walk.cuh -- the order in which a CTA visits the tiles of the other operand.
//
// Forward (a CTA holds query rows of ring chunk r): at ring iteration it the
// queries meet KV chunk (r - it) mod P (diffusers issue #14265, "Root cause":
// the query stays put while the K/V chunks rotate); with the all-gather order
// they meet chunk it.  Backward (a CTA holds one KV tile of chunk c): the
// query chunks (c + it) mod P, i.e. the chunks that met c at iteration it.
// With causal masking, tiles entirely above the diagonal are skipped.
#pragma once

#include "internal.h"

namespace ctxattn {

// ------------------------------------------------------------ launch order
// (tile, head, z) of this CTA: the grid is (tiles, heads, z) in the tile-major
// order and (heads, z, tiles) in the head-major one, which launches tile 0 of
// every head before tile 1 of any (the host picks the order per launch).
struct GridPos {
    int tile, head, z;
};
template <bool kHeadMajor>
__device__ __forceinline__ GridPos grid_pos() {
    if (kHeadMajor) return {(int)blockIdx.z, (int)blockIdx.x, (int)blockIdx.y};
    return {(int)blockIdx.x, (int)blockIdx.y, (int)blockIdx.z};
}
inline dim3 grid_dims(bool head_major, int tiles, int heads, int z) {
    return head_major ? dim3(heads, z, tiles) : dim3(tiles, heads, z);
}

// ------------------------------------------------------------ forward walk
struct KvWalk {
    int it, c, t, t0, t1;
};
struct WalkCfg {
    int r, P, causal, allgather, q_last;  // q_last: the CTA's last query row (global)
};
__device__ __forceinline__ void kv_set_chunk(const ChunkTable& ct, const WalkCfg& g, KvWalk& w) {
    w.c = g.allgather ? w.it : (g.r - w.it + g.P) % g.P;
    w.t0 = w.t = ct.tile_off[w.c];
    w.t1 = ct.tile_off[w.c + 1];
}
__device__ __forceinline__ bool kv_visible(const ChunkTable& ct, const WalkCfg& g, const KvWalk& w) {
    if (!g.causal || w.c < g.r) return true;
    if (w.c > g.r) return false;
    return ct.off[w.c] + (w.t - w.t0) * kTile <= g.q_last;
}
__device__ __forceinline__ void kv_adv(const ChunkTable& ct, const WalkCfg& g, KvWalk& w) {
    if (g.causal && w.c > g.r) w.t = w.t1 - 1;  // the whole chunk is masked
    if (++w.t == w.t1 && ++w.it < g.P) kv_set_chunk(ct, g, w);
}
__device__ __forceinline__ void kv_first(const ChunkTable& ct, const WalkCfg& g, KvWalk& w) {
    w.it = 0;
    kv_set_chunk(ct, g, w);
    while (w.it < g.P && !kv_visible(ct, g, w)) kv_adv(ct, g, w);
}
__device__ __forceinline__ void kv_next(const ChunkTable& ct, const WalkCfg& g, KvWalk& w) {
    do kv_adv(ct, g, w);
    while (w.it < g.P && !kv_visible(ct, g, w));
}
// The visited tile is the last one the walk visits in its chunk (the end of
// that chunk's partial): the chunk's last tile, or with causal masking in the
// query chunk itself the last tile starting at or before the CTA's last row.
__device__ __forceinline__ bool kv_chunk_last(const ChunkTable& ct, const WalkCfg& g, const KvWalk& w) {
    int last = w.t1 - 1;
    if (g.causal && w.c == g.r) last = min(last, w.t0 + ((g.q_last - ct.off[w.c]) >> 7));
    return w.t == last;
}
// Number of KV tiles the walk visits.
__device__ __forceinline__ int kv_count(const ChunkTable& ct, const WalkCfg& g) {
    if (!g.causal) return ct.ntiles;
    return ct.tile_off[g.r] + ((g.q_last - ct.off[g.r]) >> 7) + 1;
}

// ----------------------------------------------------------- backward walk
// Query tiles visited by one KV tile (chunk c, first row kv_start): for each
// query head of the GQA group, ring iterations it = 0..P-1 (query chunk
// (c + it) mod P) and that chunk's 128-row tiles.
struct QTileIter {
    int h, t, it, r;
};
struct QWalk {
    const ChunkTable* ct;
    int c, causal, kv_start, h_end;
    __device__ __forceinline__ int first_row(const QTileIter& q) const {
        return ct->off[q.r] + (q.t - ct->tile_off[q.r]) * kTile;
    }
    __device__ __forceinline__ bool visible(const QTileIter& q) const {
        if (!causal || q.r > c) return true;
        if (q.r < c) return false;
        const int qs = first_row(q);
        return qs + min(kTile, ct->off[q.r + 1] - qs) - 1 >= kv_start;
    }
    __device__ __forceinline__ void adv(QTileIter& q) const {
        if (causal && q.r < c) q.t = ct->tile_off[q.r + 1] - 1;  // the whole chunk is masked
        ++q.t;
        if (q.t == ct->tile_off[q.r + 1]) {
            if (++q.it == ct->P) {
                q.it = 0;
                ++q.h;
            }
            q.r = (c + q.it) % ct->P;
            q.t = ct->tile_off[q.r];
        }
    }
    __device__ __forceinline__ void next(QTileIter& q) const {
        do adv(q);
        while (q.h < h_end && !visible(q));
    }
    __device__ __forceinline__ QTileIter first(int h0) const {
        QTileIter q;
        q.h = h0;
        q.it = 0;
        q.r = c;
        q.t = ct->tile_off[c];
        while (!visible(q)) adv(q);
        return q;
    }
    // number of query tiles visited, over G query heads
    __device__ __forceinline__ int count(int G) const {
        if (!causal) return G * ct->ntiles;
        int per = ct->tile_off[c + 1] - ct->tile_off[c] - ((kv_start - ct->off[c]) >> 7);
        for (int r2 = c + 1; r2 < ct->P; ++r2) per += ct->tile_off[r2 + 1] - ct->tile_off[r2];
        return G * per;
    }
};

// ------------------------------------------------------------- window walks
// Under a window the tiles a CTA meets are at most two runs of the tile
// numbering: those that hold sinks, then those the window reaches.  They are
// visited in ascending order whatever the chunking (the merge gives the same
// result in any order), and nothing outside them is touched.
__host__ __device__ __forceinline__ int tile_of_row(const ChunkTable& ct, int row) {
    int c = 0;
    while (c + 1 < ct.P && ct.off[c + 1] <= row) ++c;
    return ct.tile_off[c] + (row - ct.off[c]) / kTile;
}
__host__ __device__ __forceinline__ int tile_first_row(const ChunkTable& ct, int t) {
    const int c = chunk_of_tile(ct, t);
    return ct.off[c] + (t - ct.tile_off[c]) * kTile;
}

// KV tiles [0, a) and [b0, b1) of query rows [q_first, q_last].
struct WinKv {
    int a, b0, b1;
    __host__ __device__ __forceinline__ int count() const { return a + b1 - b0; }
};
__host__ __device__ __forceinline__ WinKv win_kv(const ChunkTable& ct, const Window& w, int S, int q_first, int q_last) {
    const int lo = q_first > w.left ? q_first - w.left : 0;
    const int hi = q_last < S - 1 - w.right ? q_last + w.right : S - 1;
    const int sinks = w.causal && w.sinks > q_last + 1 ? q_last + 1 : w.sinks;
    WinKv r;
    r.b0 = tile_of_row(ct, lo);
    r.b1 = tile_of_row(ct, hi) + 1;
    const int full = sinks > 0 ? tile_of_row(ct, sinks - 1) + 1 : 0;
    r.a = full < r.b0 ? full : r.b0;
    if (full > r.b1) r.b1 = full;
    return r;
}
__device__ __forceinline__ void win_first(const ChunkTable& ct, const WinKv& g, KvWalk& w) {
    w.t = g.a > 0 ? 0 : g.b0;
    w.it = 0;
    w.c = chunk_of_tile(ct, w.t);
    w.t0 = ct.tile_off[w.c];
    w.t1 = ct.tile_off[w.c + 1];
}
__device__ __forceinline__ void win_next(const ChunkTable& ct, const WinKv& g, KvWalk& w) {
    if (++w.t == g.a) w.t = g.b0;
    if (w.t >= g.b1) return;
    while (w.t >= w.t1) {
        ++w.c;
        w.t0 = w.t1;
        w.t1 = ct.tile_off[w.c + 1];
    }
}

// The same walk as a step j and its chunk (fewer registers than KvWalk).
__device__ __forceinline__ int win_tile(const WinKv& g, int j) { return j < g.a ? j : g.b0 + j - g.a; }
__device__ __forceinline__ int win_chunk(const ChunkTable& ct, int t, int c) {  // chunk of t, not before c
    while (ct.tile_off[c + 1] <= t) ++c;
    return c;
}

// Bits [0, n) of the 32-bit word that holds bits [base, base + 32).
__device__ __forceinline__ uint32_t bits_below(int n, int base) {
    const int k = n - base;
    return k >= 32 ? 0xffffffffu : (k <= 0 ? 0u : (1u << k) - 1u);
}

// Masks a forward tile's 128 scores of query row q_start + row (raw fp32
// bits).  Tiles that every row of the query tile sees whole skip it; the
// test is the same for all of them, so a warp never diverges on it.  The
// visible keys of a row are two runs, as bits of four words.
__device__ __forceinline__ void mask_window(const Window& w, int q_start, int row, int kv_start, int kv_len,
                                            uint32_t* s) {
    if (kv_len == kTile && kv_start >= q_start + kTile - 1 - w.left && kv_start + kTile - 1 <= q_start + w.right) return;
    const int i = q_start + row;
    const int lo = i - w.left - kv_start, hi = min(kv_len, i + w.right + 1 - kv_start);
    const int sink = min(kv_len, (w.causal ? min(w.sinks, i + 1) : w.sinks) - kv_start);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t m = (bits_below(hi, 32 * e) & ~bits_below(lo, 32 * e)) | bits_below(sink, 32 * e);
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (!(m >> k & 1u)) s[32 * e + k] = 0xff800000u;  // -inf
    }
}
// The same for the backward's transposed tile: the probabilities of key row
// kv_start + row against 64 queries from q0 on, set to zero where masked.
__device__ __forceinline__ void zero_window(const Window& w, int q_start, int q0, int row, int kv_start, int kv_len,
                                            uint32_t* pr) {
    if (kv_len == kTile && q_start >= kv_start + kTile - 1 - w.right && q_start + kTile - 1 <= kv_start + w.left) return;
    const int j = kv_start + row;
    int lo = j - w.right - q0, hi = j + w.left + 1 - q0;
    if (j < w.sinks) {
        lo = w.causal ? j - q0 : 0;
        hi = 64;
    }
    if (row >= kv_len) hi = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t m = bits_below(hi, 32 * e) & ~bits_below(lo, 32 * e);
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (!(m >> k & 1u)) pr[32 * e + k] = 0u;
    }
}

// Query tiles of one KV tile (rows [kv_start, kv_end)): those the window
// reaches, or all of them (causal: from its own on) if it holds sinks.
struct WinQ {
    int t0, t1;
};
__host__ __device__ __forceinline__ WinQ win_near_q(const ChunkTable& ct, const Window& w, int S, int kv_start, int kv_end) {
    const int lo = kv_start > w.right ? kv_start - w.right : 0;
    const int hi = kv_end - 1 < S - 1 - w.left ? kv_end - 1 + w.left : S - 1;
    return WinQ{tile_of_row(ct, lo), tile_of_row(ct, hi) + 1};
}
__host__ __device__ __forceinline__ WinQ win_sink_q(const ChunkTable& ct, const Window& w, int kv_tile) {
    return WinQ{w.causal ? kv_tile : 0, ct.ntiles};
}
// A windowed backward launches sink_parts CTAs for each of the first
// sink_tiles KV tiles (those see far more queries than the others: their
// walks are cut into pieces of about the others' length), then one CTA for
// each of the rest.
struct WinWork {
    int kv_tile, part;  // part -1: the whole walk
};
__host__ __device__ __forceinline__ int win_grid(int ntiles, int sink_tiles, int sink_parts) {
    return sink_tiles * sink_parts + ntiles - sink_tiles;
}
__host__ __device__ __forceinline__ WinWork win_work(int i, int sink_tiles, int sink_parts) {
    const int n = sink_tiles * sink_parts;
    return i < n ? WinWork{i / sink_parts, i % sink_parts} : WinWork{sink_tiles + i - n, -1};
}
__host__ __device__ __forceinline__ WinQ win_part_q(const ChunkTable& ct, const Window& w, int kv_tile, int part, int per) {
    const WinQ all = win_sink_q(ct, w, kv_tile);
    const int t0 = all.t0 + part * per;
    return WinQ{t0 < all.t1 ? t0 : all.t1, t0 + per < all.t1 ? t0 + per : all.t1};
}
// A part outside the window's reach only touches sink rows.
__host__ __device__ __forceinline__ bool win_overlap(const WinQ& a, const WinQ& b) { return a.t0 < b.t1 && b.t0 < a.t1; }

// Where a windowed CTA's piece of a KV tile leaves its partial rows, or null
// when it is the tile's only piece (BwdParams in internal.h).
template <int D>
__device__ __forceinline__ float* win_part_rows(const BwdParams& p, const WinWork& w, int split, int b, int hk,
                                                int kv_start) {
    const bool sink = w.part >= 0;
    float* base = sink ? p.sink_part : p.dkv_part;
    if (!base) return nullptr;
    const size_t piece = sink ? w.part * p.hsplit + split : split;
    return base + (((piece * p.B + b) * p.Hkv + hk) * (sink ? p.sink_rows : p.S) + kv_start) * 2 * D;
}

struct WinQWalk {
    const ChunkTable* ct;
    WinQ q;
    int r0, h_end;  // r0: chunk of tile q.t0
    __device__ __forceinline__ int first_row(const QTileIter& i) const {
        return ct->off[i.r] + (i.t - ct->tile_off[i.r]) * kTile;
    }
    __device__ __forceinline__ QTileIter first(int h0) const { return QTileIter{h0, q.t0, 0, r0}; }
    __device__ __forceinline__ void next(QTileIter& i) const {
        if (++i.t == q.t1) {
            i.t = q.t0;
            i.r = r0;
            ++i.h;
        }
        while (i.t >= ct->tile_off[i.r + 1]) ++i.r;
    }
    __device__ __forceinline__ int count(int G) const { return G * (q.t1 - q.t0); }
};

}  // namespace ctxattn
