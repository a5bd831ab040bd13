// Attention with a sliding window and sinks: what its kernels share.
//
// Token i of a sequence sees token j <= i where i - j < window (the near pairs)
// or j < sinks (of those, the far pairs are the ones with i - j >= window). Every
// kernel treats near and far pairs apart: the near ones in tiles along the
// diagonal, the far ones as one narrow tile of the sinks.
#pragma once

#include "kda_internal.cuh"
#include "kda_linear.cuh"

namespace kda {

constexpr int kWinTile = 256;     // tokens of an entry of the tile table
constexpr int kWinMaxSinks = 128;
constexpr int kWinFarQueries = 1024;  // queries to a part of the sinks' far gradients, on the tensor cores

struct WinTile {
    int seq;    // sequence
    int start;  // its first token in the batch
    int len;    // its tokens
    int first;  // the tile's first token, counted from `start` (len 0: no such tile)
};
// Equal lengths need no table; of a packed batch launch_win_tiles writes one.
struct WinGeom {
    const int4 *tiles;         // packed: {seq, start, len, first}, else null
    const int32_t *seq_tile;   // packed: first tile of each sequence [N + 1]
    const int32_t *seq_row;    // gradients of a packed batch with sinks: see win_near_row [N + 1], else null
    int N, T, hq, hk, group;   // group: query heads to a key head
    int per_seq, ntiles;       // equal lengths: tiles per sequence; tiles (packed: an upper bound)
    int64_t tokens;
    int window, sinks;
    int rows_each, rows;       // equal lengths: rows of a sequence; of all sequences at most
    FastDiv by_seq, by_hq, by_hk;
};
__device__ __forceinline__ WinTile win_tile(const WinGeom &g, int t) {
    if (g.tiles) {
        const int4 x = g.tiles[t];
        return {x.x, x.y, x.z, x.w};
    }
    const int n = g.by_seq.div(t);
    return {n, n * g.T, g.T, (t - n * g.per_seq) * kWinTile};
}

// Where dk and dv of the sinks that far queries see are gathered: rows [hk][2][d], one
// for each sink of each sequence that is longer than the window, sequence after sequence.
// There are no more of them than tokens, whatever the number of sequences and sinks.
__host__ __device__ __forceinline__ int win_rows_of(int len, int window, int sinks) {
    return len > window ? (sinks < len ? sinks : len) : 0;
}
__device__ __forceinline__ int win_near_row(const WinGeom &g, int seq) {  // of sink 0
    return g.seq_row ? g.seq_row[seq] : seq * g.rows_each;
}
// The far queries' parts, `queries` of them to a part, cut where the sequence starts: a
// sequence's first part has such rows too, one that starts `first` > 0 tokens into its
// sequence those behind them that its place in the batch gives. (Two parts that are not
// their sequences' first start `queries` tokens apart or more.)
__device__ __forceinline__ int64_t win_far_row(const WinGeom &g, int seq, int start, int first, int queries) {
    return first / queries == g.window / queries
               ? win_near_row(g, seq)
               : g.rows + (int64_t)((start + first) / queries - 1) * g.sinks;
}
// Rows at most: of the sequences, and of parts that are not their sequences' first.
inline int64_t win_rows(int N, int64_t tokens, int sinks) {
    return (int64_t)N * sinks < tokens ? (int64_t)N * sinks : tokens;
}
inline int64_t win_part_rows(int64_t tokens, int sinks, int queries) { return tokens / queries * sinks; }

struct WinArgs {
    kda_dtype_t dt;
    const void *q, *k, *v;              // token strides in elements
    int64_t q_stride, k_stride, v_stride;
    float scale;
    int window, sinks;
    void *o;
    float *lse;                         // [tokens][hq]; forward: nullable
    const int32_t *cu_seqlens;          // nullable
    int N, T, hq, hk, d;
    int32_t *status;                    // packed: the caller's, nullable
    void *workspace;
    // backward only
    const void *out, *d_o;              // contiguous
    void *dq, *dk, *dv;                 // contiguous
};
size_t window_workspace_bytes(int N, int64_t T, int hq, int hk, int d, int sinks, kda_dtype_t dt, bool packed, bool back);
cudaError_t launch_window(const WinArgs &a, cudaStream_t s);
cudaError_t launch_window_backward(const WinArgs &a, cudaStream_t s);

// The cache of a slot: [entries][hk][d], entries = sinks + window. The token at
// position p lies at entry p (p < sinks) or sinks + (p - sinks) mod window.
struct WinCacheArgs {
    kda_dtype_t dt;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    float scale;
    int sinks, entries, pool;
    void *k_cache, *v_cache;
    const int32_t *slots, *positions;
    const int32_t *cu_seqlens;
    void *o;
    int32_t *status;
    int N, T, hq, hk, d;
};
cudaError_t launch_window_cache_write(const WinCacheArgs &a, cudaStream_t s);
cudaError_t launch_window_decode(const WinCacheArgs &a, cudaStream_t s);

}  // namespace kda
