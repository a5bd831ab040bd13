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
    int N, T, hq, hk, group;   // group: query heads to a key head
    int per_seq, ntiles;       // equal lengths: tiles per sequence; tiles (packed: an upper bound)
    int64_t tokens;
    int window, sinks;
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

// The part that far queries from tile t on write to, `per` tiles to a part: every
// sequence's are numbers in a row, and no two sequences share one.
__device__ __forceinline__ int win_far_slot(int t, int seq, int per) { return t / per + seq; }

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
