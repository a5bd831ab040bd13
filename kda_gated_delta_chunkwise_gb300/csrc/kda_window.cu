// Attention with a sliding window and sinks, and its gradients, in fp32; what both
// types share: the tile table of packed batches, the sinks' sums.
//
//   s_ij = scale q_i . k_j over the j that i sees,  lse_i = log sum_j e^{s_ij}
//   p_ij = e^{s_ij - lse_i},  o_i = sum_j p_ij v_j
//   D_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - D_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// with dk and dv summed over the query heads of a key head, in their order. (bf16:
// kda_window_tc.cu.)
//
// One CTA takes 64 rows (queries, or keys for dk and dv) and walks tiles of 32
// columns in shared memory with the running maximum and sum of the softmax in
// registers. The products run on mma.sync tf32, every operand split in two tf32
// parts, three products for each. Bound by instructions (half of the issue slots) and their
// latencies: 1474 tokens x 15 heads over 3 key heads, window 1227: 294 us, gradients 949.
#include <math_constants.h>

#include "kda_tc_ptx.cuh"
#include "kda_window.cuh"
#include "kda_window_tc.cuh"

namespace kda {
namespace {

// ================================================================ packed batches: the table of tiles
constexpr int kPrepThreads = 1024;
__global__ void __launch_bounds__(kPrepThreads)
win_tiles_kernel(const int32_t *cu, int N, int T_total, int ntiles, int4 *tiles, int32_t *seq_tile, int32_t *seq_row,
                 int window, int sinks, int32_t *user_status) {
    __shared__ int bad;
    __shared__ int wsum[kPrepThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = (cu[0] != 0 || cu[N] != T_total) ? 1 : 0;
    __syncthreads();
    for (int i = tid; i < N; i += kPrepThreads)
        if (cu[i + 1] < cu[i] || cu[i] < 0 || cu[i + 1] > T_total) atomicOr(&bad, 1);
    __syncthreads();
    const bool b = bad != 0;
    if (tid == 0 && user_status) *user_status = b ? KDA_DEV_BAD_CU_SEQLENS : KDA_DEV_OK;
    // the sums of what each sequence has, up to every one; returns that of all
    auto sums = [&](int32_t *out, auto of) {
        if (tid == 0) out[0] = 0;
        int base = 0;
        for (int i0 = 0; i0 < N; i0 += kPrepThreads) {
            const int i = i0 + tid;
            int x = i < N && !b ? of(cu[i + 1] - cu[i]) : 0;
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            if (lane == 31) wsum[warp] = x;
            __syncthreads();
            int before = base, all = base;
            for (int w = 0; w < kPrepThreads / 32; ++w) {
                if (w < warp) before += wsum[w];
                all += wsum[w];
            }
            if (i < N) out[i + 1] = before + x;
            base = all;
            __syncthreads();
        }
        return base;
    };
    const int base = sums(seq_tile, [](int len) { return (len + kWinTile - 1) / kWinTile; });
    if (seq_row) sums(seq_row, [&](int len) { return win_rows_of(len, window, sinks); });
    __threadfence_block();
    __syncthreads();
    for (int j = tid; j < ntiles; j += kPrepThreads) {
        int4 e = make_int4(0, 0, 0, 0);
        if (j < base) {
            int lo = 0, hi = N - 1;  // the last sequence whose first tile is <= j
            while (lo < hi) {
                const int m = (lo + hi + 1) >> 1;
                if (seq_tile[m] <= j) lo = m;
                else hi = m - 1;
            }
            e = make_int4(lo, cu[lo], cu[lo + 1] - cu[lo], (j - seq_tile[lo]) * kWinTile);
        }
        tiles[j] = e;
    }
}

// ================================================================ products
__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_from_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// An fp32 value in two tf32 parts, 22 bits.
__device__ __forceinline__ uint2 split(float x) {
    const uint32_t hi = tf32(x);
    return make_uint2(hi, tf32(x - __uint_as_float(hi)));
}
struct Frag {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ void set(int i, uint2 x) { hi[i] = x.x, lo[i] = x.y; }
};
// d += the product of four values of a and two of b. The three products of a step
// are summed from zero, the small ones first, and then added in fp32: the tensor
// core truncates what it accumulates, fp32 sums round (carried on through four steps
// a score was twice as far off).
__device__ __forceinline__ void add_product(float (&d)[4], const Frag &a, uint2 b0, uint2 b1) {
    float z[4];
    mma_from_zero(z, a.lo, b0.x, b1.x);
    mma(z, a.hi, b0.y, b1.y);
    mma(z, a.hi, b0.x, b1.x);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        F2 sum;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(sum.v) : "l"(f2(d[e], d[e + 1]).v), "l"(f2(z[e], z[e + 1]).v));
        f2_get(sum, d[e], d[e + 1]);
    }
}

// 16 warps: four groups of 16 rows times four groups of columns (eight of a tile's
// 32, a quarter of d in the sums). Four warps of 16 rows and all columns were a
// third as fast: one warp on a scheduler waits for its own products most of the time.
constexpr int NT = 512, ROWS = 64, COLS = 32, WS = COLS + 4, PS = COLS + 8;  // WS, PS: floats, pairs to a row of weights

// Rows of a tile in shared memory, split once for all who read them, `S` pairs
// apart. Rows past `rows` are zeros. In two steps, so that the next tile's loads
// are on their way while this one is worked on. The forward reads 16 bytes of two rows
// at a time, RS apart in different banks, and for the weights' products rows VS apart,
// where they are too; a tile that serves as both (in the gradients) is MS apart, read
// 8 bytes at a time (16 at a time there: 979 us instead of 949 for the gradients of 1474 tokens of 15
// heads, window 1227).
template <int D> constexpr int RS = D + 8;
template <int D> constexpr int VS = D + 2;
template <int D> constexpr int MS = D + 4;
template <int D, int N> struct TileLoad {
    static constexpr int PER = D / 4, COUNT = N * PER / NT;
    static_assert(N * PER % NT == 0, "whole rounds");
    float4 v[COUNT];
    __device__ __forceinline__ void load(const float *src, int64_t stride, int rows) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int r = (i * NT + threadIdx.x) / PER, c = (i * NT + threadIdx.x) % PER * 4;
            v[i] = r < rows ? *reinterpret_cast<const float4 *>(src + r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    template <int S> __device__ __forceinline__ void store(uint2 *dst) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int r = (i * NT + threadIdx.x) / PER, c = (i * NT + threadIdx.x) % PER * 4;
            uint4 *d = reinterpret_cast<uint4 *>(dst + r * S + c);
            const uint2 x = split(v[i].x), y = split(v[i].y), z = split(v[i].z), w = split(v[i].w);
            d[0] = make_uint4(x.x, x.y, y.x, y.y);
            d[1] = make_uint4(z.x, z.y, w.x, w.y);
        }
    }
};
struct Place {  // of a thread in the products
    int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
    // its rows are r0 and r0 + 8; a group of rows has a warp on every scheduler, so that rows that are not there
    // (few sinks) leave the others more of each
    int r0 = (warp >> 2) * 16 + g, group = warp & 3;
    __device__ __forceinline__ bool idle(int rows) const { return (warp >> 2) * 16 >= rows; }
    __device__ __forceinline__ void meet() const {  // the four warps of the same rows
        asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp >> 2)) : "memory");
    }
};
// acc = the products of this warp's 16 rows of `a` with its eight of b, S apart.
template <int D, int S> __device__ __forceinline__ void rows_by_rows(float (&acc)[4], const Place &w, const uint2 *a, const uint2 *b) {
    acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
    const uint2 *a0 = a + w.r0 * S + w.t, *b0 = b + (w.group * 8 + w.g) * S + w.t;
#pragma unroll 4
    for (int k = 0; k < D; k += 8) {
        Frag f;
        f.set(0, a0[k]);
        f.set(1, a0[8 * S + k]);
        f.set(2, a0[k + 4]);
        f.set(3, a0[8 * S + k + 4]);
        add_product(acc, f, b0[k], b0[k + 4]);
    }
}
// acc = the products of this warp's 16 rows of `a`, RS apart, with its eight of b, S
// apart. Channels 2 t and 2 t + 1, which a lane reads at once, stand for k = t and
// t + 4 of the product: a sum does not mind the order of its terms.
template <int D, int S> __device__ __forceinline__ void rows_by_rows_16(float (&acc)[4], const Place &w, const uint2 *a, const uint2 *b) {
    acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
    const uint2 *a0 = a + w.r0 * RS<D> + 2 * w.t, *b0 = b + (w.group * 8 + w.g) * S + 2 * w.t;
#pragma unroll 4
    for (int k = 0; k < D; k += 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(a0 + k), y = *reinterpret_cast<const uint4 *>(a0 + 8 * RS<D> + k),
                    z = *reinterpret_cast<const uint4 *>(b0 + k);
        Frag f;
        f.set(0, make_uint2(x.x, x.y)), f.set(1, make_uint2(y.x, y.y));
        f.set(2, make_uint2(x.z, x.w)), f.set(3, make_uint2(y.z, y.w));
        add_product(acc, f, make_uint2(z.x, z.y), make_uint2(z.z, z.w));
    }
}
// acc[nb] += weights (this warp's 16 rows) times its quarter of the rows of b, VS
// apart; columns 2 t and 2 t + 1 of the weights for k = t and t + 4, as above.
template <int D, int S> __device__ __forceinline__ void weights_by_rows(float (&acc)[D / 32][4], const Place &w, const Frag (&f)[COLS / 8], const uint2 *b) {
#pragma unroll
    for (int kb = 0; kb < COLS / 8; ++kb) {
        const uint2 *b0 = b + (kb * 8 + 2 * w.t) * S + w.group * (D / 4) + w.g;
#pragma unroll
        for (int nb = 0; nb < D / 32; ++nb) add_product(acc[nb], f[kb], b0[nb * 8], b0[S + nb * 8]);
    }
}
__device__ __forceinline__ void put_weights(float *w, const Place &p, const float (&s)[4]) {
    *reinterpret_cast<float2 *>(w + p.r0 * WS + p.group * 8 + 2 * p.t) = make_float2(s[0], s[1]);
    *reinterpret_cast<float2 *>(w + (p.r0 + 8) * WS + p.group * 8 + 2 * p.t) = make_float2(s[2], s[3]);
}
__device__ __forceinline__ void get_weights(Frag (&f)[COLS / 8], const float *w, const Place &p) {
#pragma unroll
    for (int kb = 0; kb < COLS / 8; ++kb) {
        const float2 x = *reinterpret_cast<const float2 *>(w + p.r0 * WS + kb * 8 + 2 * p.t);
        const float2 y = *reinterpret_cast<const float2 *>(w + (p.r0 + 8) * WS + kb * 8 + 2 * p.t);
        f[kb].set(0, split(x.x)), f[kb].set(1, split(y.x)), f[kb].set(2, split(x.y)), f[kb].set(3, split(y.y));
    }
}

// ================================================================ the general kernels
struct WinParams {
    WinGeom geo;
    const void *q, *k, *v, *out, *d_o;
    int64_t q_stride, k_stride, v_stride;
    float scale;
    void *o, *dq, *dk, *dv;
    float *lse;               // [tokens][hq], of the forward
    float *lse_h, *delta;     // [hq][tokens], of the gradients: lse, D
    float *part, *near;       // gradients of the sinks, see win_far_sum_kernel
    int fars, ranks;          // blocks of far pairs, which come first; CTAs to a block, which share its query heads
};

// Whether i sees j, among the near pairs or among the far ones.
__device__ __forceinline__ bool sees(int i, int j, int window, int sinks, bool far) {
    return far ? j < sinks && i - j >= window : j <= i && i - j < window;
}
// Token i sees itself alone: its weight is one whatever its score, so ds is zero.
__device__ __forceinline__ bool alone(int i, int window, int sinks) { return i == 0 || (window == 1 && sinks == 0); }

template <int D>
__global__ void __launch_bounds__(NT)
win_forward_kernel(WinParams p) {
    extern __shared__ __align__(16) uint2 sm[];
    uint2 *sq = sm, *sk = sq + ROWS * RS<D>, *sv = sk + COLS * RS<D>;
    uint2 *ws = sv + COLS * VS<D>;                                // weights, split [ROWS][PS]
    float *shared = reinterpret_cast<float *>(ws + ROWS * PS);  // [ROWS][4]: of the warps of the same rows
    const WinGeom &geo = p.geo;
    const int item = gridDim.x - 1 - blockIdx.x, at = geo.by_hq.div(item), h = item - at * geo.hq, hk = h / geo.group;
    const WinTile tile = win_tile(geo, at >> 2);
    const int i0 = tile.first + (at & 3) * ROWS, rows = min(ROWS, tile.len - i0);
    if (rows <= 0) return;
    const Place w;
    const float *kb = (const float *)p.k + (int64_t)tile.start * p.k_stride + hk * D;
    const float *vb = (const float *)p.v + (int64_t)tile.start * p.v_stride + hk * D;
    {
        TileLoad<D, ROWS> q;
        q.load((const float *)p.q + (int64_t)(tile.start + i0) * p.q_stride + h * D, p.q_stride, rows);
        q.template store<RS<D>>(sq);
    }
    TileLoad<D, COLS> nk, nv;
    float acc[D / 32][4], m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int nb = 0; nb < D / 32; ++nb) acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
    auto walk = [&](int from, int to, bool far) {
        auto fetch = [&](int j0) {
            nk.load(kb + (int64_t)j0 * p.k_stride, p.k_stride, to - j0);
            nv.load(vb + (int64_t)j0 * p.v_stride, p.v_stride, to - j0);
        };
        if (from < to) fetch(from);
        for (int j0 = from; j0 < to; j0 += COLS) {
            __syncthreads();
            nk.template store<RS<D>>(sk);
            nv.template store<VS<D>>(sv);
            __syncthreads();
            if (j0 + COLS < to) fetch(j0 + COLS);
            if (w.idle(rows)) continue;
            // a warp has eight of the tile's columns: it makes their weights with the rows' maximum over all four
            float s[4], keep[2];
            rows_by_rows_16<D, RS<D>>(s, w, sq, sk);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + w.r0 + (e >> 1) * 8, j = j0 + w.group * 8 + 2 * w.t + (e & 1);
                s[e] = j < to && sees(i, j, geo.window, geo.sinks, far) ? s[e] * p.scale : -CUDART_INF_F;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float top = fmaxf(s[2 * r], s[2 * r + 1]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (w.t == 0) shared[(w.r0 + 8 * r) * 4 + w.group] = top;
            }
            w.meet();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float4 y = *reinterpret_cast<const float4 *>(shared + (w.r0 + 8 * r) * 4);
                const float top = fmaxf(m[r], fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w)));
                keep[r] = top == -CUDART_INF_F ? 1.f : expf(m[r] - top);  // a row may see nothing of a tile
                m[r] = top;
                const float a = s[2 * r] == -CUDART_INF_F ? 0.f : expf(s[2 * r] - top),
                            b = s[2 * r + 1] == -CUDART_INF_F ? 0.f : expf(s[2 * r + 1] - top);
                l[r] = fmaf(l[r], keep[r], a + b);  // of this lane's columns
                const uint2 x = split(a), z = split(b);
                *reinterpret_cast<uint4 *>(ws + (w.r0 + 8 * r) * PS + w.group * 8 + 2 * w.t) = make_uint4(x.x, x.y, z.x, z.y);
            }
            w.meet();
            Frag f[COLS / 8];
#pragma unroll
            for (int k = 0; k < COLS / 8; ++k) {
                const uint4 x = *reinterpret_cast<const uint4 *>(ws + w.r0 * PS + k * 8 + 2 * w.t),
                            y = *reinterpret_cast<const uint4 *>(ws + (w.r0 + 8) * PS + k * 8 + 2 * w.t);
                f[k].set(0, make_uint2(x.x, x.y)), f[k].set(1, make_uint2(y.x, y.y));
                f[k].set(2, make_uint2(x.z, x.w)), f[k].set(3, make_uint2(y.z, y.w));
            }
#pragma unroll
            for (int nb = 0; nb < D / 32; ++nb) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nb][e] *= keep[e >> 1];
            }
            weights_by_rows<D, VS<D>>(acc, w, f, sv);
        }
    };
    if (i0 + rows > geo.window) walk(0, min(geo.sinks, i0 + rows - geo.window), true);
    walk(max(0, i0 - geo.window + 1), i0 + rows, false);
    w.meet();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if (w.t == 0) shared[(w.r0 + 8 * e) * 4 + w.group] = l[e];
    }
    w.meet();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float4 y = *reinterpret_cast<const float4 *>(shared + (w.r0 + 8 * e) * 4);
        l[e] = (y.x + y.y) + (y.z + y.w);
        const int r = w.r0 + e * 8;
        if (r >= rows) continue;
        const int64_t row = (int64_t)(tile.start + i0 + r) * geo.hq + h;
        float *o = (float *)p.o + row * D + w.group * (D / 4) + 2 * w.t;
        const float f = 1.f / l[e];
#pragma unroll
        for (int nb = 0; nb < D / 32; ++nb)
            *reinterpret_cast<float2 *>(o + nb * 8) = make_float2(acc[nb][2 * e] * f, acc[nb][2 * e + 1] * f);
        if (p.lse && w.t == 0 && w.group == 0) p.lse[row] = m[e] + logf(l[e]);
    }
}

// D_i = do_i . o_i, and lse, both by head: a tile of queries is a stretch of memory
// then. (bf16 calls, whose o is rounded, take D from the products: kda_window_tc.cu.)
// A block takes eight tokens of every head, in the order of memory, and writes a
// sector of each head's; a row is 16 bytes in each of d / 4 lanes.
template <int D>
__global__ void __launch_bounds__(256)
win_delta_kernel(const float *o, const float *d_o, const float *lse, float *lse_h, float *delta, int64_t tokens, int hq) {
    constexpr int LANES = D / 4, PER = 256 / LANES, FLIGHT = 4;
    extern __shared__ float sums[];  // [hq][8]
    let_next_start();
    const int in = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const int64_t t0 = (int64_t)blockIdx.x * 8;
    const int count = (int)(tokens - t0 < 8 ? tokens - t0 : 8), rows = count * hq;
    const float *ob = o + t0 * hq * D + in * 4, *db = d_o + t0 * hq * D + in * 4;
    for (int r0 = 0; r0 < rows; r0 += FLIGHT * PER) {
        float4 a[FLIGHT], b[FLIGHT];
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            const int r = r0 + i * PER + sub;
            a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                a[i] = *reinterpret_cast<const float4 *>(ob + (int64_t)r * D), b[i] = *reinterpret_cast<const float4 *>(db + (int64_t)r * D);
        }
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            float s = fmaf(a[i].w, b[i].w, fmaf(a[i].z, b[i].z, fmaf(a[i].y, b[i].y, a[i].x * b[i].x)));
#pragma unroll
            for (int off = LANES / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            const int r = r0 + i * PER + sub;
            if (in == 0 && r < rows) sums[r % hq * 8 + r / hq] = s;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * hq; i += 256) {
        const int h = i >> 3, t = i & 7;
        if (t >= count) continue;
        delta[h * tokens + t0 + t] = sums[i];
        lse_h[h * tokens + t0 + t] = lse[(t0 + t) * hq + h];
    }
}

template <int D>
__global__ void __launch_bounds__(NT)
win_dq_kernel(WinParams p) {
    extern __shared__ __align__(16) uint2 sm[];
    uint2 *sq = sm, *sd = sq + ROWS * MS<D>, *sv = sd + ROWS * MS<D>, *sk = sv + COLS * MS<D>;
    float *ws = reinterpret_cast<float *>(sk + COLS * MS<D>);
    const WinGeom &geo = p.geo;
    const int item = gridDim.x - 1 - blockIdx.x, at = geo.by_hq.div(item), h = item - at * geo.hq, hk = h / geo.group;
    const WinTile tile = win_tile(geo, at >> 2);
    const int i0 = tile.first + (at & 3) * ROWS, rows = min(ROWS, tile.len - i0);
    if (rows <= 0) {
        await_previous();
        return;
    }
    const Place w;
    const float *kb = (const float *)p.k + (int64_t)tile.start * p.k_stride + hk * D;
    const float *vb = (const float *)p.v + (int64_t)tile.start * p.v_stride + hk * D;
    const int64_t row0 = (int64_t)(tile.start + i0) * geo.hq + h, vec0 = (int64_t)h * geo.tokens + tile.start + i0;
    {
        TileLoad<D, ROWS> q, d;
        q.load((const float *)p.q + (int64_t)(tile.start + i0) * p.q_stride + h * D, p.q_stride, rows);
        d.load((const float *)p.d_o + row0 * D, (int64_t)geo.hq * D, rows);
        q.template store<MS<D>>(sq);
        d.template store<MS<D>>(sd);
    }
    TileLoad<D, COLS> nk, nv;
    float acc[D / 32][4], lse[2], delta[2];
#pragma unroll
    for (int nb = 0; nb < D / 32; ++nb) acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const bool there = w.r0 + e * 8 < rows;
        lse[e] = there ? p.lse_h[vec0 + w.r0 + e * 8] : 0.f;
        delta[e] = there ? p.delta[vec0 + w.r0 + e * 8] : 0.f;
    }
    auto walk = [&](int from, int to, bool far) {
        auto fetch = [&](int j0) {
            nk.load(kb + (int64_t)j0 * p.k_stride, p.k_stride, to - j0);
            nv.load(vb + (int64_t)j0 * p.v_stride, p.v_stride, to - j0);
        };
        if (from < to) fetch(from);
        for (int j0 = from; j0 < to; j0 += COLS) {
            __syncthreads();
            nk.template store<MS<D>>(sk);
            nv.template store<MS<D>>(sv);
            __syncthreads();
            if (j0 + COLS < to) fetch(j0 + COLS);
            if (!w.idle(rows)) {
                float s[4], dp[4];
                rows_by_rows<D, MS<D>>(s, w, sq, sk);
                rows_by_rows<D, MS<D>>(dp, w, sd, sv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + w.r0 + (e >> 1) * 8, j = j0 + w.group * 8 + 2 * w.t + (e & 1);
                    const bool on = j < to && sees(i, j, geo.window, geo.sinks, far) && !alone(i, geo.window, geo.sinks);
                    s[e] = on ? expf(fmaf(s[e], p.scale, -lse[e >> 1])) * (dp[e] - delta[e >> 1]) : 0.f;
                }
                put_weights(ws, w, s);
            }
            __syncthreads();
            if (w.idle(rows)) continue;
            Frag f[COLS / 8];
            get_weights(f, ws, w);
            weights_by_rows<D, MS<D>>(acc, w, f, sk);
        }
    };
    if (i0 + rows > geo.window) walk(0, min(geo.sinks, i0 + rows - geo.window), true);
    walk(max(0, i0 - geo.window + 1), i0 + rows, false);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = w.r0 + e * 8;
        if (r >= rows) continue;
        float *dq = (float *)p.dq + (row0 + (int64_t)r * geo.hq) * D + w.group * (D / 4) + 2 * w.t;
#pragma unroll
        for (int nb = 0; nb < D / 32; ++nb)
            *reinterpret_cast<float2 *>(dq + nb * 8) = make_float2(acc[nb][2 * e] * p.scale, acc[nb][2 * e + 1] * p.scale);
    }
    await_previous();  // whoever comes next waits for both kernels
}

// dk and dv of 64 keys; the first p.fars blocks: of the sinks, from the far pairs
// with one tile of 256 queries, whose sums go to `part`.
template <int D>
__global__ void __launch_bounds__(NT)
win_dkv_kernel(WinParams p) {
    extern __shared__ __align__(16) uint2 sm[];
    uint2 *sk = sm, *sv = sk + ROWS * MS<D>, *sq = sv + ROWS * MS<D>, *sd = sq + COLS * MS<D>;
    float *wp = reinterpret_cast<float *>(sd + COLS * MS<D>), *wd = wp + ROWS * WS;
    await_previous();  // in this order: dq starts early and reads what this kernel waited for
    let_next_start();
    const WinGeom &geo = p.geo;
    const int rank = blockIdx.x % p.ranks, block = blockIdx.x / p.ranks;
    const bool far = block < p.fars;
    const int item = far ? block : block - p.fars, at = geo.by_hk.div(item), hk = item - at * geo.hk;
    const WinTile tile = win_tile(geo, far ? at >> 1 : at >> 2);
    const int j0 = far ? (at & 1) * ROWS : tile.first + (at & 3) * ROWS;
    const int rows = min(ROWS, (far ? min(geo.sinks, tile.len) : tile.len) - j0);
    if (rows <= 0 || (far && min(tile.first + kWinTile, tile.len) <= geo.window)) return;  // no far query either
    const int from = far ? max(tile.first, j0 + geo.window) : j0;
    const int to = far ? min(tile.first + kWinTile, tile.len)
                       : (int)min((int64_t)tile.len, (int64_t)j0 + rows - 1 + geo.window);
    const Place w;
    {
        TileLoad<D, ROWS> k, v;
        k.load((const float *)p.k + (int64_t)(tile.start + j0) * p.k_stride + hk * D, p.k_stride, rows);
        v.load((const float *)p.v + (int64_t)(tile.start + j0) * p.v_stride + hk * D, p.v_stride, rows);
        k.template store<MS<D>>(sk);
        v.template store<MS<D>>(sv);
    }
    TileLoad<D, COLS> nq, nd;
    float lse[2], delta[2];  // of the step's queries in this thread's columns, and of the next step's
    float next_lse[2], next_delta[2];
    float ak[D / 32][4], av[D / 32][4];
#pragma unroll
    for (int nb = 0; nb < D / 32; ++nb) {
        ak[nb][0] = ak[nb][1] = ak[nb][2] = ak[nb][3] = 0.f;
        av[nb][0] = av[nb][1] = av[nb][2] = av[nb][3] = 0.f;
    }
    auto fetch = [&](int h, int i0) {
        const int64_t row0 = (int64_t)(tile.start + i0) * geo.hq + h;
        nq.load((const float *)p.q + (int64_t)(tile.start + i0) * p.q_stride + h * D, p.q_stride, to - i0);
        nd.load((const float *)p.d_o + row0 * D, (int64_t)geo.hq * D, to - i0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = i0 + w.group * 8 + 2 * w.t + e;
            const int64_t x = (int64_t)h * geo.tokens + tile.start + i;
            next_lse[e] = i < to ? p.lse_h[x] : 0.f;
            next_delta[e] = i < to ? p.delta[x] : 0.f;
        }
    };
    const int heads = geo.group / p.ranks;
    int h = hk * geo.group + rank * heads, i0 = from;
    const int h_end = h + heads;
    if (from < to) fetch(h, i0);
    while (from < to && h < h_end) {
        __syncthreads();
        nq.template store<MS<D>>(sq);
        nd.template store<MS<D>>(sd);
#pragma unroll
        for (int e = 0; e < 2; ++e) lse[e] = next_lse[e], delta[e] = next_delta[e];
        __syncthreads();
        const int i_now = i0;
        if ((i0 += COLS) >= to) i0 = from, ++h;
        if (h < h_end) fetch(h, i0);
        if (!w.idle(rows)) {
            float s[4], dp[4];
            rows_by_rows<D, MS<D>>(s, w, sk, sq);
            rows_by_rows<D, MS<D>>(dp, w, sv, sd);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = w.r0 + (e >> 1) * 8, i = i_now + w.group * 8 + 2 * w.t + (e & 1);
                const bool on = r < rows && i < to && sees(i, j0 + r, geo.window, geo.sinks, far);
                s[e] = on ? expf(fmaf(s[e], p.scale, -lse[e & 1])) : 0.f;
                dp[e] = on && !alone(i, geo.window, geo.sinks) ? s[e] * (dp[e] - delta[e & 1]) : 0.f;
            }
            put_weights(wp, w, s);
            put_weights(wd, w, dp);
        }
        __syncthreads();
        if (w.idle(rows)) continue;
        Frag f[COLS / 8];
        get_weights(f, wp, w);
        weights_by_rows<D, MS<D>>(av, w, f, sd);
        get_weights(f, wd, w);
        weights_by_rows<D, MS<D>>(ak, w, f, sq);
    }
    // where row r of dk goes, and how far behind it that of dv lies
    auto place = [&](int r, int c, float *&dk, float *&dv) {
        const int j = j0 + r;
        const int64_t row = ((int64_t)(tile.start + j) * geo.hk + hk) * D + c;
        dk = (float *)p.dk + row, dv = (float *)p.dv + row;
        if (far) {
            dk = p.part + ((win_far_row(geo, tile.seq, tile.start, tile.first, kWinTile) + j) * geo.hk + hk) * 2 * D + c;
            dv = dk + D;
        } else if (j < geo.sinks && tile.len > geo.window) {
            dk = p.near + ((int64_t)(win_near_row(geo, tile.seq) + j) * geo.hk + hk) * 2 * D + c;
            dv = dk + D;
        }
    };
    float *own = reinterpret_cast<float *>(sm);  // [2][ROWS][D + 8]: this CTA's dk and dv, for the cluster
    constexpr int OS = D + 8;
    if (p.ranks > 1) __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = w.r0 + e * 8, c = w.group * (D / 4) + 2 * w.t;
        if (r >= rows) continue;
        float *dk = own + r * OS + c, *dv = dk + ROWS * OS;
        if (p.ranks == 1) place(r, c, dk, dv);
#pragma unroll
        for (int nb = 0; nb < D / 32; ++nb) {
            *reinterpret_cast<float2 *>(dk + nb * 8) = make_float2(ak[nb][2 * e] * p.scale, ak[nb][2 * e + 1] * p.scale);
            *reinterpret_cast<float2 *>(dv + nb * 8) = make_float2(av[nb][2 * e], av[nb][2 * e + 1]);
        }
    }
    if (p.ranks == 1) return;
    tc::cluster_sync();
    // each CTA adds up its share of the rows, in the order of the heads
    const uint32_t mine = tc::smem_u32(own);
    for (int x = rank * NT + threadIdx.x; x < rows * (D / 4); x += p.ranks * NT) {
        const int r = x / (D / 4), c = x % (D / 4) * 4;
        float *dst[2];
        place(r, c, dst[0], dst[1]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < p.ranks; ++k) {
                float4 y;
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                             : "r"(tc::mapa(mine + ((u * ROWS + r) * OS + c) * 4, k))
                             : "memory");
                sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
            }
            *reinterpret_cast<float4 *>(dst[u]) = sum;
        }
    }
    tc::cluster_sync();  // nobody leaves while others read its rows
}

// dk and dv of the sinks that far queries see: the rows of `near`, from the queries
// within the window, and those of the far queries' parts (see win_far_row), added in
// order, every eighth part first, so that eight loads are on their way. A thread takes
// four channels, in the order of memory. (Rows times key heads are below 2^31: as many
// rows of k, v, dk and dv lie in memory.)
template <typename T>
__global__ void __launch_bounds__(256)
win_far_sum_kernel(WinGeom geo, const float *part, const float *near, T *dk, T *dv, int d, int queries) {
    const int quads = d / 2;  // fours of channels of a row's [2][d]
    const int64_t all = (int64_t)(geo.seq_row ? geo.seq_row[geo.N] : geo.N * geo.rows_each) * geo.hk * quads;
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < all; x += (int64_t)gridDim.x * 256) {
        const int at = (int)(x / quads), c = (int)(x - (int64_t)at * quads) * 4, row = geo.by_hk.div(at), hk = at - row * geo.hk;
        int n = 0, sink, start, len = geo.T;
        if (geo.seq_row) {
            int hi = geo.N - 1;  // the last sequence whose first row is <= row
            while (n < hi) {
                const int m = (n + hi + 1) >> 1;
                if (geo.seq_row[m] <= row) n = m;
                else hi = m - 1;
            }
            sink = row - geo.seq_row[n];
            const int4 tile = geo.tiles[geo.seq_tile[n]];
            start = tile.y, len = tile.z;
        } else {
            n = row / geo.rows_each, sink = row - n * geo.rows_each, start = n * geo.T;
        }
        float4 a[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) a[g] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int last = (len - 1) / queries;
        for (int k0 = geo.window / queries; k0 <= last; k0 += 8) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                if (k0 + g > last) continue;
                const int64_t from = win_far_row(geo, n, start, (k0 + g) * queries, queries) + sink;
                const float4 y = *reinterpret_cast<const float4 *>(part + (from * geo.hk + hk) * 2 * d + c);
                a[g].x += y.x, a[g].y += y.y, a[g].z += y.z, a[g].w += y.w;
            }
        }
#pragma unroll
        for (int g = 1; g < 8; ++g) a[0].x += a[g].x, a[0].y += a[g].y, a[0].z += a[g].z, a[0].w += a[g].w;
        const float4 y = *reinterpret_cast<const float4 *>(near + (int64_t)at * 2 * d + c);
        T *dst = (c < d ? dk : dv) + ((int64_t)(start + sink) * geo.hk + hk) * d + (c < d ? c : c - d);
        const float v[4] = {a[0].x + y.x, a[0].y + y.y, a[0].z + y.z, a[0].w + y.w};
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            const __nv_bfloat162 z[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
            *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(z);
        }
    }
}

// ================================================================ host side
constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct WinPlan {
    WinGeom geo;
    int4 *tiles;
    int32_t *seq_tile, *seq_row;
    float *lse_h, *delta, *part, *near;
    size_t bytes;
};
WinPlan make_plan(int N, int64_t T, int hq, int hk, int d, int window, int sinks, bool packed, bool back, bool bf16, void *ws) {
    WinPlan p{};
    WinGeom &g = p.geo;
    g.N = N, g.T = (int)T, g.hq = hq, g.hk = hk, g.group = hq / hk;
    g.window = window, g.sinks = sinks;
    g.tokens = packed ? T : (int64_t)N * T;
    g.per_seq = (int)((T + kWinTile - 1) / kWinTile);
    g.ntiles = packed ? (int)(T / kWinTile) + N : N * g.per_seq;
    g.by_seq = FastDiv(g.per_seq > 0 ? g.per_seq : 1);
    g.by_hq = FastDiv(hq), g.by_hk = FastDiv(hk);
    char *base = static_cast<char *>(ws);
    auto take = [&](size_t n) {
        char *at = base ? base + p.bytes : nullptr;
        p.bytes += round256(n);
        return at;
    };
    if (packed) {
        p.tiles = reinterpret_cast<int4 *>(take(sizeof(int4) * (size_t)g.ntiles));
        p.seq_tile = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * ((size_t)N + 1)));
        g.tiles = p.tiles, g.seq_tile = p.seq_tile;
    }
    if (back) {
        p.lse_h = reinterpret_cast<float *>(take(sizeof(float) * (size_t)g.tokens * hq));
        p.delta = reinterpret_cast<float *>(take(sizeof(float) * (size_t)g.tokens * hq));
        if (sinks > 0) {
            const int64_t rows = win_rows(N, g.tokens, sinks), of = sizeof(float) * 2 * hk * d;
            g.rows = (int)rows, g.rows_each = win_rows_of(g.T, window, sinks);
            p.part = reinterpret_cast<float *>(take((rows + win_part_rows(g.tokens, sinks, bf16 ? kWinFarQueries : kWinTile)) * of));
            p.near = reinterpret_cast<float *>(take(rows * of));
            if (packed) g.seq_row = p.seq_row = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * ((size_t)N + 1)));
        }
    }
    return p;
}

#define KDA_TRY(x)                             \
    do {                                       \
        const cudaError_t e_ = (x);            \
        if (e_ != cudaSuccess) return e_;      \
    } while (0)

cudaError_t prepare_tiles(const WinPlan &p, const WinArgs &a, cudaStream_t s) {
    if (!a.cu_seqlens) return cudaSuccess;
    win_tiles_kernel<<<1, kPrepThreads, 0, s>>>(a.cu_seqlens, a.N, a.T, p.geo.ntiles, p.tiles, p.seq_tile, p.seq_row, a.window,
                                                a.sinks, a.status);
    return cudaGetLastError();
}
WinParams params(const WinPlan &p, const WinArgs &a) {
    WinParams w{};
    w.geo = p.geo;
    w.q = a.q, w.k = a.k, w.v = a.v, w.out = a.out, w.d_o = a.d_o;
    w.q_stride = a.q_stride, w.k_stride = a.k_stride, w.v_stride = a.v_stride;
    w.scale = a.scale;
    w.o = a.o, w.dq = a.dq, w.dk = a.dk, w.dv = a.dv;
    w.lse = a.lse, w.lse_h = p.lse_h, w.delta = p.delta, w.part = p.part, w.near = p.near;
    return w;
}
template <typename... P>
cudaError_t run(void (*kernel)(P...), std::atomic<uint64_t> &allowed, unsigned grid, size_t smem, Launches &l, P... args) {
    KDA_TRY(allow_smem(kernel, smem, allowed));
    return l.next(kernel, grid, NT, smem, args...);
}

template <int D> cudaError_t forward(const WinPlan &p, const WinArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    constexpr size_t smem = ((ROWS + COLS) * RS<D> + COLS * VS<D> + ROWS * PS) * sizeof(uint2) + ROWS * 4 * sizeof(float);
    Launches l{s};
    return run(win_forward_kernel<D>, allowed, (unsigned)(p.geo.ntiles * 4 * a.hq), smem, l, params(p, a));
}

template <typename T, int D> cudaError_t backward(const WinPlan &p, const WinArgs &a, cudaStream_t s) {
    WinParams w = params(p, a);
    Launches l{s};
    const bool far = a.sinks > 0 && a.window < a.T;  // some sequence may be longer than the window
    if constexpr (sizeof(T) == 2) {
        KDA_TRY(launch_window_backward_tc(p.geo, a, p.lse_h, p.delta, p.part, p.near, l));
    } else {
        KDA_TRY(l.next(win_delta_kernel<D>, (unsigned)((p.geo.tokens + 7) / 8), 256, a.hq * 8 * sizeof(float),
                       (const float *)a.out, (const float *)a.d_o, a.lse, p.lse_h, p.delta, p.geo.tokens, a.hq));
        static std::atomic<uint64_t> allowed[2];
        constexpr size_t weights = ROWS * WS * sizeof(float);
        constexpr size_t dq = (2 * ROWS + 2 * COLS) * MS<D> * sizeof(uint2) + weights, dkv = dq + weights;
        static_assert(dkv <= 232448 && dq <= 232448 && 2 * ROWS * (D + 8) * sizeof(float) <= dkv, "shared memory of a block");
        w.fars = far ? p.geo.ntiles * 2 * a.hk : 0;
        // The query heads of a key head go to the CTAs of a cluster, or few key heads would leave most SMs idle. How
        // many depends on the group alone: a sequence has the same bits in any batch.
        w.ranks = 1;
        for (int r = 2; r <= 5; ++r)
            if (p.geo.group % r == 0) w.ranks = r;
        KDA_TRY(allow_smem(win_dkv_kernel<D>, dkv, allowed[0]));
        KDA_TRY(l.next_clusters(win_dkv_kernel<D>, (unsigned)(w.fars + p.geo.ntiles * 4 * a.hk), w.ranks, NT, dkv, w));
        KDA_TRY(run(win_dq_kernel<D>, allowed[1], (unsigned)(p.geo.ntiles * 4 * a.hq), dq, l, w));
    }
    if (far) {
        const int64_t blocks = ((int64_t)p.geo.rows * a.hk * (D / 2) + 255) / 256;  // at most; 152 SMs, eight on each
        win_far_sum_kernel<T><<<blocks < 152 * 8 ? (unsigned)blocks : 152 * 8, 256, 0, s>>>(
            p.geo, p.part, p.near, (T *)a.dk, (T *)a.dv, D, sizeof(T) == 2 ? kWinFarQueries : kWinTile);
    }
    return cudaGetLastError();
}

}  // namespace

size_t window_workspace_bytes(int N, int64_t T, int hq, int hk, int d, int sinks, kda_dtype_t dt, bool packed, bool back) {
    return make_plan(N, T, hq, hk, d, 1, sinks, packed, back, dt == KDA_BF16, nullptr).bytes;
}

cudaError_t launch_window(const WinArgs &a, cudaStream_t s) {
    const WinPlan p = make_plan(a.N, a.T, a.hq, a.hk, a.d, a.window, a.sinks, a.cu_seqlens != nullptr, false, a.dt == KDA_BF16,
                                a.workspace);
    KDA_TRY(prepare_tiles(p, a, s));
    if (p.geo.tokens == 0) return cudaSuccess;
    if (a.dt == KDA_BF16) return launch_window_forward_tc(p.geo, a, s);
    return a.d == 128 ? forward<128>(p, a, s) : forward<64>(p, a, s);
}

cudaError_t launch_window_backward(const WinArgs &a, cudaStream_t s) {
    const WinPlan p = make_plan(a.N, a.T, a.hq, a.hk, a.d, a.window, a.sinks, a.cu_seqlens != nullptr, true, a.dt == KDA_BF16,
                                a.workspace);
    KDA_TRY(prepare_tiles(p, a, s));
    if (p.geo.tokens == 0) return cudaSuccess;
    if (a.dt == KDA_BF16) return a.d == 128 ? backward<__nv_bfloat16, 128>(p, a, s) : backward<__nv_bfloat16, 64>(p, a, s);
    return a.d == 128 ? backward<float, 128>(p, a, s) : backward<float, 64>(p, a, s);
}

}  // namespace kda
