// Norm of every query and key head and the rotary positions, one pass each way.
//
//   n = x r,  r = 1 / sqrt(sum x^2 + eps)      (KDA_NORM_L2)
//             r = 1 / sqrt(sum x^2 / d + eps)  (KDA_NORM_RMS), r = 1 (NONE)
//   y = R(position) (w * n)
// with R turning channel pairs of the first `rot` channels by the angles whose
// cosines and sines the token's table row holds. Backward, for u = R^T dy:
//   dw = sum over rows of u n,   dn = w u,
//   dx = r (dn - n (n . dn) c),   c = 1 (L2), 1 / d (RMS), 0 (NONE).
//
// Bound by memory: forward one read and one write of q and k, backward two
// reads and one write; right behind it come the instructions, so the
// arithmetic goes two channels at a time (f32x2) and is arranged for few steps.
// A row (one head of one token) is held by 16 bytes in each of
// d * sizeof(T) / 16 lanes, so a warp reads 512 contiguous bytes at a time;
// every warp takes one token's rows four passes at once (2 KB in flight per
// warp) and keeps that token's angles in registers. With x' the partner of
// channel x (the half layout's comes from another lane, as it was loaded, so a
// shuffle moves two bf16 channels),
//   y = r (A x + B x'),  A = cos w,  B = -+ sin w',
// with A and B made once per token. Sums, norms and the rotation are in fp32;
// the only rounding to fewer bits is the store. 16384 tokens x (16 + 16) heads
// of 128 bf16 channels: forward 51.3 us (5.3 TB/s, 78 % of a copy), backward with
// both weights' gradients 73 (5.5 TB/s, 82 %), the last sum included (79 with the
// partners and both sums of a row by shuffles of their own: backward, the partners'
// pieces are in shared memory). With positions of three axes: in blocks of four pairs
// (16 bytes of the table at a time) 61 and 75, in turn over the pairs (4 bytes at a
// time) 66 and 79.
#include "kda_internal.cuh"
#include "kda_linear.cuh"
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPasses = 4;  // row groups of a warp in flight at once

// This lane's cosines and sines: element e of the lane's channels sits in
// pair (channel mod rot/2) of the half layout, channel / 2 of the interleaved.
// sn is signed for the element it multiplies into: the first of a pair takes
// its partner with a minus.
template <int N>
__device__ __forceinline__ void load_angles(const float *row, int c0, int rot, int layout, float (&cs)[N],
                                            float (&sn)[N]) {
    const int h = rot / 2;
    if (c0 >= rot) {
#pragma unroll
        for (int e = 0; e < N; ++e) cs[e] = 1.f, sn[e] = 0.f;
    } else if (layout == KDA_ROPE_HALF) {
        const int i0 = c0 < h ? c0 : c0 - h;
        load_floats<N>(row + i0, cs);
        load_floats<N>(row + h + i0, sn);
        if (c0 < h) {
#pragma unroll
            for (int e = 0; e < N; ++e) sn[e] = -sn[e];
        }
    } else {
        float c[N / 2], t[N / 2];
        load_floats<N / 2>(row + c0 / 2, c);
        load_floats<N / 2>(row + h + c0 / 2, t);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            cs[2 * e] = cs[2 * e + 1] = c[e];
            sn[2 * e] = -t[e];
            sn[2 * e + 1] = t[e];
        }
    }
}

// Positions of several axes: channel pair i turns by the table's row of its own
// axis' position. Aligned groups of four pairs that share an axis are read with
// one load (p.quads: all of them do, as with sections of a multiple of four
// pairs), others pair by pair.
__device__ __forceinline__ int pair_axis(const NormRopeArgs &p, int pair) {
    return (int)(p.axis_bits[pair >> 5] >> (2 * (pair & 31))) & 3;
}
struct AxisPositions {
    int at[kRopeAxes];
    // `mine`: in lane a of the warp, axis a's
    __device__ __forceinline__ explicit AxisPositions(int mine) {
#pragma unroll
        for (int a = 0; a < kRopeAxes; ++a) at[a] = __shfl_sync(0xffffffffu, mine, a);
    }
    __device__ __forceinline__ int of(int axis) const {
        return axis < 2 ? (axis == 0 ? at[0] : at[1]) : (axis == 2 ? at[2] : at[3]);
    }
};
// A token's positions, lane a of the warp axis a's (lanes behind the axes: axis 0's).
__device__ __forceinline__ int axis_position(const NormRopeArgs &p, int64_t token) {
    const int lane = threadIdx.x & 31;
    return __ldg(p.positions + (lane < p.axes ? lane : 0) * p.tokens + token);
}
__device__ __forceinline__ bool all_in_table(const NormRopeArgs &p, int mine) {
    return __all_sync(0xffffffffu, mine >= 0 && mine < p.max_position);
}
// N values of pairs i0 .. i0 + N - 1, from column `col` + pair of each pair's row
template <int N>
__device__ __forceinline__ void load_pairs(const NormRopeArgs &p, const AxisPositions &pos, int i0, int col, float *x) {
    constexpr int STEP = N < 4 ? N : 4;
    if (p.quads) {
#pragma unroll
        for (int e = 0; e < N; e += STEP)
            load_floats<STEP>(p.table + (int64_t)pos.of(pair_axis(p, i0 + e)) * p.rot + col + i0 + e, x + e);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] = __ldg(p.table + (int64_t)pos.of(pair_axis(p, i0 + e)) * p.rot + col + i0 + e);
    }
}
// load_angles of a row that is put together from every pair's axis.
template <int N>
__device__ __forceinline__ void load_axis_angles(const NormRopeArgs &p, const AxisPositions &pos, int c0, float (&cs)[N],
                                                 float (&sn)[N]) {
    const int h = p.rot / 2;
    if (c0 >= p.rot) {
#pragma unroll
        for (int e = 0; e < N; ++e) cs[e] = 1.f, sn[e] = 0.f;
    } else if (p.layout == KDA_ROPE_HALF) {
        const int i0 = c0 < h ? c0 : c0 - h;
        load_pairs<N>(p, pos, i0, 0, cs);
        load_pairs<N>(p, pos, i0, h, sn);
        if (c0 < h) {
#pragma unroll
            for (int e = 0; e < N; ++e) sn[e] = -sn[e];
        }
    } else {
        float c[N / 2], t[N / 2];
        load_pairs<N / 2>(p, pos, c0 / 2, 0, c);
        load_pairs<N / 2>(p, pos, c0 / 2, h, t);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            cs[2 * e] = cs[2 * e + 1] = c[e];
            sn[2 * e] = -t[e];
            sn[2 * e + 1] = t[e];
        }
    }
}

struct Geometry {
    int lane_row;  // which of the warp's rows this lane works on
    int c0;        // first channel of the lane
    int src;       // lane of the partner channels (half layout)
    bool rotated;  // the lane's channels lie in the rotated part
};
template <typename T, int D> __device__ __forceinline__ Geometry geometry(int rot) {
    constexpr int N = Vec<T>::N, LANES = D / N;
    const int lane = threadIdx.x & 31, in = lane % LANES, h = rot / 2;
    Geometry g;
    g.lane_row = lane / LANES;
    g.c0 = in * N;
    const int c = g.c0 < h ? g.c0 + h : g.c0 < rot ? g.c0 - h : g.c0;
    g.src = lane - in + c / N;
    g.rotated = g.c0 < rot;
    return g;
}
// The partner channels of x. Every lane of the warp takes part in the
// shuffles; lanes outside the rotated part get zeros (their B is zero, and zero
// times an infinity of their own would not be).
template <typename T> __device__ __forceinline__ Vec<T> partner(const Vec<T> &x, int layout, const Geometry &g) {
    Vec<T> p;
    if (layout == KDA_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p.raw[i] = __shfl_sync(0xffffffffu, x.raw[i], g.src);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p.raw[i] = __byte_perm(x.raw[i], 0u, 0x1032);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p.raw[i] = x.raw[i ^ 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) p.raw[i] = g.rotated ? p.raw[i] : 0u;
    return p;
}
// Weights of this lane's channels and of their partners.
template <int N>
__device__ __forceinline__ void load_weights(const float *w, int layout, int rot, const Geometry &g, float (&own)[N],
                                             float (&other)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) own[e] = other[e] = 1.f;
    if (!w) return;
    load_floats<N>(w + g.c0, own);
    if (layout == KDA_ROPE_HALF) {
        const int h = rot / 2;
        load_floats<N>(w + (g.c0 < h ? g.c0 + h : g.rotated ? g.c0 - h : g.c0), other);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) other[e] = own[e ^ 1];
    }
}

// A warp's unit: kPasses * ROWS consecutive rows (heads) of one token, taken
// from q's heads or from k's (never both, so that a weight is one register set).
template <typename T, int D> constexpr int unit_rows() { return kPasses * (32 / (D / Vec<T>::N)); }
struct Parts {
    int q, k;              // units of a token
    FastDiv by_all, by_q, by_k;
    int64_t tokens;
};

template <typename T, int D, bool AXES>
__global__ void __launch_bounds__(kThreads)
kda_qk_norm_rope_kernel(NormRopeArgs p, Parts parts, int units) {
    constexpr int N = Vec<T>::N, LANES = D / N, ROWS = 32 / LANES;
    const int64_t u64 = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (u64 >= units) return;
    const int u = (int)u64, tok = parts.by_all.div(u), part = u - tok * (parts.q + parts.k);
    const Geometry g = geometry<T, D>(p.rot);
    const bool is_q = part < parts.q;
    const int64_t token = tok;
    const int first = (is_q ? part : part - parts.q) * unit_rows<T, D>(), heads = is_q ? p.hq : p.hk;
    const T *x = is_q ? (const T *)p.q + token * p.q_stride : (const T *)p.k + token * p.k_stride;
    T *y = is_q ? (T *)p.yq + token * (int64_t)p.hq * D : (T *)p.yk + token * (int64_t)p.hk * D;
    const int pos = AXES ? axis_position(p, token) : p.rot > 0 ? __ldg(p.positions + token) : 0;
    Vec<T> v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int row = first + i * ROWS + g.lane_row;
        v[i].zero();
        if (row < heads) v[i].load(x + (int64_t)row * D + g.c0);
    }
    F2 A[N / 2], B[N / 2];
    {
        float wo[N], wp[N], cs[N], sn[N];
        load_weights<N>(is_q ? p.wq : p.wk, p.layout, p.rot, g, wo, wp);
        if constexpr (AXES) {
            if (!all_in_table(p, pos)) {
                if ((threadIdx.x & 31) == 0 && p.status) atomicOr(p.status, KDA_DEV_BAD_POSITION);
                return;
            }
            load_axis_angles<N>(p, AxisPositions(pos), g.c0, cs, sn);
        } else if (p.rot > 0) {
            if (pos < 0 || pos >= p.max_position) {  // uniform over the warp: the token's rows are left as they are
                if ((threadIdx.x & 31) == 0 && p.status) atomicOr(p.status, KDA_DEV_BAD_POSITION);
                return;
            }
            load_angles<N>(p.table + (int64_t)pos * p.rot, g.c0, p.rot, p.layout, cs, sn);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) cs[e] = 1.f, sn[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            A[e / 2] = f2(cs[e] * wo[e], cs[e + 1] * wo[e + 1]);
            B[e / 2] = f2(sn[e] * wp[e], sn[e + 1] * wp[e + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        if (first + i * ROWS >= heads) break;  // uniform
        const int row = first + i * ROWS + g.lane_row;
        const Vec<T> o = partner(v[i], p.layout, g);
        F2 ss = f2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) ss = fma2(v[i].get(e), v[i].get(e), ss);
        const float r = rnorm(row_sum<LANES>(f2_sum(ss)), p.norm, 1.f / D, p.eps);
        const F2 r2 = f2(r, r);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) v[i].put(e, fma2(A[e], v[i].get(e), B[e] * o.get(e)) * r2);
        if (row < heads) v[i].store(y + (int64_t)row * D + g.c0);
    }
}

// Backward. Persistent: each warp walks the units with a fixed stride and
// keeps its share of the weight gradients in registers; the block's shares
// are added in warp order and written to `partial` [blocks][2][D], which
// kda_column_sum_kernel adds in block order: the same bits on every call.
// x, dy and the token's table row come by cp.async into a ring of the warp's
// own, kStages units deep: 13 KB in flight per warp at no cost in registers
// (held in registers instead, two blocks of eight warps fit on an SM with 4 KB
// each, and 16384 x 32 rows of 128 bf16 channels took 110 us).
constexpr int kStages = 3;
constexpr int kUnitBytes = 2 * kPasses * 512 + 512;  // x, dy, table row
constexpr int kBwdSmem = kWarps * kStages * kUnitBytes;

template <typename T, int D, bool AXES>
__global__ void __launch_bounds__(kThreads, 2)
kda_qk_norm_rope_bwd_kernel(NormRopeArgs p, Parts parts) {
    constexpr int N = Vec<T>::N, LANES = D / N, ROWS = 32 / LANES;
    extern __shared__ __align__(16) unsigned char smem[];
    const Geometry g = geometry<T, D>(p.rot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned char *ring = smem + warp * kStages * kUnitBytes;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const int64_t step = (int64_t)gridDim.x * kWarps;
    float sums[2][N];
#pragma unroll
    for (int side = 0; side < 2; ++side) {  // all rows of q, then all rows of k
        const bool is_q = side == 0;
        const int per = is_q ? parts.q : parts.k, heads = is_q ? p.hq : p.hk;
        const FastDiv by = is_q ? parts.by_q : parts.by_k;
        const int64_t units = parts.tokens * per, x_stride = is_q ? p.q_stride : p.k_stride;
        const T *xb = (const T *)(is_q ? p.q : p.k), *dyb = (const T *)(is_q ? p.dyq : p.dyk);
        T *dxb = (T *)(is_q ? p.dxq : p.dxk);
        float wo[N], wp[N];
        F2 acc[N / 2], wv[N / 2];
        load_weights<N>(is_q ? p.wq : p.wk, p.layout, p.rot, g, wo, wp);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) acc[e] = f2(0.f, 0.f), wv[e] = f2(wo[2 * e], wo[2 * e + 1]);
        // AXES: lane a's is axis a's, and so is what it says of the table
        auto position = [&](int64_t u) {
            if constexpr (AXES) return u < units ? axis_position(p, by.div((int)u)) : 0;
            return p.rot > 0 && u < units ? __ldg(p.positions + by.div((int)u)) : 0;
        };
        auto in_table = [&](int pos) { return pos >= 0 && pos < p.max_position; };
        auto fetch = [&](int64_t u, int pos, int stage) {  // one group of copies, empty past the last unit
            if (u < units) {
                const int64_t token = by.div((int)u);
                const int first = (int)(u - token * per) * unit_rows<T, D>();
                const uint32_t dst = ring_s + stage * kUnitBytes + lane * 16;
                const T *x = xb + token * x_stride, *dy = dyb + token * (int64_t)heads * D;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int row = first + i * ROWS + g.lane_row;
                    const bool there = row < heads;
                    const int64_t at = there ? (int64_t)row * D + g.c0 : 0;
                    copy16(dst + i * 512, x + at, there);
                    copy16(dst + (kPasses + i) * 512, dy + at, there);
                }
                if constexpr (AXES) {  // the row is put together here
                    const bool good = all_in_table(p, pos);
                    const AxisPositions at(good ? pos : 0);
                    if (4 * lane < p.rot) {
                        const int pair = 4 * lane < p.rot / 2 ? 4 * lane : 4 * lane - p.rot / 2;
                        const uint32_t row = dst + 2 * kPasses * 512;
                        if (p.quads) {
                            copy16(row, p.table + (int64_t)at.of(pair_axis(p, pair)) * p.rot + 4 * lane, good);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                copy4(row + 4 * e,
                                      p.table + (int64_t)at.of(pair_axis(p, pair + e)) * p.rot + 4 * lane + e, good);
                        }
                    }
                } else if (4 * lane < p.rot)
                    copy16(dst + 2 * kPasses * 512, p.table + (in_table(pos) ? (int64_t)pos * p.rot + 4 * lane : 0),
                           in_table(pos));
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int64_t u = (int64_t)blockIdx.x * kWarps + warp;
        int pos[kStages];  // of the units in the ring; the next one's is loaded a unit ahead of its copies
#pragma unroll
        for (int i = 0; i < kStages; ++i) pos[i] = position(u + i * step);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(u + i * step, pos[i], i);
        int stage = 0;
        for (; u < units; u += step) {
            const int next = stage == 0 ? kStages - 1 : stage - 1;  // the stage read last
            __syncwarp();  // by every lane
            fetch(u + (kStages - 1) * step, pos[kStages - 1], next);
            const int ahead = position(u + kStages * step);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const unsigned char *buf = ring + stage * kUnitBytes;
            const bool good = AXES ? all_in_table(p, pos[0]) : p.rot == 0 || in_table(pos[0]);
#pragma unroll
            for (int i = 0; i + 1 < kStages; ++i) pos[i] = pos[i + 1];
            pos[kStages - 1] = ahead;
            stage = stage == kStages - 1 ? 0 : stage + 1;
            if (!good) {  // the token is left out
                if (lane == 0 && p.status) atomicOr(p.status, KDA_DEV_BAD_POSITION);
                continue;
            }
            const int64_t token = by.div((int)u);
            const int first = (int)(u - token * per) * unit_rows<T, D>();
            T *dx = dxb + token * (int64_t)heads * D;
            F2 cs[N / 2], sn[N / 2];  // turning back: the sines change sign
            {
                float c[N], t[N];
#pragma unroll
                for (int e = 0; e < N; ++e) c[e] = 1.f, t[e] = 0.f;
                if (p.rot > 0)
                    load_angles<N>(reinterpret_cast<const float *>(buf + 2 * kPasses * 512), g.c0, p.rot, p.layout, c, t);
#pragma unroll
                for (int e = 0; e < N / 2; ++e) cs[e] = f2(c[2 * e], c[2 * e + 1]), sn[e] = f2(-t[2 * e], -t[2 * e + 1]);
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                if (first + i * ROWS >= heads) break;
                const int row = first + i * ROWS + g.lane_row;
                Vec<T> vx, vd;
                vx.load(reinterpret_cast<const T *>(buf + i * 512 + lane * 16));
                vd.load(reinterpret_cast<const T *>(buf + (kPasses + i) * 512 + lane * 16));
                Vec<T> o;
                if (p.layout == KDA_ROPE_HALF) {  // another lane's piece
                    o.load(reinterpret_cast<const T *>(buf + (kPasses + i) * 512 + g.src * 16));
                    if (p.rot < D && !g.rotated) o.zero();
                } else {
                    o = partner(vd, p.layout, g);
                }
                F2 d[N / 2], dn[N / 2], ss = f2(0.f, 0.f), xd = ss;
#pragma unroll
                for (int e = 0; e < N / 2; ++e) {
                    d[e] = fma2(cs[e], vd.get(e), sn[e] * o.get(e));
                    dn[e] = d[e] * wv[e];
                    const F2 xe = vx.get(e);
                    ss = fma2(xe, xe, ss);
                    xd = fma2(xe, dn[e], xd);
                }
                float xx = f2_sum(ss), xdn = f2_sum(xd);
                row_sums<LANES>(xx, xdn);
                const float r = rnorm(xx, p.norm, 1.f / D, p.eps);
                // n . dn c: r meets x before it meets itself, since r^3 has a third of fp32's range (a zero row
                // under eps = 1e-30, a row of 1e13)
                const float c = p.norm == KDA_NORM_NONE
                                    ? 0.f
                                    : xdn * r * (p.norm == KDA_NORM_RMS ? 1.f / D : 1.f);
                const F2 r2 = f2(r, r), c2 = f2(-c, -c);
#pragma unroll
                for (int e = 0; e < N / 2; ++e) {
                    const F2 n = vx.get(e) * r2;
                    acc[e] = fma2(n, d[e], acc[e]);
                    vd.put(e, fma2(n, c2, dn[e]) * r2);
                }
                if (row < heads) vd.store(dx + (int64_t)row * D + g.c0);
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        // rows of the warp first (lanes LANES apart hold the same channels)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float a, b;
            f2_get(acc[e / 2], a, b);
            if (e & 1) a = b;
#pragma unroll
            for (int off = 16; off >= LANES; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
            sums[side][e] = a;
        }
    }
    if (!p.partial) return;
    float *red = reinterpret_cast<float *>(ring);  // [2][D] in each warp's own ring
    if (g.lane_row == 0) {
#pragma unroll
        for (int e = 0; e < 2 * N; ++e) red[(e / N) * D + g.c0 + e % N] = sums[e / N][e % N];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) a += reinterpret_cast<const float *>(smem + k * kStages * kUnitBytes)[i];
        p.partial[(int64_t)blockIdx.x * 2 * D + i] = a;
    }
}

template <typename T, int D, bool AXES> cudaError_t launch(const NormRopeArgs &p, bool back, cudaStream_t s) {
    constexpr int R = unit_rows<T, D>();
    Parts parts;
    parts.q = (p.hq + R - 1) / R;
    parts.k = (p.hk + R - 1) / R;
    parts.by_all = FastDiv(parts.q + parts.k);
    parts.by_q = FastDiv(parts.q > 0 ? parts.q : 1);
    parts.by_k = FastDiv(parts.k > 0 ? parts.k : 1);
    parts.tokens = p.tokens;
    const int64_t units = p.tokens * (parts.q + parts.k), blocks = (units + kWarps - 1) / kWarps;
    if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (!back) {
        kda_qk_norm_rope_kernel<T, D, AXES><<<(unsigned)blocks, kThreads, 0, s>>>(p, parts, (int)units);
        return cudaGetLastError();
    }
    const int grid = (int)(blocks < kNormRopeBwdBlocks ? blocks : kNormRopeBwdBlocks);
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kda_qk_norm_rope_bwd_kernel<T, D, AXES>, kBwdSmem, allowed);
    if (e != cudaSuccess) return e;
    Launches l{s};
    e = l.next(kda_qk_norm_rope_bwd_kernel<T, D, AXES>, grid, kThreads, kBwdSmem, p, parts);
    if (e != cudaSuccess || !p.partial) return e;
    return column_sum(l, p.partial, grid, D, 2, p.dwq, p.dwk);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &p, bool back, cudaStream_t s) {
    auto of = [&](auto axes) {
        constexpr bool AXES = decltype(axes)::value;
        if (p.dt == KDA_BF16)
            return p.d == 128 ? launch<__nv_bfloat16, 128, AXES>(p, back, s) : launch<__nv_bfloat16, 64, AXES>(p, back, s);
        return p.d == 128 ? launch<float, 128, AXES>(p, back, s) : launch<float, 64, AXES>(p, back, s);
    };
    return p.axes > 0 ? of(std::true_type{}) : of(std::false_type{});
}

}  // namespace kda
