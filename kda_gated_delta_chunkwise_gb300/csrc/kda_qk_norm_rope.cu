// Norm of every query and key head and the rotary positions, one pass each way.
//
//   n = x r,  r = 1 / sqrt(sum x^2 + eps)      (KDA_NORM_L2)
//             r = 1 / sqrt(sum x^2 / d + eps)  (KDA_NORM_RMS), r = 1 (NONE)
//   y = R(position) (w * n)
// with R turning channel pairs of the first `rot` channels by the angles whose
// cosines and sines the token's table row holds. Backward, for u = R^T dy:
//   dw = sum over rows of u n,   dn = w u,
//   dx = r dn - x r^3 (x . dn) c,   c = 1 (L2), 1 / d (RMS), 0 (NONE).
//
// Bound by memory: forward one read and one write of q and k, backward two
// reads and one write. A row (one head of one token) is held by 16 bytes in
// each of d * sizeof(T) / 16 lanes, so a warp reads 512 contiguous bytes at a
// time; every warp takes one token's rows four passes at once (2 KB in flight
// per warp) and keeps that token's cosines and sines in registers. The
// partner channel of the half layout comes from another lane by a shuffle.
// Sums, norms and the rotation are in fp32; the only rounding to fewer bits
// is the store.
#include "kda_internal.cuh"
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPasses = 4;  // row groups of a warp in flight at once

template <typename T> struct Vec {  // 16 bytes of a row
    static constexpr int N = 16 / sizeof(T);
    uint4 raw;
    __device__ __forceinline__ void load(const T *p) { raw = __ldg(reinterpret_cast<const uint4 *>(p)); }
    // plain loads, for what the same kernel may write
    __device__ __forceinline__ void load_rw(const T *p) { raw = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&x)[N]) const {
        const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = to_f32(e[i]);
    }
    __device__ __forceinline__ void put(const float (&x)[N]) {
        T *e = reinterpret_cast<T *>(&raw);
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from_f32<T>(x[i]);
    }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
};

template <int LANES> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <int N> __device__ __forceinline__ void load_floats(const float *p, float *x) {  // 4 N-byte aligned
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p + e));
            x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
        }
    } else {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
        x[0] = v.x, x[1] = v.y;
    }
}
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

// y = cos * x + sin * partner (sgn = -1 turns back). Every lane of the warp
// takes part in the shuffles; `src` is the lane of the partner channels. Lanes
// outside the rotated channels keep theirs (no 0 * infinity).
template <int N>
__device__ __forceinline__ void turn(float (&x)[N], const float (&cs)[N], const float (&sn)[N], float sgn, int layout,
                                     const Geometry &g) {
    if (layout == KDA_ROPE_HALF) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float o = __shfl_sync(0xffffffffu, x[e], g.src);
            if (g.rotated) x[e] = cs[e] * x[e] + sgn * sn[e] * o;
        }
    } else if (g.rotated) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float a = x[e], b = x[e + 1];
            x[e] = cs[e] * a + sgn * sn[e] * b;
            x[e + 1] = cs[e + 1] * b + sgn * sn[e + 1] * a;
        }
    }
}

__device__ __forceinline__ float rnorm(float ss, int norm, float inv_d, float eps) {
    // 1 / sqrtf, both correctly rounded, instead of the approximate reciprocal root
    return norm == KDA_NORM_NONE ? 1.f : 1.f / sqrtf((norm == KDA_NORM_RMS ? ss * inv_d : ss) + eps);
}

// A warp's unit: kPasses * ROWS consecutive rows (heads) of one token, taken
// from q's heads or from k's (never both, so that a weight is one register set).
template <typename T, int D> constexpr int unit_rows() { return kPasses * (32 / (D / Vec<T>::N)); }
struct Parts {
    int q, k;              // units of a token
    FastDiv by_all, by_q, by_k;
    int64_t tokens;
};

template <typename T, int D>
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
    const float *w = is_q ? p.wq : p.wk;
    Vec<T> v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int row = first + i * ROWS + g.lane_row;
        v[i].raw = make_uint4(0u, 0u, 0u, 0u);
        if (row < heads) v[i].load_rw(x + (int64_t)row * D + g.c0);  // y may be x: no read-only path
    }
    float cs[N], sn[N];
    if (p.rot > 0) {
        const int pos = __ldg(p.positions + token);
        if (pos < 0 || pos >= p.max_position) {  // uniform over the warp: the token's rows are left as they are
            if ((threadIdx.x & 31) == 0 && p.status) atomicOr(p.status, KDA_DEV_BAD_POSITION);
            return;
        }
        load_angles<N>(p.table + (int64_t)pos * p.rot, g.c0, p.rot, p.layout, cs, sn);
    }
    float wv[N];
    if (w) {
        load_floats<N>(w + g.c0, wv);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) wv[e] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        if (first + i * ROWS >= heads) break;  // uniform
        const int row = first + i * ROWS + g.lane_row;
        float f[N], ss = 0.f;
        v[i].get(f);
#pragma unroll
        for (int e = 0; e < N; ++e) ss += f[e] * f[e];
        const float r = rnorm(row_sum<LANES>(ss), p.norm, 1.f / D, p.eps);
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = f[e] * r * wv[e];
        if (p.rot > 0) turn<N>(f, cs, sn, 1.f, p.layout, g);
        v[i].put(f);
        if (row < heads) v[i].store(y + (int64_t)row * D + g.c0);
    }
}

// Backward. Persistent: each warp walks the units with a fixed stride and
// keeps its share of the weight gradients in registers; the block's shares
// are added in warp order and written to `partial` [blocks][2][D], which
// kda_weight_sum_kernel adds in block order: the same bits on every call.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
kda_qk_norm_rope_bwd_kernel(NormRopeArgs p, Parts parts) {
    constexpr int N = Vec<T>::N, LANES = D / N, ROWS = 32 / LANES;
    __shared__ float red[kWarps][2][D];
    const Geometry g = geometry<T, D>(p.rot);
    const int warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {  // all rows of q, then all rows of k
        const bool is_q = side == 0;
        const int per = is_q ? parts.q : parts.k, heads = is_q ? p.hq : p.hk;
        const FastDiv by = is_q ? parts.by_q : parts.by_k;
        const int units = (int)(parts.tokens * per);
        const float *w = is_q ? p.wq : p.wk;
        float wv[N], acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) wv[e] = 1.f, acc[e] = 0.f;
        if (w) load_floats<N>(w + g.c0, wv);
        for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < units; u += (int64_t)gridDim.x * kWarps) {
            const int64_t token = by.div((int)u);
            const int first = (int)(u - token * per) * unit_rows<T, D>();
            const T *x = (is_q ? (const T *)p.q + token * p.q_stride : (const T *)p.k + token * p.k_stride);
            const int64_t at = token * (int64_t)heads * D;
            const T *dy = (is_q ? (const T *)p.dyq : (const T *)p.dyk) + at;
            T *dx = (is_q ? (T *)p.dxq : (T *)p.dxk) + at;
            Vec<T> vx[kPasses], vd[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int row = first + i * ROWS + g.lane_row;
                vx[i].raw = vd[i].raw = make_uint4(0u, 0u, 0u, 0u);
                if (row < heads) {
                    vx[i].load(x + (int64_t)row * D + g.c0);
                    vd[i].load(dy + (int64_t)row * D + g.c0);
                }
            }
            float cs[N], sn[N];
            if (p.rot > 0) {
                const int pos = __ldg(p.positions + token);
                if (pos < 0 || pos >= p.max_position) {
                    if ((threadIdx.x & 31) == 0 && p.status) atomicOr(p.status, KDA_DEV_BAD_POSITION);
                    continue;
                }
                load_angles<N>(p.table + (int64_t)pos * p.rot, g.c0, p.rot, p.layout, cs, sn);
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                if (first + i * ROWS >= heads) break;
                const int row = first + i * ROWS + g.lane_row;
                float f[N], d[N], ss = 0.f, xd = 0.f;
                vx[i].get(f);
                vd[i].get(d);
                if (p.rot > 0) turn<N>(d, cs, sn, -1.f, p.layout, g);
#pragma unroll
                for (int e = 0; e < N; ++e) ss += f[e] * f[e];
                const float r = rnorm(row_sum<LANES>(ss), p.norm, 1.f / D, p.eps);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    acc[e] += d[e] * (f[e] * r);
                    d[e] *= wv[e];
                    xd += f[e] * d[e];
                }
                const float c = p.norm == KDA_NORM_NONE ? 0.f
                                                        : row_sum<LANES>(xd) * (r * r * r) *
                                                              (p.norm == KDA_NORM_RMS ? 1.f / D : 1.f);
#pragma unroll
                for (int e = 0; e < N; ++e) d[e] = r * d[e] - f[e] * c;
                vd[i].put(d);
                if (row < heads) vd[i].store(dx + (int64_t)row * D + g.c0);
            }
        }
        // rows of the warp first (lanes LANES apart hold the same channels), then the warps
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float a = acc[e];
#pragma unroll
            for (int off = 16; off >= LANES; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
            if (g.lane_row == 0) red[warp][side][g.c0 + e] = a;
        }
    }
    if (!p.partial) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) a += red[k][i / D][i % D];
        p.partial[(int64_t)blockIdx.x * 2 * D + i] = a;
    }
}

// dw[s][c] = sum over blocks of partial[block][s][c], in a fixed order: one
// warp per output, lanes striding over the blocks, then a shuffle tree.
__global__ void __launch_bounds__(kThreads)
kda_weight_sum_kernel(const float *__restrict__ partial, int blocks, int d, float *dwq, float *dwk) {
    const int o = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (o >= 2 * d) return;
    float a = 0.f;
    for (int b = lane; b < blocks; b += 32) a += partial[(int64_t)b * 2 * d + o];
    a = row_sum<32>(a);
    float *dst = o < d ? dwq : dwk;
    if (lane == 0 && dst) dst[o % d] = a;
}

template <typename T, int D> cudaError_t launch(const NormRopeArgs &p, bool back, cudaStream_t s) {
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
        kda_qk_norm_rope_kernel<T, D><<<(unsigned)blocks, kThreads, 0, s>>>(p, parts, (int)units);
        return cudaGetLastError();
    }
    const int grid = (int)(blocks < kNormRopeBwdBlocks ? blocks : kNormRopeBwdBlocks);
    kda_qk_norm_rope_bwd_kernel<T, D><<<grid, kThreads, 0, s>>>(p, parts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.partial) return e;
    kda_weight_sum_kernel<<<(2 * D + kWarps - 1) / kWarps, kThreads, 0, s>>>(p.partial, grid, D, p.dwq, p.dwk);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &p, bool back, cudaStream_t s) {
    if (p.dt == KDA_BF16)
        return p.d == 128 ? launch<__nv_bfloat16, 128>(p, back, s) : launch<__nv_bfloat16, 64>(p, back, s);
    return p.d == 128 ? launch<float, 128>(p, back, s) : launch<float, 64>(p, back, s);
}

}  // namespace kda
