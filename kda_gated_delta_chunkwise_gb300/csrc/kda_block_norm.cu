// The norm of every head times a gate, and the residual stream with its norm.
//
// Gated: n = x r (r as in kda_qk_norm_rope.cu), a the gate's sigmoid, or g times it,
//   y = w n a;   back: u = a dy, dw = sum over rows of u n, dn = w u,
//   dx = r (dn - n (n . dn) c),  dg = w n a' dy,
//   a' = a (1 - a) (sigmoid), a (1 + g (1 - a)) (silu).
// Residual: u = b, or w_b b r_b; h = x + s c u, y = w h r. Back, for the
// gradient dh that reaches h by the stream:
//   g = dh + r (w dy - n (n . w dy) / D),  n = h r        -> the residual's
//   du = s c g,   db = du, or r_b (w_b du - m (m . w_b du) k),  m = b r_b
//   dw = sum n dy,  dw_b = sum m du,  dc = sum s u g.
// The sum m . w_b du wants g, and so r; with q = w_b s c b it is
//   sum q dh + r sum q w dy - r^2 ((n . w dy) / D) sum q h  times r_b,
// so that one round of sums over a row serves both norms.
//
// Bound by memory, each input read once and each output written once. Sums and
// everything in between are fp32; the only rounding to fewer bits is the store
// (y is made from the unrounded h). Sums over rows have a fixed order. 16384 rows of
// 16 x 128 bf16 channels, as calls one after the other: gated 34.5 us (5.8 TB/s), its
// gradients 65 (5.2); residual with a stream in fp32 66 (6.1), its gradients 101 (6.0).
#include <cfloat>
#include <type_traits>

#include "kda_block_norm.cuh"
#include "kda_rows.cuh"
#include "kda_tc_roles.cuh"

namespace kda {
namespace {

// ================================================================ heads times a gate
constexpr int GT = 256, GW = GT / 32;
constexpr int kPasses = 4;  // row groups of a warp in flight at once (forward)

// e^-g. fp32 gates take the accurate exponential; to a bf16 result the 2^-22 of
// the approximate one is nothing.
template <typename T> __device__ __forceinline__ float exp_neg(float g) {
    return sizeof(T) == 2 ? exp2_approx(g * -1.4426950408889634f) : expf(-g);
}
template <typename T> __device__ __forceinline__ float recip(float x) {
    if constexpr (sizeof(T) == 2) {
        float y;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
        return y;
    } else {
        return 1.f / x;
    }
}
// The gate's value and its derivative; 1 - sigmoid as e / (1 + e), which keeps its
// digits, and is one where e is large, infinite even: there the sigmoid is e^g down
// to nothing. A gate of -inf or the type's lowest value is closed, in silu too, where
// g is kept finite for that.
template <typename T> __device__ __forceinline__ void gate_of(float g, int act, float &a, float &da) {
    const float e = exp_neg<T>(g), s = recip<T>(1.f + e), c = e > 1e30f ? 1.f : e * s;
    const float f = fmaxf(g, -FLT_MAX);
    a = act == KDA_ACT_SILU ? f * s : s;
    da = act == KDA_ACT_SILU ? s * fmaf(f, c, 1.f) : s * c;
}

// A row (one head of one token) is held by 16 bytes in each of d sizeof(T) / 16
// lanes, as in kda_qk_norm_rope.cu; rows are taken in the order of memory.
template <typename T, int D>
__global__ void __launch_bounds__(GT)
kda_gated_norm_kernel(GatedArgs p, int rows) {
    constexpr int N = Vec<T>::N, LANES = D / N, ROWS = 32 / LANES;
    const int lane = threadIdx.x & 31, c0 = (lane % LANES) * N;
    const int64_t first = ((int64_t)blockIdx.x * GW + (threadIdx.x >> 5)) * (kPasses * ROWS) + lane / LANES;
    Vec<T> x[kPasses], g[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t row = first + i * ROWS;
        x[i].zero(), g[i].zero();
        if (row < rows) {
            const int token = p.by_heads.div((int)row), head = (int)row - token * p.h;
            x[i].load((const T *)p.x + token * p.x_stride + head * D + c0);
            g[i].load((const T *)p.gate + token * p.g_stride + head * D + c0);
        }
    }
    float w[N];
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 1.f;
    if (p.w) load_floats<N>(p.w + c0, w);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t row = first + i * ROWS;
        F2 ss = f2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) ss = fma2(x[i].get(e), x[i].get(e), ss);
        const float r = rnorm(row_sum<LANES>(f2_sum(ss)), p.norm, 1.f / D, p.eps);
        const F2 r2 = f2(r, r);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            float g0, g1, a0, a1, unused;
            f2_get(g[i].get(e), g0, g1);
            gate_of<T>(g0, p.act, a0, unused);
            gate_of<T>(g1, p.act, a1, unused);
            x[i].put(e, x[i].get(e) * r2 * f2(w[2 * e], w[2 * e + 1]) * f2(a0, a1));
        }
        if (row < rows) x[i].store((T *)p.y + row * D + c0);
    }
}

// Persistent; x, gate and dy come by cp.async into a ring of the warp's own. Each
// warp keeps its share of the weight's gradient in registers, the block's are
// added in warp order into `partial` [blocks][D].
constexpr int GB_PASSES = 2, GB_STAGES = 4;
constexpr int GB_UNIT = 3 * GB_PASSES * 512;
constexpr int GB_SMEM = GW * GB_STAGES * GB_UNIT;

template <typename T, int D>
__global__ void __launch_bounds__(GT, 2)
kda_gated_norm_bwd_kernel(GatedArgs p, int rows) {
    constexpr int N = Vec<T>::N, LANES = D / N, ROWS = 32 / LANES, PER = GB_PASSES * ROWS;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = (lane % LANES) * N, sub = lane / LANES;
    unsigned char *ring = smem + warp * GB_STAGES * GB_UNIT;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring) + lane * 16;
    const int units = (rows + PER - 1) / PER, step = gridDim.x * GW;
    float w[N];
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 1.f;
    if (p.w) load_floats<N>(p.w + c0, w);
    F2 acc[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) acc[e] = f2(0.f, 0.f);
    auto fetch = [&](int64_t u, int stage) {  // one group of copies, empty past the last unit
        if (u < units) {
#pragma unroll
            for (int i = 0; i < GB_PASSES; ++i) {
                const int64_t row = u * PER + i * ROWS + sub;
                const bool there = row < rows;
                const int at = there ? (int)row : 0, token = p.by_heads.div(at), in = (at - token * p.h) * D + c0;
                const uint32_t dst = ring_s + stage * GB_UNIT + i * 512;
                copy16(dst, (const T *)p.x + token * p.x_stride + in, there);
                copy16(dst + GB_PASSES * 512, (const T *)p.gate + token * p.g_stride + in, there);
                copy16(dst + 2 * GB_PASSES * 512, (const T *)p.dy + (int64_t)at * D + c0, there);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int64_t u = (int64_t)blockIdx.x * GW + warp;
#pragma unroll
    for (int i = 0; i < GB_STAGES - 1; ++i) fetch(u + (int64_t)i * step, i);
    int stage = 0;
    for (; u < units; u += step) {
        // every lane reads what it copied itself, so its own wait is enough
        fetch(u + (int64_t)(GB_STAGES - 1) * step, (stage + GB_STAGES - 1) % GB_STAGES);
        asm volatile("cp.async.wait_group %0;" ::"n"(GB_STAGES - 1) : "memory");
        const unsigned char *buf = ring + stage * GB_UNIT + lane * 16;
        stage = (stage + 1) % GB_STAGES;
#pragma unroll
        for (int i = 0; i < GB_PASSES; ++i) {
            const int64_t row = u * PER + i * ROWS + sub;
            Vec<T> x, g, dy;
            x.load(reinterpret_cast<const T *>(buf + i * 512));
            g.load(reinterpret_cast<const T *>(buf + (GB_PASSES + i) * 512));
            dy.load(reinterpret_cast<const T *>(buf + (2 * GB_PASSES + i) * 512));
            F2 ud[N / 2], dg[N / 2], ss = f2(0.f, 0.f), xd = ss;  // a dy, w a' dy
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                float g0, g1, a0, a1, d0, d1;
                f2_get(g.get(e), g0, g1);
                gate_of<T>(g0, p.act, a0, d0);
                gate_of<T>(g1, p.act, a1, d1);
                const F2 wv = f2(w[2 * e], w[2 * e + 1]), xe = x.get(e);
                ud[e] = f2(a0, a1) * dy.get(e);
                dg[e] = f2(d0, d1) * dy.get(e) * wv;
                ss = fma2(xe, xe, ss);
                xd = fma2(xe, ud[e] * wv, xd);
            }
            float xx = f2_sum(ss), xdn = f2_sum(xd);
            row_sums<LANES>(xx, xdn);
            const float r = rnorm(xx, p.norm, 1.f / D, p.eps);
            const float c = p.norm == KDA_NORM_NONE ? 0.f : xdn * r * (p.norm == KDA_NORM_RMS ? 1.f / D : 1.f);
            const F2 r2 = f2(r, r), c2 = f2(-c, -c);
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const F2 n = x.get(e) * r2;
                acc[e] = fma2(n, ud[e], acc[e]);
                x.put(e, fma2(n, c2, ud[e] * f2(w[2 * e], w[2 * e + 1])) * r2);
                g.put(e, n * dg[e]);
            }
            if (row < rows) {
                x.store((T *)p.dx + row * D + c0);
                g.store((T *)p.dgate + row * D + c0);
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!p.partial) return;
    __syncwarp();
    float *red = reinterpret_cast<float *>(ring);  // [D] in each warp's own ring
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float a, b;
        f2_get(acc[e / 2], a, b);
        if (e & 1) a = b;
#pragma unroll
        for (int off = 16; off >= LANES; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
        if (sub == 0) red[c0 + e] = a;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += GT) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < GW; ++k) a += reinterpret_cast<const float *>(smem + k * GB_STAGES * GB_UNIT)[i];
        p.partial[(int64_t)blockIdx.x * D + i] = a;
    }
}

// ================================================================ the residual stream
// A row is held by `tr` threads, a power of two from a warp up to 512, eight
// channels V times in each (tr the least that does with V <= 2 forward, V = 1
// backward up to 4096 channels).
template <typename T> struct Eight {  // eight channels
    static constexpr int CHUNKS = 8 * sizeof(T) / 16;
    Vec<T> v[CHUNKS];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) v[i].zero();
    }
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) v[i].load(p + i * Vec<T>::N);
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (CHUNKS == 2) {
            const uint32_t r[8] = {v[0].raw[0], v[0].raw[1], v[0].raw[2], v[0].raw[3],
                                   v[1].raw[0], v[1].raw[1], v[1].raw[2], v[1].raw[3]};
            st_v8(p, r);
        } else {
            v[0].store(p);
        }
    }
    __device__ __forceinline__ F2 get(int i) const { return v[i / (Vec<T>::N / 2)].get(i % (Vec<T>::N / 2)); }
    __device__ __forceinline__ void put(int i, F2 x) { v[i / (Vec<T>::N / 2)].put(i % (Vec<T>::N / 2), x); }
};
__device__ __forceinline__ void load_eight(const float *p, int c, F2 (&x)[4]) {  // ones without a pointer
    if (p) {
        float v[8];
        load_floats<8>(p + c, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2(1.f, 1.f);
    }
}

// The sum of a value over a row's tr threads, the same in all of them. `scratch`
// [warps of the block]; calls in turn take one and the other half of it, so one
// barrier a call is enough.
__device__ __forceinline__ void row_barrier(int tr, int group) {
    if (tr == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tr) : "memory");
}
__device__ __forceinline__ float row_total(float v, int tr, float *scratch, int group) {
    v = row_sum<32>(v);
    if (tr == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = tr >> 5;
    if (lane == 0) scratch[warp] = v;
    row_barrier(tr, group);
    return row_sum<32>(lane < warps ? scratch[group * warps + lane] : 0.f);
}
// The same of six values at once, in two halves. In a warp the lanes share the values
// out as they add them up, nine shuffles in all instead of thirty, and leave them at
// scratch [16 warps][8]; after a barrier of the row each warp adds up the row's.
__device__ __forceinline__ void warp_totals(float (&v)[8], float *scratch) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int bit = 16, n = 4; n > 0; bit >>= 1, n >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
        }
    }
    float x = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);  // of value lane / 4
    if ((lane & 3) == 0) scratch[(threadIdx.x >> 5) * 8 + (lane >> 2)] = x;
}
__device__ __forceinline__ void read_totals(float (&v)[6], int tr, const float *scratch, int group) {
    const int lane = threadIdx.x & 31, warps = tr >> 5;
    const float *mine = scratch + group * warps * 8 + (lane & 3) * 8 + (lane >> 2);  // four lanes a value
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < 16; w += 4) {
        if (w + (lane & 3) < warps) x += mine[w * 8];
    }
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
#pragma unroll
    for (int k = 0; k < 6; ++k) v[k] = __shfl_sync(0xffffffffu, x, 4 * k);
}

template <typename S, typename T, int V>
__global__ void __launch_bounds__(512)
kda_residual_norm_kernel(ResidualArgs p, int tr) {
    __shared__ float scratch[2][16];
    const int group = threadIdx.x / tr, in = threadIdx.x % tr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tr) + group;
    if (row >= p.tokens) return;  // uniform over the row's threads
    Eight<S> x[V];
    Eight<T> b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (in + v * tr) * 8;
        x[v].zero(), b[v].zero();
        if (c < p.D) {
            x[v].load((const S *)p.x + row * p.D + c);
            b[v].load((const T *)p.b + row * p.D + c);
        }
    }
    const float inv_d = 1.f / (float)p.D;
    float rb = 1.f;
    if (p.branch_norm != KDA_NORM_NONE) {
        F2 ss = f2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fma2(b[v].get(i), b[v].get(i), ss);
        }
        rb = rnorm(row_total(f2_sum(ss), tr, scratch[0], group), p.branch_norm, inv_d, p.eps);
    }
    F2 h[V][4], ss = f2(0.f, 0.f);
    const F2 s2 = f2(p.scale * rb, p.scale * rb);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (in + v * tr) * 8;
        const bool there = c < p.D;
        F2 wb[4], ch[4];
        load_eight(there ? p.wb : nullptr, c, wb);
        load_eight(there ? p.c : nullptr, c, ch);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[v][i] = fma2(b[v].get(i), s2 * wb[i] * ch[i], x[v].get(i));
            ss = fma2(h[v][i], h[v][i], ss);
            x[v].put(i, h[v][i]);
        }
        if (there) x[v].store((S *)p.h + row * p.D + c);
    }
    const float r = rnorm(row_total(f2_sum(ss), tr, scratch[1], group), KDA_NORM_RMS, inv_d, p.eps);
    const F2 r2 = f2(r, r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (in + v * tr) * 8;
        if (c >= p.D) continue;
        F2 w[4];
        load_eight(p.w, c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[v].put(i, h[v][i] * r2 * w[i]);
        b[v].store((T *)p.y + row * p.D + c);
    }
}

// Persistent: the threads of a row walk the rows with a fixed stride and keep the
// sums over them in registers. A row's inputs come as bulk copies into a ring of
// its threads (copied by the threads themselves, 16 bytes at a time, 16384 rows of
// 2048 with a stream in fp32 took 137 us instead of 101); while a row's gradients are
// made, the sums of the next one are added up, and one barrier a row serves its
// totals and the ring. A row that fills
// the ring by itself stays in registers, and the next one comes meanwhile.
constexpr int RT = 512;
template <typename S, typename T, int V> struct ResidualRing {
    static constexpr int STAGE = RT * V * 8 * 2 * (sizeof(S) + sizeof(T));  // of the block's rows
    static constexpr int FIT = 200 * 1024 / STAGE, STAGES = FIT < 4 ? FIT : 4;
    static constexpr int BYTES = STAGES * STAGE;
};

template <typename S, typename T, int V>
__global__ void __launch_bounds__(RT, 1)
kda_residual_norm_bwd_kernel(ResidualArgs p, int tr) {
    using R = ResidualRing<S, T, V>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) float scratch[2][8 * 16];
    __shared__ uint64_t full[R::STAGES][RT / 32];
    __shared__ int abort_flag;
    const Abort stop{&abort_flag};
    const int group = threadIdx.x / tr, in = threadIdx.x % tr, groups = RT / tr;
    const bool branch = p.branch_norm != KDA_NORM_NONE || p.wb || p.c || p.dwb || p.dc;  // the branch is read
    const float inv_d = 1.f / (float)p.D;
    const int64_t step = (int64_t)gridDim.x * groups;
    if (in == 0) {
        for (int i = 0; i < R::STAGES; ++i) mbar_init(&full[i][group], 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    __syncthreads();
    F2 aw[V][4], ab[V][4], ac[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) aw[v][i] = ab[v][i] = ac[v][i] = f2(0.f, 0.f);
    }
    // the weights of this thread's channels: with eight channels kept, with sixteen read again for every row
    F2 w[4], wb[4], ch[4];
    auto weights = [&](int v) {
        const int c = (in + v * tr) * 8;
        const bool there = c < p.D;
        load_eight(there ? p.w : nullptr, c, w);
        load_eight(there ? p.wb : nullptr, c, wb);
        load_eight(there ? p.c : nullptr, c, ch);
    };
    if constexpr (V == 1) weights(0);
    // a stage holds a row's h, dh, dy, b one after the other
    unsigned char *ring = smem + group * (R::STAGE / groups);
    const uint32_t row_s = p.D * (uint32_t)sizeof(S), row_t = p.D * (uint32_t)sizeof(T);
    auto fetch = [&](int64_t row, int stage) {  // one thread
        if (row >= p.tokens) return;
        uint64_t *bar = &full[stage][group];
        unsigned char *to = ring + stage * R::STAGE;
        mbar_arrive_expect_tx(bar, row_s + (p.dh ? row_s : 0u) + row_t + (branch ? row_t : 0u));
        bulk_load(to, (const S *)p.x + row * p.D, row_s, bar);
        if (p.dh) bulk_load(to + row_s, (const S *)p.dh + row * p.D, row_s, bar);
        bulk_load(to + 2 * row_s, (const T *)p.dy + row * p.D, row_t, bar);
        if (branch) bulk_load(to + 2 * row_s + row_t, (const T *)p.b + row * p.D, row_t, bar);
    };
    Eight<S> h[V], dh[V];
    Eight<T> dy[V], b[V];
    auto load = [&](int stage, int v) {
        const int c = (in + v * tr) * 8;
        const unsigned char *from = ring + stage * R::STAGE;
        h[v].zero(), dh[v].zero(), dy[v].zero(), b[v].zero();
        if (c >= p.D) return;
        h[v].load((const S *)from + c);
        if (p.dh) dh[v].load((const S *)(from + row_s) + c);
        dy[v].load((const T *)(from + 2 * row_s) + c);
        if (branch) b[v].load((const T *)(from + 2 * row_s + row_t) + c);
    };
    // a row's sums: h h, h w dy, b b, and q dh, q w dy, q h with q = b w_b c
    auto sums = [&](int stage, float *at) {
        F2 a[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) a[k] = f2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            load(stage, v);
            if constexpr (V > 1) weights(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 hv = h[v].get(i), bv = b[v].get(i), wd = w[i] * dy[v].get(i), q = bv * wb[i] * ch[i];
                a[0] = fma2(hv, hv, a[0]);
                a[1] = fma2(hv, wd, a[1]);
                a[2] = fma2(bv, bv, a[2]);
                a[3] = fma2(q, dh[v].get(i), a[3]);
                a[4] = fma2(q, wd, a[4]);
                a[5] = fma2(q, hv, a[5]);
            }
        }
        float sum[8];
#pragma unroll
        for (int k = 0; k < 6; ++k) sum[k] = f2_sum(a[k]);
        sum[6] = sum[7] = 0.f;
        warp_totals(sum, at);
    };
    constexpr bool AHEAD = R::STAGES > 1;  // the sums of the next row are made with a row's gradients
    int64_t row = (int64_t)blockIdx.x * groups + group;
    if (in == 0) {
        for (int i = 0; i < (AHEAD ? R::STAGES - 1 : 1); ++i) fetch(row + i * step, i);
    }
    int stage = 0, half = 0;
    uint32_t parity = 0;  // of this row's stage
    if (AHEAD && row < p.tokens) {
        stop.wait_warp(smem_u32(&full[0][group]), 0);
        sums(0, scratch[0]);
    }
    for (; row < p.tokens; row += step, half ^= 1) {
        if constexpr (!AHEAD) {
            stop.wait_warp(smem_u32(&full[0][group]), parity);
            sums(0, scratch[half]);
        }
        row_barrier(tr, group);
        // all of the row's threads have read the row before it, or this one if there is one stage
        const int last = stage == 0 ? R::STAGES - 1 : stage - 1, next = stage == R::STAGES - 1 ? 0 : stage + 1;
        if (in == 0) fetch(row + (AHEAD ? R::STAGES - 1 : 1) * step, AHEAD ? last : 0);
        float sum[6];
        read_totals(sum, tr, scratch[half], group);
        if (AHEAD && row + step < p.tokens) {
            stop.wait_warp(smem_u32(&full[next][group]), parity ^ (next == 0));
            sums(next, scratch[half ^ 1]);
        }
        const float r = rnorm(sum[0], KDA_NORM_RMS, inv_d, p.eps), c = sum[1] * r * inv_d;
        const float rb = rnorm(sum[2], p.branch_norm, inv_d, p.eps);
        // (m . w_b du) k, without the scale
        const float e = p.branch_norm == KDA_NORM_NONE
                            ? 0.f
                            : rb * (p.branch_norm == KDA_NORM_RMS ? inv_d : 1.f) *
                                  (sum[3] + r * sum[4] - (r * c) * (r * sum[5]));
        const F2 r2 = f2(r, r), c2 = f2(-c, -c), rb2 = f2(rb, rb), e2 = f2(-e, -e),
                 srb2 = f2(p.scale * rb, p.scale * rb);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c0 = (in + v * tr) * 8;
            if constexpr (AHEAD) load(stage, v);
            if (c0 >= p.D) continue;
            if constexpr (V > 1) weights(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 n = h[v].get(i) * r2, dyv = dy[v].get(i);
                const F2 g = fma2(fma2(n, c2, w[i] * dyv), r2, dh[v].get(i));
                aw[v][i] = fma2(n, dyv, aw[v][i]);
                const F2 m = b[v].get(i) * rb2, du = ch[i] * g;  // without the scale
                ab[v][i] = fma2(m, du, ab[v][i]);
                ac[v][i] = fma2(wb[i] * m, g, ac[v][i]);
                h[v].put(i, g);
                dy[v].put(i, fma2(m, e2, wb[i] * du) * srb2);
            }
            h[v].store((S *)p.dx + row * p.D + c0);
            dy[v].store((T *)p.db + row * p.D + c0);
        }
        stage = next;
        parity ^= next == 0;
    }
    __syncthreads();
    settle(stop);
    if (!p.partial) return;
    // the groups' shares, one set of sums after the other: [groups][D] in shared memory
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (in + v * tr) * 8;
            if (c >= p.D) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a, b;
                f2_get(k == 0 ? aw[v][i] : k == 1 ? ab[v][i] : ac[v][i], a, b);
                const float f = k == 0 ? 1.f : p.scale;
                *reinterpret_cast<float2 *>(red + group * p.D + c + 2 * i) = make_float2(f * a, f * b);
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += RT) {
            float a = 0.f;
            for (int j = 0; j < groups; ++j) a += red[j * p.D + c];
            p.partial[((int64_t)blockIdx.x * 3 + k) * p.D + c] = a;
        }
    }
}

// ================================================================ launches
template <typename T, int D> cudaError_t launch_gated(const GatedArgs &p, bool back, cudaStream_t s) {
    constexpr int ROWS = 32 / (D / Vec<T>::N);
    const int rows = (int)(p.tokens * p.h);
    if (!back) {
        const int per = GW * kPasses * ROWS;
        kda_gated_norm_kernel<T, D><<<(rows - 1) / per + 1, GT, 0, s>>>(p, rows);
        return cudaGetLastError();
    }
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kda_gated_norm_bwd_kernel<T, D>, GB_SMEM, allowed);
    if (e != cudaSuccess) return e;
    const int per = GW * GB_PASSES * ROWS, blocks = (rows - 1) / per + 1;
    const int grid = blocks < kGatedBwdBlocks ? blocks : kGatedBwdBlocks;
    Launches l{s};
    e = l.next(kda_gated_norm_bwd_kernel<T, D>, grid, GT, GB_SMEM, p, rows);
    if (e != cudaSuccess || !p.partial) return e;
    return column_sum(l, p.partial, grid, D, 1, p.dw);
}

template <typename S, typename T> cudaError_t launch_residual(const ResidualArgs &p, bool back, cudaStream_t s) {
    const int eights = p.D / 8;
    int tr = 32;
    while (tr * (back ? 1 : 2) < eights && tr < 512) tr *= 2;
    const bool two = eights > tr;
    if (!back) {
        const int threads = tr < 256 ? 256 : tr, per = threads / tr;
        const int64_t blocks = (p.tokens + per - 1) / per;
        if (two) kda_residual_norm_kernel<S, T, 2><<<(unsigned)blocks, threads, 0, s>>>(p, tr);
        else kda_residual_norm_kernel<S, T, 1><<<(unsigned)blocks, threads, 0, s>>>(p, tr);
        return cudaGetLastError();
    }
    const int groups = RT / tr;
    const int64_t blocks = (p.tokens + groups - 1) / groups;
    const int grid = (int)(blocks < kResidualBwdBlocks ? blocks : kResidualBwdBlocks);
    Launches l{s};
    auto run = [&](auto v) {
        constexpr int V = decltype(v)::value;
        static std::atomic<uint64_t> allowed{0};
        constexpr int bytes = ResidualRing<S, T, V>::BYTES;
        static_assert(V * RT * 8 * 4 <= bytes, "the groups' sums fit in the ring");
        const cudaError_t e = allow_smem(kda_residual_norm_bwd_kernel<S, T, V>, bytes, allowed);
        return e != cudaSuccess ? e : l.next(kda_residual_norm_bwd_kernel<S, T, V>, grid, RT, bytes, p, tr);
    };
    const cudaError_t e = two ? run(std::integral_constant<int, 2>{}) : run(std::integral_constant<int, 1>{});
    if (e != cudaSuccess || !p.partial) return e;
    return column_sum(l, p.partial, grid, p.D, 3, p.dw, p.dwb, p.dc);
}

}  // namespace

cudaError_t launch_gated_norm(const GatedArgs &p, bool back, cudaStream_t s) {
    if (p.dt == KDA_BF16)
        return p.d == 128 ? launch_gated<__nv_bfloat16, 128>(p, back, s) : launch_gated<__nv_bfloat16, 64>(p, back, s);
    return p.d == 128 ? launch_gated<float, 128>(p, back, s) : launch_gated<float, 64>(p, back, s);
}

cudaError_t launch_residual_norm(const ResidualArgs &p, bool back, cudaStream_t s) {
    if (p.dt == KDA_F32) return launch_residual<float, float>(p, back, s);
    return p.stream_dt == KDA_F32 ? launch_residual<float, __nv_bfloat16>(p, back, s)
                                  : launch_residual<__nv_bfloat16, __nv_bfloat16>(p, back, s);
}

cudaError_t read_block_error(int *out, bool reset) { return read_tc_error(out, reset); }

}  // namespace kda
