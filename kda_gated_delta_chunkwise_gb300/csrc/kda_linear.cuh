// Declarations shared by the linear-attention operators, the query/key norm
// with rotary positions, and the host checks in front of them.
#pragma once

#include <atomic>

#include "kda_internal.cuh"

namespace kda {

// Two fp32 values, one instruction for both.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_get(F2 a, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float f2_sum(F2 a) {
    float x, y;
    f2_get(a, x, y);
    return x + y;
}

// n / d by a multiplication, for 0 <= n < 2^31: with l = ceil(log2 d) and
// m = floor(2^(31 + l) / d) + 1 <= 2^32, the error (m d - 2^(31 + l)) n / (d 2^(31 + l))
// stays below 1 / d. (The divisions of a work item's number sat in front of
// every item in the roles that run on one thread.)
struct FastDiv {
    uint32_t d, m, l;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div), l(0) {
        while ((1ull << l) < div) ++l;
        m = (uint32_t)((1ull << (31 + l)) / div + 1);  // div = 1: 2^31 + 1
    }
    __device__ __forceinline__ int div(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + l)); }
};

// ---------------------------------------------------------------- norm + rotation
// Blocks of the backward's persistent grid at most: two of 256 threads on each
// of the 152 SMs.
constexpr int kNormRopeBwdBlocks = 152 * 2;

// Lets `kernel` have `bytes` of dynamic shared memory, once per device: the call
// takes a microsecond of host time.
template <typename F> inline cudaError_t allow_smem(F *kernel, size_t bytes, std::atomic<uint64_t> &devices) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_release);
    return e;
}

// The kernels of one call, one after the other. One launched by next, but for the
// call's first, may be put on the SMs while the one before it runs out: it waits until
// that one and its writes are done (and so everything before it), at its start
// (after_previous) or later (await_previous), and what an earlier kernel of the call
// wrote it reads behind that, with plain loads, not through the read-only path. It
// may read without a wait what kernels before the previous one wrote where the
// previous one lets it start (let_next_start) only behind a wait of its own, as
// the kernels of dk and dv in front of those of dq do; it still waits before it ends,
// since whoever comes next waits for it alone. Measured with it and without: the scan
// of a forward over 4 x 4096 tokens x 16 heads, 122.7 and 125.2 us for the call; a
// backward over 2 x 999 x 4, fp32, 63.0 and 63.5; the window's gradients of 4 x 4096 x
// 16, 469 and 474. Linear attention's tensor-core kernels, one CTA an SM, are launched
// by whole, as usual: launched early they made the long forward (131072 tokens) 1502
// us from 1372 and the backward of 4 x 4096 x 16 468 from 454.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void after_previous() {
    let_next_start();
    await_previous();
}
struct Launches {
    cudaStream_t stream;
    bool first = true;
    template <typename... P, typename... A>
    cudaError_t next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, A &&...args) {
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t c{};
        c.gridDim = grid;
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = smem;
        c.stream = stream;
        c.attrs = &early;
        c.numAttrs = first ? 0 : 1;
        first = false;
        return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
    }
    template <typename... P, typename... A>
    cudaError_t next_clusters(void (*kernel)(P...), unsigned clusters, unsigned size, int threads, size_t smem, A &&...args) {
        cudaLaunchAttribute attr[2]{};
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(clusters * size);
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = smem;
        c.stream = stream;
        c.attrs = attr;
        c.numAttrs = first ? 1 : 2;
        first = false;
        return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
    }
    template <typename... P, typename... A>
    cudaError_t whole(void (*kernel)(P...), dim3 grid, int threads, size_t smem, A &&...args) {
        first = false;
        kernel<<<grid, threads, smem, stream>>>(static_cast<P>(args)...);
        return cudaGetLastError();
    }
};

struct NormRopeArgs {
    kda_dtype_t dt;
    const void *q, *k;            // token strides in elements, heads contiguous
    int64_t q_stride, k_stride;
    const void *dyq, *dyk;        // backward: gradients of the outputs, contiguous
    void *yq, *yk, *dxq, *dxk;    // contiguous
    const int32_t *positions;     // [tokens], of several axes [axes][tokens]
    const float *table;           // [max_position][rot]: cosines, then sines
    const float *wq, *wk;         // [d], nullable
    float *dwq, *dwk, *partial;   // backward: [d], nullable; partial null when neither is wanted
    int32_t *status;              // nullable
    int64_t tokens;
    int hq, hk, d, rot, max_position, norm, layout;
    float eps;
    int axes;                     // 0: one position a token
    uint64_t axis_bits[2];        // several: the axis of every channel pair, two bits each
    bool quads;                   // aligned groups of four pairs share an axis
};
constexpr int kRopeAxes = 4;      // at most
cudaError_t launch_norm_rope(const NormRopeArgs &p, bool back, cudaStream_t s);

// ---------------------------------------------------------------- linear attention
// A sequence is cut into blocks of at most `sb` tokens (its own grid, from its
// first token). Packed batches keep a table of blocks, written on the device
// by launch_linear_blocks; equal lengths need none.
struct LinBlock {
    int seq;    // sequence
    int start;  // first token
    int len;    // tokens (0: no such block, nothing to do)
};
struct LinGeom {
    const int4 *blocks;        // packed: {seq, start, len, 0} per block, in the order they are worked on, else null
    const int32_t *seq_block;  // packed: first block of each sequence [N + 1]
    const int32_t *status;     // packed: nonzero = bad cu_seqlens, nothing is written
    const int32_t *place;      // packed, nullable: where in `blocks` the i-th block from the front of the batch is
    int N, T, H;               // equal lengths: T tokens each; packed: T_total
    int sb;                    // tokens per block, a multiple of kLinChunk
    int per_seq;               // equal lengths: blocks per sequence
    int nblocks;               // blocks (packed: an upper bound)
    FastDiv by_heads, by_seq;  // divisions by H and by per_seq
};
constexpr int kLinChunk = 64;

// FRESH: in a kernel that may have been launched before the table was written.
template <bool FRESH = false> __device__ __forceinline__ LinBlock lin_block(const LinGeom &g, int b) {
    if (g.blocks) {
        const int4 x = FRESH ? g.blocks[b] : __ldg(g.blocks + b);
        return {x.x, x.y, x.z};
    }
    const int n = g.by_seq.div(b), i = b - n * g.per_seq;
    const int off = i * g.sb;
    return {n, n * g.T + off, min(g.sb, g.T - off)};
}
// Blocks [first, last) of sequence n, counted from the front of the batch.
template <bool FRESH = false>
__device__ __forceinline__ void lin_seq_blocks(const LinGeom &g, int n, int &first, int &last) {
    if (g.blocks) {
        first = FRESH ? g.seq_block[n] : __ldg(g.seq_block + n);
        last = FRESH ? g.seq_block[n + 1] : __ldg(g.seq_block + n + 1);
    } else {
        first = n * g.per_seq;
        last = first + g.per_seq;
    }
}

// Log decays. A sum over a block is taken in fixed point (base 2, steps of
// 2^-40, exact in 64 bits), so that the difference of two sums has no
// cancellation error however far down the block it lies; it is handed on as a
// pair of floats, the nearest whole number and the rest. (All conversions are
// 32-bit ones: in fp64 this pair took 8 us of a warp's time for 256 tokens.) A
// token's rounding comes out the same for every token where the decay is
// constant: with steps of 2^-31 the initial state was 1.9e-5 off after 131,072
// tokens of g = -3e-6.
// A decay of e^-128 already leaves nothing of an fp32 state (2^-185 of its
// largest value), so every log decay is clamped there, -inf (a reset) included.
// That is 184.7 octaves a token, so the whole part of a sum is exact in a
// float's 24 bits over 90,000 tokens at most; kLongestSegment is the longest
// stretch that is ever summed.
// A NaN is clamped too, so that sums and ratios stay numbers; it is carried on
// beside them (nan_before, nan_after): the decay of a stretch is NaN where the
// stretch's NaN nearest to the token it leads to has no reset in between, as in
// the recurrence, where the state is NaN from a NaN decay to the next reset.
constexpr float kMinLogDecay = -128.f;
constexpr int kDecayBits = 40;
constexpr int kLongestSegment = 4096;
static_assert(kLongestSegment <= (1 << 24) / 185, "whole parts of sums are exact as floats");
static_assert(kLongestSegment <= (1ll << (62 - kDecayBits)) / 185, "sums fit in 64 bits");
__device__ __forceinline__ long long decay_fixed(float g) {
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = (float)(1.4426950408889634074 - (double)kLog2e);
    const float x = fminf(fmaxf(g, kMinLogDecay), -kMinLogDecay);
    const float hi = x * kLog2e, lo = fmaf(x, kLog2e, -hi) + x * kLog2eLow, whole = truncf(hi);
    // hi's fraction in steps of 2^-31, then what is left of it and lo
    const float part = (hi - whole) * 2147483648.f;
    const int p = __float2int_rn(part);
    return (long long)(int)whole * (1ll << kDecayBits) + (long long)p * (1ll << (kDecayBits - 31)) +
           __float2int_rn((part - (float)p) * 512.f + lo * 1099511627776.f);
}
static_assert(kDecayBits == 40, "the constants of decay_fixed and decay_pair");
__device__ __forceinline__ float2 decay_pair(long long fixed) {
    const unsigned long long q = (unsigned long long)fixed + (1ull << (kDecayBits - 1));
    const uint32_t lo = (uint32_t)q, hi = (uint32_t)(q >> 32);
    const int whole = (int)hi >> 8, rest = (int)(__funnelshift_r(lo, hi, 8) ^ 0x80000000u);  // 2^-32 steps from the half up
    return make_float2((float)whole, (float)rest * (1.f / 4294967296.f));
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^{a - b} of two sums
__device__ __forceinline__ float decay_ratio(float2 a, float2 b) {
    return exp2_approx((a.x - b.x) + (a.y - b.y));
}
// The NaN and the reset log decays among 64 tokens, one bit each.
struct DecayEvents {
    uint32_t nan[2], reset[2];
    __device__ __forceinline__ bool any_nan() const { return (nan[0] | nan[1]) != 0u; }
    __device__ __forceinline__ unsigned long long nans() const { return nan[0] | (unsigned long long)nan[1] << 32; }
    __device__ __forceinline__ unsigned long long all() const {
        return nans() | reset[0] | (unsigned long long)reset[1] << 32;
    }
    // the decay over tokens 0 .. i is NaN
    __device__ __forceinline__ bool nan_before(int i) const {
        if (!any_nan()) return false;
        const unsigned long long e = all() & ((2ull << i) - 1);
        return e && (nans() >> (63 - __clzll((long long)e)) & 1);
    }
    // the decay over tokens i + 1 .. 63 is NaN
    __device__ __forceinline__ bool nan_after(int i) const {
        if (!any_nan()) return false;
        const unsigned long long e = i < 0 ? all() : all() & ~((2ull << i) - 1);
        return e && (nans() >> (__ffsll((long long)e) - 1) & 1);
    }
};
// The decay f over a whole block, for the scan. A slow decay is a number close to
// one, the same for every block where it is constant, and its rounding then adds
// up with the blocks: so f - 1 stands for an f above 2^-1/2 (negative, or -0), and
// f itself (0 or positive) for the others.
__device__ __forceinline__ float decay_total(long long fixed) {
    if (fixed > 0 || fixed < -(1ll << (kDecayBits - 1))) return decay_ratio(decay_pair(fixed), make_float2(0.f, 0.f));
    return fixed ? expm1f((float)fixed * (0.693147181f / 1099511627776.f)) : -0.f;
}
__device__ __forceinline__ float decay_times(float total, float s) {  // f s; a reset leaves nothing, whatever s held
    const int bits = __float_as_int(total);
    return bits == 0 ? 0.f : bits > 0 ? total * s : fmaf(total, s, s);
}
// Four elements of the scan, S <- f S + c own. The rounding of S itself adds up
// with the blocks too: what a slow decay takes off is the same few units of S's
// last place from block to block, and so is what rounds away of it (2048 blocks
// of 64 tokens at g = -3e-8: 5e-5 of S). So under a slow decay what a sum rounds
// off is put into the next one (Kahan 1965). f is the same for a whole CTA.
struct ScanElements {
    float s[4], e[4];
    __device__ __forceinline__ explicit ScanElements(float4 x) {
        s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w;
        e[0] = e[1] = e[2] = e[3] = 0.f;
    }
    __device__ __forceinline__ float4 value() const { return make_float4(s[0], s[1], s[2], s[3]); }
    // Whether the state, the next COUNT blocks' own states and their totals are all numbers.
    template <int COUNT>
    __device__ __forceinline__ bool finite(const float4 (&own)[COUNT], const float (&total)[COUNT], int count) const {
        float z = 0.f;  // 0 times anything else is NaN
#pragma unroll
        for (int i = 0; i < 4; ++i) z = fmaf(0.f, s[i], z);
#pragma unroll
        for (int u = 0; u < COUNT; ++u)
            if (u < count)
                z = fmaf(0.f, own[u].x, fmaf(0.f, own[u].y, fmaf(0.f, own[u].z, fmaf(0.f, own[u].w, fmaf(0.f, total[u], z)))));
        return z == 0.f;
    }
    // a slow decay: s + y with y = (f - 1) s + e + c own; another: y = f (s + e) + c own alone
    __device__ __forceinline__ void step(float total, float c, float4 own) {
        const bool slow = __float_as_int(total) < 0;
        const float x[4] = {own.x, own.y, own.z, own.w}, keep = slow ? 1.f : 0.f, ef = slow ? 1.f : total;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float y = fmaf(c, x[i], fmaf(total, s[i], e[i] * ef)), t = fmaf(s[i], keep, y);
            e[i] = __fsub_rn(y, fmaf(-keep, s[i], t));
            s[i] = t;
        }
    }
    // with infinities or NaN: a reset leaves nothing of them, another decay leaves them as they are
    __device__ __forceinline__ void step_any(float total, float c, float4 own) {
        const float f = __float_as_int(total) < 0 ? 1.f + total : total, x[4] = {own.x, own.y, own.z, own.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = fmaf(c, x[i], f == 0.f ? 0.f : f * s[i]);
            e[i] = 0.f;
        }
    }
};
// Prefix sums of a block's log decays: for threads 0 .. NT - 1 (all of them
// call), a[i + 1] = sum of the first i + 1, a[0] = 0, for i < len; entries up
// to `upto` (64 at most) repeat the total. `scan` is NT / 32 long longs of shared
// memory; `events` lies there too. Returns the total. Ends with a barrier.
template <int NT>
__device__ __forceinline__ long long decay_prefix(const float *log_decay, int kind, int64_t start, int H, int h, int len,
                                             int upto, float2 *a, long long *scan, DecayEvents *events) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long base = 0;
    if (tid == 0) a[0] = make_float2(0.f, 0.f);
    for (int i0 = 0; i0 < upto; i0 += NT) {
        const int i = i0 + tid;
        float g = 0.f;
        if (i < len && kind != KDA_DECAY_NONE) g = kind == KDA_DECAY_HEAD ? log_decay[h] : log_decay[(start + i) * H + h];
        long long x = decay_fixed(g);
        if (warp < 2) {
            const uint32_t n = __ballot_sync(0xffffffffu, g != g), r = __ballot_sync(0xffffffffu, g <= kMinLogDecay);
            if (lane == 0) events->nan[warp] = n, events->reset[warp] = r;
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        long long before = base, all = base;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) before += scan[w];
            all += scan[w];
        }
        if (i < upto) a[i + 1] = decay_pair(before + x);
        base = all;
        __syncthreads();
    }
    return base;
}

struct LinArgs {
    kda_dtype_t dt;
    const void *q, *k, *v;           // token strides in elements
    int64_t q_stride, k_stride, v_stride;
    const float *log_decay;
    int decay;                       // kda_decay_t
    const float *s0;                 // nullable
    void *o;
    float *sT;                       // nullable
    float scale;
    int dk, dv;
    const int32_t *cu_seqlens;       // nullable
    int N, T, H;
    int32_t *status;                 // packed: the caller's, nullable
    void *workspace;
    // backward only
    const void *d_o;
    const float *dsT;                // nullable
    void *dq, *dk_out, *dv_out;
    float *d_decay, *ds0;            // nullable
};
size_t linear_workspace_bytes(int N, int64_t T, int H, int dk, int dv, kda_dtype_t dt, bool packed);
size_t linear_backward_workspace_bytes(int N, int64_t T, int H, int dk, int dv, kda_dtype_t dt, bool packed);
cudaError_t launch_linear(const LinArgs &a, cudaStream_t s);
cudaError_t launch_linear_backward(const LinArgs &a, cudaStream_t s);
cudaError_t launch_linear_status(int32_t *status, int value, cudaStream_t s);

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, kda_dtype_t dt, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, const float *log_decay, int decay, float scale,
                                 float *state, const int32_t *slots, int pool_size, int32_t *status, void *o, int N,
                                 int H, int dk, int dv, cudaStream_t s);

}  // namespace kda
