// Linear attention with a decay on the tensor cores of sm_103a: bf16 inputs,
// d_k = d_v = 128. The same three steps as the general kernels (a block's own
// state, the scan over the blocks, the outputs), with tcgen05.mma, TMEM and TMA.
//
// The state, attend and roll kernels are persistent, one CTA per SM, with the
// pipeline running on from one work item to the next; roles are warps that meet
// at mbarriers. Every
// wait is bounded: a wait that runs out sets the device error word and the
// CTA's abort flag, every role leaves its loop, and the CTA ends normally.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include "kda_linear.cuh"
#include "kda_linear_tc.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int D = 128;
__device__ int g_lin_error;

// ---------------------------------------------------------------- waits
struct Abort {
    volatile int *flag;  // shared memory
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (*flag) return false;
            if (clock64() - t0 > kWaitCycles) {
                *flag = 1;
                atomicOr(&g_lin_error, 1);
                return false;
            }
        }
        return true;
    }
};
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {  // two bf16 products, each rounded once
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// One arrival for the warp, after all its lanes have come here.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// After an abort: copies that were on their way land before the CTA leaves.
__device__ __forceinline__ void settle(const Abort &ab) {
    if (*ab.flag) {
        const long long t0 = clock64();
        while (clock64() - t0 < 100000) {
        }
        __syncthreads();
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ F2 pair_f(uint32_t x) { return f2(lo_f(x), hi_f(x)); }  // two bf16
__device__ __forceinline__ F2 pair_w(uint32_t a, uint32_t b) { return f2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ uint32_t pack2(F2 x) {
    float a, b;
    f2_get(x, a, b);
    return pack2(a, b);
}
__device__ __forceinline__ F2 minus(F2 x, F2 y) { return fma2(y, f2(-1.f, -1.f), x); }
// x = h + m + l, each a bf16 (24 bits of x kept), two values at a time.
__device__ __forceinline__ void split3(F2 x, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = pack2(x);
    x = minus(x, pair_f(h));
    m = pack2(x);
    l = pack2(minus(x, pair_f(m)));
}
// v *= f, 32 accumulator columns; f = 0 (a reset) leaves zeros whatever v held.
__device__ __forceinline__ void scale32(uint32_t (&v)[32], float f) {
    if (__any_sync(0xffffffffu, f == 0.f)) {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = f == 0.f ? 0u : v[e];
    }
    const F2 ff = f2(f, f);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float a, b;
        f2_get(pair_w(v[e], v[e + 1]) * ff, a, b);
        v[e] = __float_as_uint(a), v[e + 1] = __float_as_uint(b);
    }
}
__device__ __forceinline__ void scale16(uint32_t (&v)[16], float f) {  // the same for 16 columns
    if (f == 0.f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0u;
    }
    const F2 ff = f2(f, f);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        float a, b;
        f2_get(pair_w(v[e], v[e + 1]) * ff, a, b);
        v[e] = __float_as_uint(a), v[e + 1] = __float_as_uint(b);
    }
}
__device__ __forceinline__ void st_v8(void *p, const uint32_t (&r)[8]) {  // one 32-byte sector
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z) {  // into L2
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// D[tmem] += A[tmem] * B[smem]: A holds two bf16 of K per 32-bit column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, 1, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc)
        : "memory");
}
// MMA descriptors of a tile, advanced by constants: the address field counts
// 16-byte steps. One thread issues every MMA, so its instructions between two
// of them are time the tensor core waits.
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }     // K-major
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, uint32_t atom) { return sdesc_sw128(tile, atom, 1024); }
// offset of step ks (16 of K): K-major tiles have 64 of K per atom of `atom` bytes
__device__ __forceinline__ constexpr uint64_t step_k(int ks, uint32_t atom) {
    return ((ks >> 2) * atom + (ks & 3) * 32) >> 4;
}
__device__ __forceinline__ constexpr uint64_t step_mn(int ks) { return (uint64_t)(ks * 2048) >> 4; }
template <bool ACC> __device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}
// NaN log decays among a warp's tokens (laid out as in warp_decay): which of the
// decays are NaN, by the rule at kMinLogDecay.
struct WarpNan {
    uint32_t bits;  // below; 0 where there is no NaN
    bool event;     // there is a NaN or a reset
    // bit u: the decay over the tokens up to this lane's u-th, that one included; over those behind it
    __device__ __forceinline__ uint32_t before() const { return bits & 0xff; }
    __device__ __forceinline__ uint32_t after() const { return bits >> 8 & 0xff; }
    // the first of them, the last of them is a NaN: the decay over all, in reverse and forward
    __device__ __forceinline__ bool first() const { return bits >> 16 & 1; }
    __device__ __forceinline__ bool last() const { return bits >> 17 & 1; }
};
// Out of line: the kernels' loops are short for the instruction cache.
__device__ __noinline__ uint32_t warp_nan_bits(uint32_t nan, uint32_t events) {
    const uint32_t lanes = __ballot_sync(0xffffffffu, events != 0u),
                   ends = __ballot_sync(0xffffffffu, events && (nan >> (31 - __clz(events)) & 1)),
                   starts = __ballot_sync(0xffffffffu, events && (nan >> (__ffs(events) - 1) & 1)),
                   lane = threadIdx.x & 31, earlier = lanes & ((1u << lane) - 1), later = lanes & ~((2u << lane) - 1);
    uint32_t r = (starts >> (__ffs(lanes) - 1) & 1) << 16 | (ends >> (31 - __clz(lanes)) & 1) << 17;
    uint32_t on = earlier ? ends >> (31 - __clz(earlier)) & 1 : 0u;
#pragma unroll 1
    for (int u = 0; u < 8; ++u) {
        if (events >> u & 1) on = nan >> u & 1;
        r |= on << u;
    }
    on = later ? starts >> (__ffs(later) - 1) & 1 : 0u;
#pragma unroll 1
    for (int u = 7; u >= 0; --u) {
        r |= on << (8 + u);
        if (events >> u & 1) on = nan >> u & 1;
    }
    return r;
}
template <int PER> __device__ __forceinline__ WarpNan warp_nan(const float (&g)[PER]) {
    static_assert(PER <= 8, "bits of a lane");
    uint32_t nan = 0, events = 0;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        nan |= (g[u] != g[u] ? 1u : 0u) << u;
        events |= (!(g[u] > kMinLogDecay) ? 1u : 0u) << u;
    }
    WarpNan r{0u, __any_sync(0xffffffffu, events != 0u) != 0};
    if (r.event && __any_sync(0xffffffffu, nan != 0u)) r.bits = warp_nan_bits(nan, events);
    return r;
}
// A warp's prefix sums of a block's log decays (fixed point): lane l holds
// tokens l * per .. l * per + per - 1; `mine` receives its inclusive sums.
template <int PER>
__device__ __forceinline__ long long warp_decay(const LinGeom &geo, const float *log_decay, int decay,
                                                const LinBlock &blk, int h, long long (&mine)[PER], WarpNan &nan) {
    const int lane = threadIdx.x & 31;
    float g[PER];  // all loads first: one after the other they cost a memory latency each
    const float head = decay == KDA_DECAY_HEAD ? __ldg(log_decay + h) : 0.f;
    const bool token = decay == KDA_DECAY_TOKEN;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int i = lane * PER + u;
        g[u] = i < blk.len ? head : 0.f;
        if (token && i < blk.len) g[u] = __ldg(log_decay + (int64_t)(blk.start + i) * geo.H + h);
    }
    nan = warp_nan<PER>(g);
    long long run = 0;
#pragma unroll
    for (int u = 0; u < PER; ++u) mine[u] = run += decay_fixed(g[u]);
    long long x = run;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    const long long before = x - run;
#pragma unroll
    for (int u = 0; u < PER; ++u) mine[u] += before;
    return __shfl_sync(0xffffffffu, x, 31);
}

// ================================================================ a block's own state
// out = sum_s w_s x_s y_s^T (see lin_state_kernel) as a GEMM with M = d_v,
// N = d_k and the block's tokens as K, 64 at a time (the transposed state, so
// that a warp's 32 accumulator rows are 32 neighbours in memory). x is scaled by
// w in fp32 and split in three bf16 parts, so the products keep 24 bits; the
// high part and the two lower ones have accumulators of their own, since the
// tensor core cuts a sum off at its accumulator's last bit: the lower products
// would cost the high ones that many cuts. High and middle part lie side by
// side, so one MMA with N = 256 takes both and reads y once.
// Bound by memory: 32 KB of x and y a tile; next come the 176 KB that a tile
// moves through shared memory. 4 x 4096 tokens x 16 heads, d = 128: 39-42 us for
// 135 MB (3.4 TB/s, a block or two per SM and its first loads unhidden);
// 131072 x 32: 450-466 us for 2.15 GB (4.7 TB/s, 70 % of a copy).
// A block longer than kLinMaxBlock goes in parts of that length, joined by the
// decays of the parts, as the blocks are by the scan.
//
// warp 0: TMA; 1: MMA; 2: weights, an item ahead; 4-7: accumulators out;
// 8-15 and 16-23: x -> three parts (the high one in place), tiles in turn. Each
// of the two groups has full barriers of its own (of a shared one it would miss
// the phases of the other's tiles).
constexpr int ST_TOK = 64;
constexpr int ST_TILE = ST_TOK * D * 2;       // 16 KB
constexpr int ST_STAGE = 4 * ST_TILE;         // x (then its high part), middle, low, y
constexpr int ST_STAGES = 3;
// The parts' join factors, from the weights' warp to the accumulator warps. The
// ring needs no barrier of its own: the factor of part q is written once part
// q - 2 is converted, so its last tile, n, is in shared memory and tile
// n - ST_STAGES, of part q - 5 or a later one, multiplied; that part's
// accumulators were free, so those of part q - 7 had been read out, and its
// factor with them. Seven factors may be waiting to be read.
constexpr int ST_JOIN = 8;
static_assert(ST_STAGES == 3 && ST_JOIN >= 7, "factors that may be waiting");
constexpr int ST_THREADS = 768;
constexpr int ST_W = ST_STAGES * ST_STAGE;                   // weights [2][kLinMaxBlock]
constexpr int ST_BAR = ST_W + 2 * kLinMaxBlock * 4;
enum { SB_FULL = 0, SB_CONV = 6, SB_EMPTY = 9, SB_ACC_FULL = 12, SB_ACC_EMPTY = 14, SB_W_FULL = 16, SB_W_EMPTY = 18,
       SB_COUNT = 20 };
constexpr int ST_SMEM = ST_BAR + SB_COUNT * 8 + 16 + 1024;

struct StateTcArgs {
    LinGeom geo;
    const float *log_decay;
    int decay;
    float *out, *total, *total_rev;
    int items;
};

template <bool REV>
__global__ void __launch_bounds__(ST_THREADS, 1)
lin_state_tc_kernel(StateTcArgs p, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my) {
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + ST_BAR);
    float *wts = reinterpret_cast<float *>(sm + ST_W);
    __shared__ float join[ST_JOIN];
    uint32_t *tm = reinterpret_cast<uint32_t *>(bar + SB_COUNT);
    const Abort ab{reinterpret_cast<volatile int *>(tm + 1)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LinGeom &geo = p.geo;
    if (tid == 0) {
        *ab.flag = 0;
        for (int i = 0; i < 3; ++i) {
            mbar_init(bar + SB_FULL + i, 1);
            mbar_init(bar + SB_FULL + 3 + i, 1);
            mbar_init(bar + SB_CONV + i, 8);
            mbar_init(bar + SB_EMPTY + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + SB_ACC_FULL + i, 1);
            mbar_init(bar + SB_ACC_EMPTY + i, 4);
            mbar_init(bar + SB_W_FULL + i, 1);
            mbar_init(bar + SB_W_EMPTY + i, 16);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&mx);
            prefetch_tmap(&my);
            int n = 0;  // tiles so far
            for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
                const int b = geo.by_heads.div(it), h = it - b * geo.H;
                const LinBlock blk = lin_block(geo, b);
                for (int t0 = 0; t0 < blk.len; t0 += ST_TOK, ++n) {
                    const int s = n % ST_STAGES, ph = (n / ST_STAGES) & 1;
                    if (!(ok = ab.wait(bar + SB_EMPTY + s, ph ^ 1))) break;
                    unsigned char *st = sm + s * ST_STAGE;
                    uint64_t *f = bar + SB_FULL + n % 6;
                    mbar_arrive_expect_tx(f, 2 * ST_TILE);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tma_load_3d(st + c * (ST_TILE / 2), &mx, f, 64 * c, h, blk.start + t0);
                        tma_load_3d(st + 3 * ST_TILE + c * (ST_TILE / 2), &my, f, 64 * c, h, blk.start + t0);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t I2 = idesc_bf16(128, 256, true, true), I1 = idesc_bf16(128, 128, true, true);
            int n = 0, q = 0;
            for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
                const LinBlock blk = lin_block(geo, geo.by_heads.div(it));
                if (blk.len <= 0) continue;
                for (int p0 = 0; p0 < blk.len && ok; p0 += kLinMaxBlock, ++q) {
                    const int buf = q & 1, end = min(blk.len, p0 + kLinMaxBlock);
                    if (!(ok = ab.wait(bar + SB_ACC_EMPTY + buf, ((q >> 1) & 1) ^ 1))) break;
                    const uint32_t hi = tmem + buf * 256, lo = hi + 128;
                    for (int t0 = p0; t0 < end; t0 += ST_TOK, ++n) {
                        const int s = n % ST_STAGES;
                        if (!(ok = ab.wait(bar + SB_CONV + s, (n / ST_STAGES) & 1))) break;
                        tc_fence_after();
                        const uint64_t x = desc_mn(smem_u32(sm + s * ST_STAGE), ST_TILE / 2);
                        constexpr uint64_t L = (2 * ST_TILE) >> 4, Y = (3 * ST_TILE) >> 4;
                        if (t0 == p0) mma_ss<false>(hi, x + Y, x, I2);
                        else mma_ss<true>(hi, x + Y, x, I2);
                        mma_ss<true>(lo, x + Y, x + L, I1);
#pragma unroll
                        for (int ks = 1; ks < ST_TOK / 16; ++ks) {
                            mma_ss<true>(hi, x + Y + step_mn(ks), x + step_mn(ks), I2);
                            mma_ss<true>(lo, x + Y + step_mn(ks), x + L + step_mn(ks), I1);
                        }
                        umma_commit(bar + SB_EMPTY + s);
                    }
                    if (!ok) break;
                    umma_commit(bar + SB_ACC_FULL + buf);
                }
            }
        }
    } else if (warp == 2) {
        int q = 0;  // parts so far
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const int b = geo.by_heads.div(it), h = it - b * geo.H;
            const LinBlock blk = lin_block(geo, b);
            long long sum = 0;  // over the block's earlier parts
            bool event = false, first = false, last = false;  // as in WarpNan, over the block
            for (int p0 = 0; p0 < blk.len; p0 += kLinMaxBlock, ++q) {
                constexpr int PER = kLinMaxBlock / 32;
                long long a[PER];
                const LinBlock part{blk.seq, blk.start + p0, min(kLinMaxBlock, blk.len - p0)};
                WarpNan nan;
                const long long all = warp_decay<PER>(geo, p.log_decay, p.decay, part, h, a, nan);
                if (nan.event) {
                    first = event ? first : nan.first();
                    last = nan.last();
                    event = true;
                }
                ok = __all_sync(0xffffffffu, ab.wait(bar + SB_W_EMPTY + (q & 1), ((q >> 1) & 1) ^ 1));
                if (!ok) break;
                float *w = wts + (q & 1) * kLinMaxBlock;
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    w[lane * PER + u] = decay_ratio(decay_pair(REV ? a[u] : all - a[u]), make_float2(0.f, 0.f));
                // what the sum so far (forward) or this part (reverse) is multiplied by when they are joined
                if (lane == 0)
                    join[q % ST_JOIN] = decay_ratio(decay_pair(REV ? sum : all), make_float2(0.f, 0.f));
                warp_arrive(bar + SB_W_FULL + (q & 1));
                sum += all;
            }
            if (!REV && lane == 0 && blk.len > 0) {
                const int64_t at = (int64_t)b * geo.H + h;
                const float total = decay_total(sum);
                if (p.total) p.total[at] = last ? CUDART_NAN_F : total;
                if (p.total_rev) p.total_rev[at] = first ? CUDART_NAN_F : total;
            }
        }
    } else if (warp >= 4 && warp < 8) {
        int q = 0;
        const int row = tid - 128;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const LinBlock blk = lin_block(geo, geo.by_heads.div(it));
            if (blk.len <= 0) continue;
            float *dst = p.out + (int64_t)it * D * D + row;  // row: the value column
            for (int p0 = 0; p0 < blk.len; p0 += kLinMaxBlock, ++q) {
                const int buf = q & 1;
                ok = __all_sync(0xffffffffu, ab.wait(bar + SB_ACC_FULL + buf, (q >> 1) & 1));
                if (!ok) break;
                tc_fence_after();
                // a later part joins the sum in memory (in L2: it is this CTA's own 64 KB), in fp32 sums that
                // round, where the tensor core's would cut
                const float f = join[q % ST_JOIN], f_old = REV ? 1.f : f, f_new = REV ? f : 1.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t x[32], y[32];
                    tmem_ld32(tmem + lanes + buf * 256 + c, x);
                    tmem_ld32(tmem + lanes + buf * 256 + 128 + c, y);
                    tmem_wait_ld();
                    if (p0 == 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            dst[(c + e) * D] = __uint_as_float(x[e]) + __uint_as_float(y[e]);
                    } else {
                        float old[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) old[e] = dst[(c + e) * D];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            dst[(c + e) * D] =
                                f_old * old[e] + f_new * (__uint_as_float(x[e]) + __uint_as_float(y[e]));
                    }
                }
                tc_fence_before();
                warp_arrive(bar + SB_ACC_EMPTY + buf);
            }
        }
    } else if (warp >= 8) {
        const int t = (tid - 256) & 255, group = (tid - 256) >> 8;
        const uint32_t off = kmajor_chunk(t >> 4, t & 15, ST_TOK);
        int n = 0, q = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const LinBlock blk = lin_block(geo, geo.by_heads.div(it));
            if (blk.len <= 0) continue;
            for (int p0 = 0; p0 < blk.len && ok; p0 += kLinMaxBlock, ++q) {
                ok = __all_sync(0xffffffffu, ab.wait(bar + SB_W_FULL + (q & 1), (q >> 1) & 1));
                const float *w = wts + (q & 1) * kLinMaxBlock;
                const int end = min(blk.len, p0 + kLinMaxBlock);
                for (int t0 = p0; t0 < end && ok; t0 += ST_TOK, ++n) {
                    const int s = n % ST_STAGES, rows = blk.len - t0;
                    if ((n & 1) != group) continue;
                    if (!(ok = __all_sync(0xffffffffu, ab.wait(bar + SB_FULL + n % 6, (n / 6) & 1)))) break;
                    unsigned char *st = sm + s * ST_STAGE;
                    uint4 v[4];
                    float f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // rows 16 i + t / 16, channels 8 (t % 16) ..
                        v[i] = *reinterpret_cast<const uint4 *>(st + off + i * 2048);
                        f[i] = w[t0 - p0 + 16 * i + (t >> 4)];
                    }
                    if (rows < ST_TOK) {  // past the block's end: neither operand may hold what lies there
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (16 * i + (t >> 4) >= rows) {
                                v[i] = make_uint4(0u, 0u, 0u, 0u);
                                *reinterpret_cast<uint4 *>(st + 3 * ST_TILE + off + i * 2048) = v[i];
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint4 h, m, l;
                        const F2 ff = f2(f[i], f[i]);
                        split3(pair_f(v[i].x) * ff, h.x, m.x, l.x);
                        split3(pair_f(v[i].y) * ff, h.y, m.y, l.y);
                        split3(pair_f(v[i].z) * ff, h.z, m.z, l.z);
                        split3(pair_f(v[i].w) * ff, h.w, m.w, l.w);
                        *reinterpret_cast<uint4 *>(st + off + i * 2048) = h;
                        *reinterpret_cast<uint4 *>(st + ST_TILE + off + i * 2048) = m;
                        *reinterpret_cast<uint4 *>(st + 2 * ST_TILE + off + i * 2048) = l;
                    }
                    fence_proxy_async();
                    warp_arrive(bar + SB_CONV + s);
                }
                if (ok) warp_arrive(bar + SB_W_EMPTY + (q & 1));
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    settle(ab);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ================================================================ joining the blocks
// As lin_scan_kernel, with the states handed on as three bf16 parts (24 bits),
// which the output kernel with row dots multiplies with; the first part alone
// is the state rounded to bf16. In reverse also <S, G> of every block. Bound by
// memory: 1024 blocks and heads of 128 x 128, 24 us forward (67 MB in, 101 out:
// 7.0 TB/s), 40-42 us in reverse (another 101 MB in: 6.4-6.7 TB/s).
constexpr int SC_THREADS = 256;
template <bool REV>
__global__ void __launch_bounds__(SC_THREADS)
lin_scan_tc_kernel(LinGeom geo, const float *__restrict__ own, const float *__restrict__ total,
                   const float *__restrict__ s0, float *__restrict__ sT, float c, __nv_bfloat16 *__restrict__ parts,
                   int64_t part_stride, const __nv_bfloat16 *__restrict__ other, float *__restrict__ inner) {
    if (geo.status && *geo.status != KDA_DEV_OK) return;
    constexpr int SIZE4 = D * D / 4, PER = SIZE4 / SC_THREADS;
    const int64_t nh = blockIdx.x / PER;
    const int n = (int)(nh / geo.H), h = (int)(nh % geo.H);
    const int64_t e = (int64_t)(blockIdx.x % PER) * SC_THREADS + threadIdx.x;
    int first, last;
    lin_seq_blocks(geo, n, first, last);
    ScanElements state(s0 ? reinterpret_cast<const float4 *>(s0)[nh * SIZE4 + e] : make_float4(0.f, 0.f, 0.f, 0.f));
    const float4 *p = reinterpret_cast<const float4 *>(own);
    const int count = last - first;
    constexpr bool INNER = REV;  // <S, G> of every block: G is here, S in `other`
    constexpr int AHEAD = 4;
    float4 x[AHEAD];
    float f[AHEAD];
    uint2 so[AHEAD][3];
    auto at = [&](int i) { return (int64_t)(REV ? last - 1 - i : first + i) * geo.H + h; };
    for (int i0 = 0; i0 < count; i0 += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i0 + u < count) {
                x[u] = __ldcs(p + at(i0 + u) * SIZE4 + e);
                f[u] = __ldg(total + at(i0 + u));
                if (INNER) {
                    const uint2 *o = reinterpret_cast<const uint2 *>(other) + at(i0 + u) * SIZE4 + e;
#pragma unroll
                    for (int k = 0; k < 3; ++k) so[u][k] = __ldg(o + k * (part_stride / 4));
                }
            }
        const bool finite = state.finite(x, f, count - i0);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i0 + u < count) {
                const float4 S = state.value();
                if (INNER) {
                    float v = S.x * (lo_f(so[u][0].x) + lo_f(so[u][1].x) + lo_f(so[u][2].x)) +
                              S.y * (hi_f(so[u][0].x) + hi_f(so[u][1].x) + hi_f(so[u][2].x)) +
                              S.z * (lo_f(so[u][0].y) + lo_f(so[u][1].y) + lo_f(so[u][2].y)) +
                              S.w * (hi_f(so[u][0].y) + hi_f(so[u][1].y) + hi_f(so[u][2].y));
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
                    if ((threadIdx.x & 31) == 0)
                        inner[at(i0 + u) * kScanPartials + (blockIdx.x % PER) * (SC_THREADS / 32) + (threadIdx.x >> 5)] = v;
                }
                uint2 a, b, d;
                split3(f2(S.x, S.y), a.x, b.x, d.x);
                split3(f2(S.z, S.w), a.y, b.y, d.y);
                uint2 *o = reinterpret_cast<uint2 *>(parts) + at(i0 + u) * SIZE4 + e;
                *o = a;
                o[part_stride / 4] = b;
                o[part_stride / 2] = d;
                if (finite) state.step(f[u], c, x[u]);
                else state.step_any(f[u], c, x[u]);
            }
    }
    if (sT) reinterpret_cast<float4 *>(sT)[nh * SIZE4 + e] = state.value();
}

// ================================================================ outputs
// What the backward with a gradient of the log decay runs: dv, and dq and dk
// with their row dots. One item is a block of one or two 128-token tiles, and a
// head. Two contexts (an MMA-issuing warp, 256 row threads, one O and one P
// accumulator in TMEM each) take its two tiles of rows: the near one sees its own
// tokens alone, the far one those of both tiles (in reverse time the second tile
// is the near one); they change places from item to item. The operands come
// through two rings: x (and w) of the near tile and of the far one, which stay
// until their tile's last scores, and S, then y and z of the near tile and of the
// far one, which flow past and are read by both contexts.
// Two threads share a row, a half of the columns each.
//   O = x S, rows scaled by the decay from the block's edge (in TMEM);
//   P = x y^T, scaled by D_ij and the mask, rounded to bf16 in place (each half
//   of the columns into the front of its own half);
//   O += P z, P read from TMEM.
// P and S are the two roundings to bf16 (2^-9 relative each, as small as the
// rounding of the result itself: dv is 2.35e-3 from 64 bits in the 2-norm, the
// result's rounding alone 1.66e-3); sums are fp32. With DOTS S is exact to 24
// bits and P alone is rounded: dq and dk 1.9e-3 to 2.3e-3.
// 4 x 4096 tokens x 16 heads, 256-token blocks: dq 97 us and dk 108 with their
// dots (371 MB, 3.4 to 3.8 TB/s), dv 59 (236 MB, 4.0 TB/s). Bound by the latency
// of its loads: shared memory holds one item's operands and the first of the
// next one's. Measured before: one ring of six 32 KB slots, which gave the next S
// no room before the item's end, 106-113, 111 and 54 us; and items of their own
// for the two contexts, each loading its own S, y and z, 123, 129 and 65. With
// that one ring, prefetching the next item into L2 made the whole backward 458 us
// from 454, or 510 issued earlier: the prefetches queue before the loads.
//
// DOTS adds w_i . out_i per row, for the gradient of the decay, to fp32
// accuracy: its state part from all three parts of S, and the rest not from
// the rounded P but as sum_j c D_ij (x_i . y_j) (w_i . z_j), both dots exact in
// bf16 with fp32 sums. That takes S in three parts, w after each x, and a
// second score accumulator, so the scores go 64 columns at a time.
//
// A slot is filled again when both contexts are done with it; both wait for
// every load of a ring in turn, used or not, and so see every phase of the
// slots' barriers (a parity wait cannot tell a phase from the one two before it;
// checked with a model of the roles).
static_assert(kLinMaxBlock <= 256, "an item is one or two tiles");
// Rings in shared memory: `ROWS` slots of 32 KB for x and w, then `FLOW` of 16 KB
// (DOTS: half a part of S, or 64 tokens of y or z) or 32 KB (S whole, 128 tokens).
template <bool DOTS> struct AttendRings {
    static constexpr int SUB = DOTS ? 64 : 128;  // tokens of a flow slot, score columns at a time
    static constexpr int ROWS = DOTS ? 4 : 2, FLOW = DOTS ? 5 : 4;
    static constexpr int ROW_SLOT = 128 * D * 2, FLOW_SLOT = SUB * D * 2, HALF = FLOW_SLOT / 2;  // HALF: 64 channels
    static constexpr int FLOW_AT = ROWS * ROW_SLOT;
};
constexpr int AT_THREADS = 640;
constexpr int AT_PREFIX = 4;                                         // blocks whose prefix sums are kept
constexpr int AT_A = AttendRings<true>::FLOW_AT + AttendRings<true>::FLOW * AttendRings<true>::FLOW_SLOT;
static_assert(AT_A >= AttendRings<false>::FLOW_AT + AttendRings<false>::FLOW * AttendRings<false>::FLOW_SLOT, "rings");
constexpr int AT_COL = AT_A + AT_PREFIX * (kLinMaxBlock + 2) * 8;    // AT_A: prefix sums; column factors [16 warps][128]
constexpr int AT_NAN = AT_COL + 16 * kLinMaxBlock / 2 * 4;           // whether the state's decay is NaN, a bit a token
constexpr int AT_BAR = AT_NAN + AT_PREFIX * kLinMaxBlock / 8;
enum { AB_ROW_FULL = 0, AB_ROW_EMPTY = 4, AB_FLOW_FULL = 8, AB_FLOW_EMPTY = 13, AB_O_IN = 18, AB_O_FULL = 20,
       AB_O_EMPTY = 22, AB_P_FULL = 24, AB_P_READY = 26, AB_A_FULL = 28, AB_A_EMPTY = 32, AB_COUNT = 36 };
constexpr int AT_SMEM = AT_BAR + AB_COUNT * 8 + 16 + 1024;
static_assert(AT_SMEM <= 232448, "shared memory of an SM");

struct AttendTcArgs {
    LinGeom geo;
    const float *log_decay;
    int decay;
    __nv_bfloat16 *out;
    float c_state, c_intra;
    float *dot, *dot_state;
    int64_t dot_stride;  // between the two column halves' sums
    int state_rows;      // rows of one part of S
    int items;           // blocks and heads
};
struct Item {
    LinBlock blk;
    int b, h, tiles, near;
    // the t-th tile: the near one, then the far one
    __device__ __forceinline__ int tile(int t) const { return t ? 1 - near : near; }
};
template <bool REV> __device__ __forceinline__ Item item_of(const AttendTcArgs &p, int it) {
    Item x;
    x.b = p.geo.by_heads.div(it);
    x.h = it - x.b * p.geo.H;
    x.blk = lin_block(p.geo, x.b);
    x.tiles = (x.blk.len + 127) / 128;
    x.near = REV ? x.tiles - 1 : 0;
    return x;
}

template <bool REV, bool ST, bool DOTS>
__global__ void __launch_bounds__(AT_THREADS, 1)
lin_attend_tc_kernel(AttendTcArgs p, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                     const __grid_constant__ CUtensorMap mz, const __grid_constant__ CUtensorMap ms,
                     const __grid_constant__ CUtensorMap mw) {
    using R = AttendRings<DOTS>;
    constexpr int SUB = R::SUB;
    constexpr int NS = DOTS ? 6 : 1;          // loads of S: three parts, a half of the columns each
    constexpr int XW = DOTS ? 2 : 1;          // row loads of a tile
    constexpr int YZ = 2 * (128 / SUB);       // flow loads of a tile
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + AT_BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(bar + AB_COUNT);
    const Abort ab{reinterpret_cast<volatile int *>(tm + 1)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LinGeom &geo = p.geo;
    if (tid == 0) {
        *ab.flag = 0;
        for (int i = 0; i < R::ROWS; ++i) {
            mbar_init(bar + AB_ROW_FULL + i, 1);
            mbar_init(bar + AB_ROW_EMPTY + i, 2);
        }
        for (int i = 0; i < R::FLOW; ++i) {
            mbar_init(bar + AB_FLOW_FULL + i, 1);
            mbar_init(bar + AB_FLOW_EMPTY + i, 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + AB_O_IN + i, 1);
            mbar_init(bar + AB_O_FULL + i, 1);
            mbar_init(bar + AB_O_EMPTY + i, 8);
            mbar_init(bar + AB_P_FULL + i, 1);
            mbar_init(bar + AB_P_READY + i, 8);
        }
        for (int i = 0; i < AT_PREFIX; ++i) {
            mbar_init(bar + AB_A_FULL + i, 1);
            mbar_init(bar + AB_A_EMPTY + i, 16);
        }
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;
    bool ok = true;

    auto row_at = [&](int i) { return sm + (i % R::ROWS) * R::ROW_SLOT; };
    auto flow_at = [&](int i) { return sm + R::FLOW_AT + (i % R::FLOW) * R::FLOW_SLOT; };

    if (warp == 0) {  // S, y and z
        if (lane == 0) {
            int n = 0;
            uint64_t *f = nullptr;  // the barrier of the slot's load
            auto slot = [&]() -> unsigned char * {
                const int s = n % R::FLOW;
                if (!(ok = ok && ab.wait(bar + AB_FLOW_EMPTY + s, ((n / R::FLOW) & 1) ^ 1))) return nullptr;
                f = bar + AB_FLOW_FULL + s;
                mbar_arrive_expect_tx(f, R::FLOW_SLOT);
                return flow_at(n++);
            };
            auto tokens = [&](const CUtensorMap *m, int h, int tok) {  // SUB tokens
                unsigned char *d = slot();
                if (!d) return;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int t = 0; t < SUB / 64; ++t)
                        tma_load_3d(d + x * R::HALF + t * 8192, m, f, 64 * x, h, tok + 64 * t);
            };
            for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
                const Item x = item_of<REV>(p, it);
                for (int i = 0; i < NS && x.tiles > 0; ++i)  // the lowest part first
                    if (unsigned char *d = slot()) {
                        const int row = (DOTS ? 2 - i / 2 : 0) * p.state_rows + (x.b * geo.H + x.h) * D;
                        tma_load_2d(d, &ms, f, DOTS ? 64 * (i & 1) : 0, row);
                        if (!DOTS) tma_load_2d(d + R::HALF, &ms, f, 64, row);
                    }
                for (int t = 0; t < x.tiles; ++t)
                    for (int u = 0; u < 128; u += SUB) {
                        tokens(&my, x.h, x.blk.start + 128 * x.tile(t) + u);
                        tokens(&mz, x.h, x.blk.start + 128 * x.tile(t) + u);
                    }
            }
        }
    } else if (warp == 1 || warp == 2) {
        const int c = warp - 1;
        if (lane == 0) {
            constexpr uint32_t I_S = idesc_bf16(128, 128, false, !ST), I_P = idesc_bf16(128, SUB, false, false),
                               I_O = idesc_bf16(128, 128, false, true);
            static_assert(!DOTS || ST, "halves of a part of S are read transposed");
            const uint32_t to = tmem + c * 256, tp = to + 128, tp2 = tp + SUB;
            // row and flow loads and items before this one, tiles and pieces of this context
            int nr = 0, nf = 0, k = 0, q = 0, np = 0;
            auto row_full = [&](int i) { return ok = ok && ab.wait(bar + AB_ROW_FULL + i % R::ROWS, (i / R::ROWS) & 1); };
            auto flow_full = [&](int i) {
                return ok = ok && ab.wait(bar + AB_FLOW_FULL + i % R::FLOW, (i / R::FLOW) & 1);
            };
            auto row_free = [&](int i) { umma_commit(bar + AB_ROW_EMPTY + i % R::ROWS); };
            auto flow_free = [&](int i) { umma_commit(bar + AB_FLOW_EMPTY + i % R::FLOW); };
            // loads that only the other context uses
            auto row_skip = [&](int first, int last) {
                for (int i = first; i < last && row_full(i); ++i) mbar_arrive(bar + AB_ROW_EMPTY + i % R::ROWS);
            };
            auto flow_skip = [&](int first, int last) {
                for (int i = first; i < last && flow_full(i); ++i) mbar_arrive(bar + AB_FLOW_EMPTY + i % R::FLOW);
            };
            for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
                const Item x = item_of<REV>(p, it);
                if (x.tiles == 0) continue;
                const bool near = (k++ & 1) == c;
                const int r0 = nr, f0 = nf;
                nr += XW * x.tiles;
                nf += NS + YZ * x.tiles;
                if (!near && x.tiles == 1) {
                    row_skip(r0, nr);
                    flow_skip(f0, nf);
                    continue;
                }
                const int count = near ? 1 : 2, nx = r0 + (near ? 0 : XW);
                if (!(ok = ab.wait(bar + AB_O_EMPTY + c, (q & 1) ^ 1))) break;
                row_skip(r0, nx);
                if (!row_full(nx)) break;
                const uint64_t xd = desc_k(smem_u32(row_at(nx)));
                for (int i = 0; i < NS; ++i) {  // the lowest part first, while the sum is small
                    if (!flow_full(f0 + i)) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(flow_at(f0 + i));
                    const uint64_t sd = ST ? desc_k(sa) : desc_mn(sa, R::HALF);
                    const uint64_t xh = xd + (DOTS && (i & 1) ? step_k(4, 16384) : 0);
                    if (i == 0) mma_ss<false>(to, xh, sd, I_S);
                    else mma_ss<true>(to, xh, sd, I_S);
#pragma unroll
                    for (int ks = 1; ks < (DOTS ? 4 : 8); ++ks)
                        mma_ss<true>(to, xh + step_k(ks, 16384), sd + (ST ? step_k(ks, R::HALF) : step_mn(ks)), I_S);
                    flow_free(f0 + i);
                }
                if (!ok) break;
                umma_commit(bar + AB_O_IN + c);
                if (DOTS && !row_full(nx + 1)) break;
                const uint64_t wd = desc_k(smem_u32(row_at(nx + XW - 1)));
                int ny = f0 + NS;
                for (int j = 0; j < count && ok; ++j) {
#pragma unroll
                    for (int sub = 0; sub < 128 / SUB; ++sub, ++np, ny += 2) {
                        if (!flow_full(ny) || (DOTS && !flow_full(ny + 1))) break;
                        const uint64_t yd = desc_k(smem_u32(flow_at(ny))), zk = desc_k(smem_u32(flow_at(ny + 1))),
                                       zd = desc_mn(smem_u32(flow_at(ny + 1)), R::HALF);
                        tc_fence_after();
                        mma_ss<false>(tp, xd, yd, I_P);
#pragma unroll
                        for (int ks = 1; ks < 8; ++ks)
                            mma_ss<true>(tp, xd + step_k(ks, 16384), yd + step_k(ks, R::HALF), I_P);
                        if (DOTS) {
                            mma_ss<false>(tp2, wd, zk, I_P);
#pragma unroll
                            for (int ks = 1; ks < 8; ++ks)
                                mma_ss<true>(tp2, wd + step_k(ks, 16384), zk + step_k(ks, R::HALF), I_P);
                        }
                        flow_free(ny);
                        if (sub == 128 / SUB - 1 && j == count - 1) row_free(nx);
                        umma_commit(bar + AB_P_FULL + c);
                        if (!DOTS && !flow_full(ny + 1)) break;
                        if (!(ok = ab.wait(bar + AB_P_READY + c, np & 1))) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < SUB / 16; ++ks)
                            umma_bf16_ts(to, tp + (ks * 16 / (SUB / 2)) * (SUB / 2) + (ks * 16 % (SUB / 2)) / 2,
                                         zd + step_mn(ks), I_O);
                        flow_free(ny + 1);
                    }
                }
                if (!ok) break;
                if (DOTS) row_free(nx + 1);  // the row threads read it before their last P_READY
                umma_commit(bar + AB_O_FULL + c);
                row_skip(nx + XW, nr);
                flow_skip(ny, nf);
                ++q;
            }
        }
    } else if (warp == 3) {
        // an item's prefix sums of the log decays, then its x and w
        int k = 0, n = 0;
        auto rows = [&](const CUtensorMap *m, int h, int tok) {  // 128 tokens in 64-token, 64-channel boxes
            const int s = n % R::ROWS;
            if (!(ok = ok && ab.wait(bar + AB_ROW_EMPTY + s, ((n / R::ROWS) & 1) ^ 1))) return;
            unsigned char *d = row_at(n++);
            mbar_arrive_expect_tx(bar + AB_ROW_FULL + s, R::ROW_SLOT);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    tma_load_3d(d + x * 16384 + t * 8192, m, bar + AB_ROW_FULL + s, 64 * x, h, tok + 64 * t);
        };
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const Item x = item_of<REV>(p, it);
            if (x.tiles == 0) continue;
            constexpr int PER = kLinMaxBlock / 32;
            long long s[PER];
            WarpNan nan;
            warp_decay<PER>(geo, p.log_decay, p.decay, x.blk, x.h, s, nan);
            static_assert(PER == 8, "a lane's bits make a byte");
            const int slot = k % AT_PREFIX;
            ok = __all_sync(0xffffffffu, ab.wait(bar + AB_A_EMPTY + slot, ((k / AT_PREFIX) & 1) ^ 1));
            if (!ok) break;
            float2 *a = reinterpret_cast<float2 *>(sm + AT_A) + slot * (kLinMaxBlock + 2);
            if (lane == 0) a[0] = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < PER; ++u) a[lane * PER + u + 1] = decay_pair(s[u]);
            sm[AT_NAN + slot * (kLinMaxBlock / 8) + lane] = (unsigned char)(REV ? nan.after() : nan.before());
            warp_arrive(bar + AB_A_FULL + slot);
            ++k;
            if (lane == 0)
                for (int t = 0; t < x.tiles; ++t) {
                    rows(&mx, x.h, x.blk.start + 128 * x.tile(t));
                    if (DOTS) rows(&mw, x.h, x.blk.start + 128 * x.tile(t));
                }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        }
    } else {
        const int c = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1, r = (tid - 128) & 127, w = warp & 3;
        constexpr int HSUB = SUB / 2;  // this thread's score columns of a piece: from hf * HSUB
        float *col = reinterpret_cast<float *>(sm + AT_COL) + (warp - 4) * (kLinMaxBlock / 2);
        const uint32_t to = tmem + c * 256 + ((uint32_t)w << 21), tp = to + 128, tp2 = tp + SUB;
        auto wait = [&](uint64_t *b, uint32_t ph) { return ok = __all_sync(0xffffffffu, ab.wait(b, ph)); };
        // row and flow loads and items before this one, tiles and pieces of this context
        int nr = 0, nf = 0, k = 0, q = 0, np = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const Item x = item_of<REV>(p, it);
            if (x.tiles == 0) continue;
            const int slot = k % AT_PREFIX;
            if (!wait(bar + AB_A_FULL + slot, (k / AT_PREFIX) & 1)) break;
            const bool near = (k++ & 1) == c;
            const int nw = nr + (near ? 1 : XW + 1), count = near ? 1 : 2;
            int nz = nf + NS + 1;
            nr += XW * x.tiles;
            nf += NS + YZ * x.tiles;
            if (!near && x.tiles == 1) {
                warp_arrive(bar + AB_A_EMPTY + slot);
                continue;
            }
            const float2 *a = reinterpret_cast<const float2 *>(sm + AT_A) + slot * (kLinMaxBlock + 2);
            const int i0 = 128 * x.tile(near ? 0 : 1), i = i0 + r, len = x.blk.len;
            const float2 ai = a[min(i, len - 1) + 1];
            float f = p.c_state * (REV ? decay_ratio(a[len], ai) : decay_ratio(ai, make_float2(0.f, 0.f)));
            if (sm[AT_NAN + slot * (kLinMaxBlock / 8) + (i >> 3)] >> (i & 7) & 1) f = CUDART_NAN_F;
            // D_ij = row factor x column factor for the columns on the far side of the warp's 32 rows, the
            // decays to and from their edge (both <= 1); only the 32 x 32 piece on the diagonal takes an
            // exponential per element
            const int i32 = i0 + 32 * w;
            const float2 edge = a[REV ? i32 + 32 : i32];
            const float rf = p.c_intra * (REV ? decay_ratio(edge, ai) : decay_ratio(ai, edge));
#pragma unroll
            for (int u = 0; u < kLinMaxBlock / 64; ++u) {  // the u-th 32 of this thread's columns
                const int o = (32 * u / HSUB) * SUB + hf * HSUB + 32 * u % HSUB + lane;
                const int j = 128 * x.tile(o >> 7) + (o & 127);
                col[32 * u + lane] = REV ? (j >= i32 + 32 ? decay_ratio(a[j + 1], edge) : 0.f)
                                         : (j < i32 ? decay_ratio(edge, a[j + 1]) : 0.f);
            }
            __syncwarp();
            const F2 rf2 = f2(rf, rf);
            F2 dots = f2(0.f, 0.f);
            float dot = 0.f, dot_state = 0.f;
            if (!wait(bar + AB_O_IN + c, q & 1) ||
                (DOTS && !wait(bar + AB_ROW_FULL + nw % R::ROWS, (nw / R::ROWS) & 1)))
                break;
            tc_fence_after();
            {
                uint32_t v[2][32];
                tmem_ld32(to + 64 * hf, v[0]);
                tmem_ld32(to + 64 * hf + 32, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    scale32(v[u], f);
                    tmem_st32(to + 64 * hf + 32 * u, v[u]);
                    if (DOTS) {
                        const unsigned char *wt = row_at(nw);
#pragma unroll
                        for (int k8 = 0; k8 < 4; ++k8) {
                            const uint4 g =
                                *reinterpret_cast<const uint4 *>(wt + kmajor_chunk(r, 8 * hf + 4 * u + k8, 128));
                            const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                dot_state += lo_f(gw[e]) * __uint_as_float(v[u][8 * k8 + 2 * e]) +
                                             hi_f(gw[e]) * __uint_as_float(v[u][8 * k8 + 2 * e + 1]);
                        }
                    }
                }
            }
            for (int j = 0; j < count && ok; ++j) {
                const int j0 = 128 * x.tile(j);
                for (int sub = 0; sub < 128 / SUB; ++sub, ++np, nz += 2) {
                    if (!wait(bar + AB_P_FULL + c, np & 1)) break;
                    tc_fence_after();
                    const int left = len - j0 - sub * SUB;
                    if (left < SUB) {  // what lies past the block's end must not meet P's zeros
                        if (!wait(bar + AB_FLOW_FULL + nz % R::FLOW, (nz / R::FLOW) & 1)) break;
                        if (r < SUB && r >= left) {
                            unsigned char *z = flow_at(nz) + hf * R::HALF + r * 128;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4 *>(z + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async();
                    }
#pragma unroll
                    for (int u = 0; u < HSUB / 32; ++u) {
                        uint32_t v[32], v2[32], o[16];
                        const int c0 = hf * HSUB + 32 * u, jc = j0 + sub * SUB + c0;
                        if (REV ? jc < i32 || jc >= len : jc > i32) {  // outside the mask
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = 0u;
                            tmem_st16(tp + hf * HSUB + 16 * u, o);  // inside this thread's own columns
                            continue;
                        }
                        tmem_ld32(tp + c0, v);
                        if (DOTS) tmem_ld32(tp2 + c0, v2);
                        tmem_wait_ld();
                        if (jc != i32 && (!REV || jc + 32 <= len)) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 cf = *reinterpret_cast<const float4 *>(
                                    col + j * 64 + sub * HSUB + 32 * u + e);
                                const F2 y0 = pair_w(v[e], v[e + 1]) * f2(cf.x, cf.y) * rf2;
                                const F2 y1 = pair_w(v[e + 2], v[e + 3]) * f2(cf.z, cf.w) * rf2;
                                if (DOTS) {
                                    dots = fma2(y0, pair_w(v2[e], v2[e + 1]), dots);
                                    dots = fma2(y1, pair_w(v2[e + 2], v2[e + 3]), dots);
                                }
                                o[e / 2] = pack2(y0);
                                o[e / 2 + 1] = pack2(y1);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float y[2];
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const int jj = jc + e + u;
                                    const float2 aj = a[jj + 1];  // entries past the end repeat the total
                                    const float d = REV ? decay_ratio(aj, ai) : decay_ratio(ai, aj);
                                    const bool in = jj < len && (REV ? jj >= i : jj <= i);
                                    y[u] = in ? p.c_intra * d * __uint_as_float(v[e + u]) : 0.f;
                                    if (DOTS && in) dot += y[u] * __uint_as_float(v2[e + u]);
                                }
                                o[e / 2] = pack2(y[0], y[1]);
                            }
                        }
                        tmem_st16(tp + hf * HSUB + 16 * u, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(bar + AB_P_READY + c);
                }
            }
            if (!ok) break;
            warp_arrive(bar + AB_A_EMPTY + slot);
            if (DOTS && i < len) {
                const int64_t at = (int64_t)(x.blk.start + i) * geo.H + x.h;
                p.dot[hf * p.dot_stride + at] = dot + f2_sum(dots) + dot_state;
                if (p.dot_state) p.dot_state[hf * p.dot_stride + at] = dot_state;
            }
            if (!wait(bar + AB_O_FULL + c, q & 1)) break;
            tc_fence_after();
            __nv_bfloat16 *dst = p.out + ((int64_t)(x.blk.start + i) * geo.H + x.h) * D;
            {
                uint32_t v[2][32];
                tmem_ld32(to + 64 * hf, v[0]);
                tmem_ld32(to + 64 * hf + 32, v[1]);
                tmem_wait_ld();
                if (i < len) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = pack2(__uint_as_float(v[u >> 1][16 * (u & 1) + 2 * e]),
                                         __uint_as_float(v[u >> 1][16 * (u & 1) + 2 * e + 1]));
                        st_v8(dst + 64 * hf + 16 * u, o);
                    }
                }
            }
            tc_fence_before();
            warp_arrive(bar + AB_O_EMPTY + c);
            ++q;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    settle(ab);
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ================================================================ outputs, the state carried along
// One item is a segment (a block of any length) and head. The state lives in
// TMEM in fp32 and moves on by 128 tokens at a time, so a segment reads its
// tokens once and no state goes through memory but the segment's first:
//   P = x y^T, masked, times a column factor e^{-L_j}, rounded to bf16 in place;
//   O = x Sb + P z, Sb the state rounded to bf16; row i times e^{L_i} on its way
//   out, which makes D_ij of the column factor and the state's own factor at once
//   (in a chunk that decays by less than 2^40; one that decays by more takes D_ij
//   itself in P, an exponential per element, and has x Sb scaled in between. The
//   factors of up to 2^40 leave 2^87 of fp32's range to scores times z; at 2^80
//   scores and z of 1e5-size inputs overflowed, and the chunks in between cost
//   nothing: 131072 x 32 with a slope per head, 1394-1404 us for both);
//   S <- e^{L_end} S + (w y)^T z, w y in two bf16 parts (16 bits: the state in
//   here only feeds bf16 products).
// In reverse time (REV) the chunks go from the segment's end, the state is the
// gradient after the chunk, and the mask and the decays are mirrored. ST: the
// first state is read transposed. P, Sb and the result are the roundings to
// bf16 (2.35e-3 from 64 bits in the 2-norm, the result's alone 1.66e-3; P or Sb
// in two parts would add 8 of a chunk's 40 tensor-core steps each, and Sb 32 KB
// of shared memory that is not there). Bound by memory in principle (4 x 4096 tokens x 16 heads: 75 us, 268 MB,
// 3.5 TB/s; 131072 x 32: 885 us, 4.3 GB, 4.9 TB/s, 72 % of a copy); a 128-token chunk
// costs 40 tensor-core steps, and two
// loops run from one chunk to the next, each to stay under the time that the
// chunk's 128 KB take: S -> Sb, scale -> MMA -> S, and x Sb -> scale -> P z -> out.
// Everything else of a chunk is done ahead of them: P (two in TMEM), its mask,
// and y's two parts. Instructions are the next bound: twenty-eight warps of
// seven roles share an SM's instruction caches, so the loops are short.
//
// warp 0: TMA of x and y (two tiles of 32 KB each); 1: MMA of P and O; 2: TMA of
// z (one tile, its next one already in L2) and MMA of S; 3: the tables of
// the decays, three chunks ahead; 4-11: rows of P and O, two threads a row; 12-19: y -> two parts
// (the high one in place); 20-27: S -> Sb. Every barrier is waited on by its
// waiters in every phase, and no phase comes twice between two waits (checked
// with a model of the roles).
constexpr int RL_TILE = 128 * D * 2;                 // 32 KB
constexpr int RL_X = 0, RL_Y = 2 * RL_TILE, RL_Z = 4 * RL_TILE, RL_SB = 5 * RL_TILE, RL_LO = 6 * RL_TILE;
constexpr int RL_T = RL_LO + RL_TILE / 2;            // tables of the decays, RL_SLOTS chunks
constexpr int RL_SLOTS = 3;
constexpr int RL_THREADS = 896;
// The decays of one chunk, as its roles use them (made by one warp, ahead of
// them; every role on its own spent 1,700 of a chunk's 8,000 cycles on them).
struct RollTable {
    float row[128];       // row i's factor on its way out (mild) or of the state part, c_state included
    float col[128];       // column factors of P, c_intra / c_state included (mild)
    uint2 weight[128];    // what token s enters the state with, c_roll included: two bf16 parts, each twice
    float mild, total;    // whether the chunk decays by less than 2^kMild; e^{L_end}
    float pad[2];
    float2 a[130];        // prefix sums
};
constexpr float kMild = 40.f;
constexpr int RL_BAR = RL_T + RL_SLOTS * (int)sizeof(RollTable);
enum { RB_FX = 0, RB_EX = 2, RB_FY = 4, RB_EY = 6, RB_PF = 8, RB_YD = 10, RB_PR = 12, RB_FZ = 14, RB_EZ, RB_OIN, RB_OF, RB_OE,
       RB_SR, RB_SS, RB_SBF, RB_KC, RB_LOF, RB_SF, RB_ZZ, RB_AF,
       RB_AE = RB_AF + RL_SLOTS, RB_COUNT = RB_AE + RL_SLOTS };
constexpr int RL_SMEM = RL_BAR + RB_COUNT * 8 + 16 + 1024;
static_assert(RL_SMEM <= 232448, "shared memory of a block");

struct RollTcArgs {
    LinGeom geo;
    const float *log_decay;
    int decay;
    const float *states;  // [block][head][128][128]
    __nv_bfloat16 *out;
    float c_state, c_intra, c_ratio, c_roll;  // c_intra / c_state; what y z products enter the state with
    int items;
};

template <bool REV, bool ST>
__global__ void __launch_bounds__(RL_THREADS, 1)
lin_roll_tc_kernel(RollTcArgs p, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                   const __grid_constant__ CUtensorMap mz) {
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + RL_BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(bar + RB_COUNT);
    const Abort ab{reinterpret_cast<volatile int *>(tm + 1)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LinGeom &geo = p.geo;
    if (tid == 0) {
        *ab.flag = 0;
        for (int i = 0; i < RB_COUNT; ++i) {
            uint32_t n = 1;
            if (i == RB_EZ) n = 2;                                             // both MMA warps
            if (i == RB_PR || i == RB_PR + 1 || i == RB_OE || i == RB_ZZ) n = 8;  // the row warps
            if (i == RB_SR || i == RB_SS || i == RB_KC) n = 8;                 // the state warps; those of y
            if (i >= RB_AE) n = 24;                                            // all three
            mbar_init(bar + i, n);
        }
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;  // S | O | P, two of them
    bool ok = true;
    // g: chunks so far over all items; a walk goes through them in order
    struct Walk {
        LinBlock blk;
        int it, h, n, c;  // item, head, chunks of the item, chunk
    };
    auto enter = [&](Walk &x) {  // the first chunk of the first item from x.it on that has one
        for (; x.it < p.items; x.it += gridDim.x) {
            const int b = geo.by_heads.div(x.it);
            x.h = x.it - b * geo.H;
            x.blk = lin_block(geo, b);
            x.n = (x.blk.len + 127) / 128;
            x.c = 0;
            if (x.n > 0) return;
        }
    };
    auto start = [&]() {
        Walk x;
        x.it = blockIdx.x;
        enter(x);
        return x;
    };
    auto more = [&](const Walk &x) { return x.it < p.items; };
    auto next = [&](Walk &x) {
        if (++x.c < x.n) return;
        x.it += gridDim.x;
        enter(x);
    };
    auto table = [&](int g) { return reinterpret_cast<RollTable *>(sm + RL_T) + g % RL_SLOTS; };
    auto first_token = [&](const Walk &x) { return (REV ? x.n - 1 - x.c : x.c) * 128; };
    auto tile = [&](const CUtensorMap *m, unsigned char *d, uint64_t *full, const Walk &x) {
        mbar_arrive_expect_tx(full, RL_TILE);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                tma_load_3d(d + c * 16384 + t * 8192, m, full, 64 * c, x.h, x.blk.start + first_token(x) + 64 * t);
    };

    if (warp == 0) {
        if (lane == 0) {
            int g = 0;
            for (Walk x = start(); more(x); next(x), ++g) {
                const int s = g & 1;
                const uint32_t ph = ((g >> 1) & 1) ^ 1;
                if (!(ok = ab.wait(bar + RB_EX + s, ph))) break;
                tile(&mx, sm + RL_X + s * RL_TILE, bar + RB_FX + s, x);
                if (!(ok = ab.wait(bar + RB_EY + s, ph))) break;
                tile(&my, sm + RL_Y + s * RL_TILE, bar + RB_FY + s, x);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        tma_prefetch_3d(&mz, 64 * c, x.h, x.blk.start + first_token(x) + 64 * t);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t I_P = idesc_bf16(128, 128, false, false), I_O = idesc_bf16(128, 128, false, true);
            const uint64_t sd = desc_mn(smem_u32(sm + RL_SB), 16384), zd = desc_mn(smem_u32(sm + RL_Z), 16384);
            const uint32_t to = tmem + 128;
            int m = 0;  // chunks whose y makes state
            auto scores = [&](const Walk &x, int g) {
                const int s = g & 1;
                const uint32_t ph = (g >> 1) & 1, tp = tmem + 256 + 128 * s;
                if (!(ok = ab.wait(bar + RB_FX + s, ph) && ab.wait(bar + RB_FY + s, ph))) return;
                tc_fence_after();
                const uint64_t xd = desc_k(smem_u32(sm + RL_X + s * RL_TILE)),
                               yd = desc_k(smem_u32(sm + RL_Y + s * RL_TILE));
                mma_ss<false>(tp, xd, yd, I_P);
#pragma unroll
                for (int ks = 1; ks < 8; ++ks) mma_ss<true>(tp, xd + step_k(ks, 16384), yd + step_k(ks, 16384), I_P);
                umma_commit(bar + RB_PF + s);
                umma_commit(bar + (x.c == x.n - 1 ? RB_EY + s : RB_YD + (m++ & 1)));  // the last chunk's y makes none
            };
            int g = 0;
            Walk ahead = start();
            if (more(ahead)) {
                scores(ahead, 0);
                next(ahead);
            }
            for (Walk x = start(); more(x) && ok; next(x), ++g) {
                const int s = g & 1;
                if (!(ok = ab.wait(bar + RB_SR, g & 1) && ab.wait(bar + RB_OE, (g & 1) ^ 1))) break;
                tc_fence_after();
                const uint64_t xd = desc_k(smem_u32(sm + RL_X + s * RL_TILE));
                mma_ss<false>(to, xd, sd, I_O);
#pragma unroll
                for (int ks = 1; ks < 8; ++ks) mma_ss<true>(to, xd + step_k(ks, 16384), sd + step_mn(ks), I_O);
                umma_commit(bar + RB_OIN);
                umma_commit(bar + RB_SBF);
                umma_commit(bar + RB_EX + s);
                if (more(ahead)) {
                    scores(ahead, g + 1);
                    if (!ok) break;
                    next(ahead);
                }
                if (!(ok = ab.wait(bar + RB_FZ, g & 1) && ab.wait(bar + RB_PR + s, (g >> 1) & 1))) break;
                tc_fence_after();
                const uint32_t tp = tmem + 256 + 128 * s;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)  // each half of P's columns lies in the front of its 64
                    umma_bf16_ts(to, tp + (ks >> 2) * 64 + (ks & 3) * 8, zd + step_mn(ks), I_O);
                umma_commit(bar + RB_OF);
                umma_commit(bar + RB_EZ);
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            constexpr uint32_t I_S = idesc_bf16(128, 128, true, true);
            const uint64_t lo = desc_mn(smem_u32(sm + RL_LO), 8192), zd = desc_mn(smem_u32(sm + RL_Z), 16384);
            int g = 0, m = 0, zz = 0;
            for (Walk x = start(); more(x); next(x), ++g) {
                const int s = g & 1;
                if (!(ok = ab.wait(bar + RB_EZ, (g & 1) ^ 1))) break;  // z's one slot is this warp's to fill
                tile(&mz, sm + RL_Z, bar + RB_FZ, x);
                if (!(ok = ab.wait(bar + RB_FZ, g & 1))) break;
                if (x.c == x.n - 1) {
                    mbar_arrive(bar + RB_EZ);
                    continue;
                }
                // the segment's ragged end (first in reverse): its rows past the end are zeroed first
                if (x.blk.len - first_token(x) < 128 && !(ok = ab.wait(bar + RB_ZZ, zz++ & 1))) break;
                if (!(ok = ab.wait(bar + RB_SS, m & 1))) break;
                const uint64_t yd = desc_mn(smem_u32(sm + RL_Y + s * RL_TILE), 16384);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!(ok = ab.wait(bar + RB_KC, h))) break;
                    tc_fence_after();
                    constexpr uint64_t ROWS64 = 8192 >> 4;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        mma_ss<true>(tmem, lo + step_mn(ks), zd + h * ROWS64 + step_mn(ks), I_S);
                        mma_ss<true>(tmem, yd + h * ROWS64 + step_mn(ks), zd + h * ROWS64 + step_mn(ks), I_S);
                    }
                    umma_commit(bar + RB_LOF);
                }
                if (!ok) break;
                umma_commit(bar + RB_SF);
                umma_commit(bar + RB_EY + s);
                umma_commit(bar + RB_EZ);
                ++m;
            }
        }
    } else if (warp == 3) {
        int g = 0;
        for (Walk x = start(); more(x); next(x), ++g) {
            const int t0 = first_token(x);
            const LinBlock part{x.blk.seq, x.blk.start + t0, min(128, x.blk.len - t0)};
            long long sums[4];
            WarpNan nan;
            const long long all = warp_decay<4>(geo, p.log_decay, p.decay, part, x.h, sums, nan);
            ok = __all_sync(0xffffffffu, ab.wait(bar + RB_AE + g % RL_SLOTS, ((g / RL_SLOTS) & 1) ^ 1));
            if (!ok) break;
            RollTable *t = table(g);
            const float2 zero = make_float2(0.f, 0.f), end = decay_pair(all);
            float2 a[4];  // this lane's tokens 4 lane ..
#pragma unroll
            for (int u = 0; u < 4; ++u) a[u] = decay_pair(sums[u]);
            auto four = [](float *d, float x, float y, float z, float w) {
                *reinterpret_cast<float4 *>(d) = make_float4(x, y, z, w);
            };
            if (lane == 0) {
                t->a[0] = zero;
                t->total = (REV ? nan.first() : nan.last()) ? CUDART_NAN_F : decay_ratio(end, zero);
                t->mild = -(end.x + end.y) < kMild ? 1.f : 0.f;
            }
            float v[4];
            uint32_t wt[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                t->a[4 * lane + u + 1] = a[u];
                const float w = p.c_roll * (REV ? decay_ratio(a[u], zero) : decay_ratio(end, a[u]));
                wt[2 * u] = pack2(w, w);
                const float low = w - lo_f(wt[2 * u]);
                wt[2 * u + 1] = pack2(low, low);
            }
            *reinterpret_cast<uint4 *>(t->weight + 4 * lane) = make_uint4(wt[0], wt[1], wt[2], wt[3]);
            *reinterpret_cast<uint4 *>(t->weight + 4 * lane + 2) = make_uint4(wt[4], wt[5], wt[6], wt[7]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[u] = p.c_state * (REV ? decay_ratio(end, a[u]) : decay_ratio(a[u], zero));
                if ((REV ? nan.after() : nan.before()) >> u & 1) v[u] = CUDART_NAN_F;  // such a chunk is never mild
            }
            four(t->row + 4 * lane, v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = p.c_ratio * (REV ? decay_ratio(a[u], end) : decay_ratio(zero, a[u]));
            four(t->col + 4 * lane, v[0], v[1], v[2], v[3]);
            warp_arrive(bar + RB_AF + g % RL_SLOTS);
        }
    } else if (warp < 12) {  // rows of P and O
        const int hf = (warp - 4) >> 2, w = warp & 3, r = 32 * w + lane, i32 = 32 * w;
        const uint32_t tl = tmem + ((uint32_t)w << 21), to = tl + 128 + 64 * hf;
        auto wait = [&](int b, uint32_t ph) { return ok = __all_sync(0xffffffffu, ab.wait(bar + b, ph)); };
        // P of chunk g to bf16; returns its rows' factor and whether the chunk is mild
        float f = 0.f;
        bool mild = true;
        auto mask = [&](const Walk &x, int g) {
            const int s = g & 1, rows = min(128, x.blk.len - first_token(x));
            const uint32_t tp = tl + 256 + 128 * s + 64 * hf;
            if (!wait(RB_AF + g % RL_SLOTS, (g / RL_SLOTS) & 1)) return;
            const RollTable *t = table(g);
            f = t->row[r];
            mild = t->mild != 0.f;
            if (!wait(RB_PF + s, (g >> 1) & 1)) return;
            tc_fence_after();
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {  // 16 columns: short loops, for the instruction cache
                const int jc = 64 * hf + 16 * u, jb = jc & ~31;  // the 32 columns they belong to
                uint32_t o[8];
                if (REV ? jb < i32 || jc >= rows : jb > i32) {  // outside the mask
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = 0u;
                } else if (mild && (!REV || jc + 16 <= rows)) {
                    uint32_t v[16];
                    tmem_ld16(tp + 16 * u, v);
                    tmem_wait_ld();
                    if (jb == i32) {
                        const int l = lane - (jc & 31);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = (REV ? e >= l : e <= l) ? v[e] : 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 cf = *reinterpret_cast<const float4 *>(t->col + jc + e);
                        o[e / 2] = pack2(pair_w(v[e], v[e + 1]) * f2(cf.x, cf.y));
                        o[e / 2 + 1] = pack2(pair_w(v[e + 2], v[e + 3]) * f2(cf.z, cf.w));
                    }
                } else {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t v[4];
                        tmem_ld4(tp + 16 * u + 4 * q, v);
                        tmem_wait_ld();
                        float y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = jc + 4 * q + e;
                            const float d = mild ? t->col[j]
                                            : p.c_intra * (REV ? decay_ratio(t->a[j + 1], t->a[r + 1])
                                                               : decay_ratio(t->a[r + 1], t->a[j + 1]));
                            const bool in = j < rows && (REV ? j >= r : j <= r);
                            y[e] = in ? d * __uint_as_float(v[e]) : 0.f;
                        }
                        const uint32_t w2[2] = {pack2(y[0], y[1]), pack2(y[2], y[3])};
                        tmem_st2(tp + 8 * u + 2 * q, w2);  // behind the reads
                    }
                    continue;
                }
                tmem_st8(tp + 8 * u, o);
            }
            tmem_wait_st();
            warp_arrive(bar + RB_AE + g % RL_SLOTS);
            if (mild && rows == 128) {  // nothing more to do before P z
                tc_fence_before();
                warp_arrive(bar + RB_PR + s);
            }
        };
        int g = 0;
        Walk x = start(), ahead = x;
        if (more(ahead)) {
            mask(ahead, 0);
            next(ahead);
        }
        for (; more(x) && ok; next(x), ++g) {
            const int t0 = first_token(x), rows = min(128, x.blk.len - t0);
            const float out = mild ? f : 1.f;
            if (!wait(RB_OIN, g & 1)) break;
            if (!mild || rows < 128) {
                tc_fence_after();
                if (!mild) {  // scaled now, not on the way out
#pragma unroll 1
                    for (int u = 0; u < 4; ++u) {
                        uint32_t v[16];
                        tmem_ld16(to + 16 * u, v);
                        tmem_wait_ld();
                        scale16(v, f);  // a reset drops the state
                        tmem_st16(to + 16 * u, v);
                    }
                }
                if (rows < 128) {  // what lies past the segment's end must not meet zeros
                    if (!wait(RB_FZ, g & 1)) break;
                    if (r >= rows) {
                        unsigned char *z = sm + RL_Z + hf * 16384 + r * 128;
#pragma unroll
                        for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4 *>(z + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async();
                    if (x.c < x.n - 1) warp_arrive(bar + RB_ZZ);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar + RB_PR + (g & 1));
            }
            if (more(ahead)) {
                mask(ahead, g + 1);
                if (!ok) break;
                next(ahead);
            }
            if (!wait(RB_OF, g & 1)) break;
            tc_fence_after();
            const F2 out2 = f2(out, out);
            __nv_bfloat16 *dst = p.out + ((int64_t)(x.blk.start + t0 + r) * geo.H + x.h) * D + 64 * hf;
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                uint32_t v[16], o[8];
                tmem_ld16(to + 16 * u, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = pack2(pair_w(v[2 * e], v[2 * e + 1]) * out2);
                if (r < rows) st_v8(dst + 16 * u, o);
            }
            tc_fence_before();
            warp_arrive(bar + RB_OE);
        }
    } else if (warp < 20) {  // y -> two parts
        const int t = tid - 384, c8 = t & 15;
        auto wait = [&](int b, uint32_t ph) { return ok = __all_sync(0xffffffffu, ab.wait(bar + b, ph)); };
        int g = 0, m = 0;
        for (Walk x = start(); more(x); next(x), ++g) {
            const int s = g & 1, rows = min(128, x.blk.len - first_token(x));
            if (!wait(RB_AF + g % RL_SLOTS, (g / RL_SLOTS) & 1)) break;
            if (x.c < x.n - 1) {
                const uint2 *weight = table(g)->weight;
                unsigned char *yt = sm + RL_Y + s * RL_TILE + kmajor_chunk(t >> 4, c8, 128),
                              *lt = sm + RL_LO + kmajor_chunk(t >> 4, c8, 64);
                if (!wait(RB_YD + (m & 1), (m >> 1) & 1)) break;
                // (a loop that stays one: the roles' code together has to fit the instruction cache)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {  // 64 tokens: the high part in place, the low one to its buffer
                    // the products with the low buffer's last contents are done
                    if (2 * m + h > 0 && !wait(RB_LOF, (h + 1) & 1)) break;
#pragma unroll 1
                    for (int i = 0; i < 4; i += 2) {
                        uint4 v[2];
                        uint2 f[2];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int row = 64 * h + 16 * (i + q) + (t >> 4);
                            v[q] = *reinterpret_cast<const uint4 *>(yt + h * 8192 + (i + q) * 2048);
                            f[q] = weight[row];
                            if (row >= rows) v[q] = make_uint4(0u, 0u, 0u, 0u);  // past the segment's end
                        }
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t in[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
                            uint32_t hi[4], l[4];
                            // two channels an instruction: hi = y w_h rounded, what that left off, plus y w_l
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                hi[e] = bf2_mul(in[e], f[q].x);
                                l[e] = bf2_fma(in[e], f[q].y, bf2_fma(in[e], f[q].x, hi[e] ^ 0x80008000u));
                            }
                            *reinterpret_cast<uint4 *>(yt + h * 8192 + (i + q) * 2048) =
                                make_uint4(hi[0], hi[1], hi[2], hi[3]);
                            *reinterpret_cast<uint4 *>(lt + (i + q) * 2048) = make_uint4(l[0], l[1], l[2], l[3]);
                        }
                    }
                    fence_proxy_async();
                    warp_arrive(bar + RB_KC);
                }
                if (!ok) break;
                ++m;
            }
            warp_arrive(bar + RB_AE + g % RL_SLOTS);
        }
    } else {  // the state before a chunk: to bf16 for O, and on by the chunk's decay for S
        const int hf = (warp - 20) >> 2, w = warp & 3, r = 32 * w + lane;
        const uint32_t ts = tmem + ((uint32_t)w << 21) + 64 * hf;
        auto wait = [&](int b, uint32_t ph) { return ok = __all_sync(0xffffffffu, ab.wait(bar + b, ph)); };
        int g = 0, m = 0;
        for (Walk x = start(); more(x); next(x), ++g) {
            const bool last = x.c == x.n - 1;
            if (!wait(RB_AF + g % RL_SLOTS, (g / RL_SLOTS) & 1)) break;
            const float fs = table(g)->total;
            warp_arrive(bar + RB_AE + g % RL_SLOTS);
            if (x.c > 0 && !wait(RB_SF, (m - 1) & 1)) break;
            if (g > 0 && !wait(RB_SBF, (g - 1) & 1)) break;
            tc_fence_after();
            const float *S0 = p.states + (int64_t)x.it * D * D;
            unsigned char *sb = sm + RL_SB + hf * 16384 + r * 128;
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                uint32_t v[16];
                if (x.c > 0) {
                    tmem_ld16(ts + 16 * u, v);
                    tmem_wait_ld();
                } else if (ST) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__ldg(S0 + (64 * hf + 16 * u + e) * D + r));
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 q = __ldg(reinterpret_cast<const float4 *>(S0 + r * D + 64 * hf + 16 * u + e));
                        v[e] = __float_as_uint(q.x), v[e + 1] = __float_as_uint(q.y);
                        v[e + 2] = __float_as_uint(q.z), v[e + 3] = __float_as_uint(q.w);
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = pack2(pair_w(v[8 * k + 2 * e], v[8 * k + 2 * e + 1]));
                    *reinterpret_cast<uint4 *>(sb + (((2 * u + k) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                if (!last) {
                    scale16(v, fs);
                    tmem_st16(ts + 16 * u, v);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            if (!last) {
                warp_arrive(bar + RB_SS);
                ++m;
            }
            fence_proxy_async();
            warp_arrive(bar + RB_SR);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    settle(ab);
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}
// [tokens][H][128] bf16 with a token stride, boxes of 64 channels x 1 head x 64 tokens.
bool token_map(CUtensorMap *m, const void *ptr, int64_t stride, int H, int64_t tokens) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {D, (cuuint64_t)H, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {D * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, 64}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// [rows][128] bf16 states, boxes of 64 columns x 128 rows.
bool state_map(CUtensorMap *m, const void *ptr, int64_t rows) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {D, (cuuint64_t)rows}, strides[1] = {D * 2};
    cuuint32_t box[2] = {64, 128}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
int sm_count() {
    static int n = [] {
        int dev = 0, v = 152;
        if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        return v;
    }();
    return n;
}

#define KDA_TRY(x)                        \
    do {                                  \
        const cudaError_t e_ = (x);       \
        if (e_ != cudaSuccess) return e_; \
    } while (0)

}  // namespace

cudaError_t launch_state_tc(const LinGeom &geo, bool rev, const void *x, int64_t xs, const void *y, int64_t ys,
                            int64_t tokens, const float *log_decay, int decay, float *out, float *total,
                            float *total_rev, Launches &l) {
    CUtensorMap mx, my;
    if (!token_map(&mx, x, xs, geo.H, tokens) || !token_map(&my, y, ys, geo.H, tokens)) return cudaErrorInvalidValue;
    StateTcArgs p{geo, log_decay, decay, out, total, total_rev, geo.nblocks * geo.H};
    auto k = rev ? lin_state_tc_kernel<true> : lin_state_tc_kernel<false>;
    static std::atomic<uint64_t> allowed[2];
    KDA_TRY(allow_smem(k, ST_SMEM, allowed[rev]));
    return l.whole(k, min(p.items, sm_count()), ST_THREADS, ST_SMEM, p, mx, my);
}

cudaError_t launch_scan_tc(const LinGeom &geo, bool rev, const float *own, const float *total,
                           const float *s0, float *sT, float c, void *out, int64_t part_stride, const void *other,
                           float *inner, Launches &l) {
    auto k = rev ? lin_scan_tc_kernel<true> : lin_scan_tc_kernel<false>;
    return l.whole(k, (unsigned)((int64_t)geo.N * geo.H * (D * D / 4 / SC_THREADS)), SC_THREADS, 0, geo, own, total, s0, sT,
                   c, (__nv_bfloat16 *)out, part_stride, (const __nv_bfloat16 *)other, inner);
}

cudaError_t launch_roll_tc(const RollTc &a, Launches &l) {
    const LinGeom &geo = a.geo;
    CUtensorMap mx, my, mz;
    if (!token_map(&mx, a.x, a.x_stride, geo.H, a.tokens) || !token_map(&my, a.y, a.y_stride, geo.H, a.tokens) ||
        !token_map(&mz, a.z, a.z_stride, geo.H, a.tokens))
        return cudaErrorInvalidValue;
    const float ratio = a.c_intra == a.c_state ? 1.f : a.c_intra / a.c_state;  // c_state is c_intra or 1
    RollTcArgs p{geo, a.log_decay, a.decay, a.states, (__nv_bfloat16 *)a.out, a.c_state, a.c_intra, ratio, a.c_roll,
                 geo.nblocks * geo.H};
    auto k = a.rev ? (a.state_t ? lin_roll_tc_kernel<true, true> : lin_roll_tc_kernel<true, false>)
                   : (a.state_t ? lin_roll_tc_kernel<false, true> : lin_roll_tc_kernel<false, false>);
    static std::atomic<uint64_t> allowed[4];
    KDA_TRY(allow_smem(k, RL_SMEM, allowed[a.rev * 2 + a.state_t]));
    return l.whole(k, min(p.items, sm_count()), RL_THREADS, RL_SMEM, p, mx, my, mz);
}

cudaError_t launch_attend_tc(const AttendTc &a, Launches &l) {
    const LinGeom &geo = a.geo;
    const bool dots = a.dot != nullptr;
    const int64_t rows = (int64_t)geo.nblocks * geo.H * D;
    if (geo.sb != kLinMaxBlock || rows * 3 > INT32_MAX) return cudaErrorInvalidConfiguration;
    CUtensorMap mx, my, mz, ms, mw;
    if (!token_map(&mx, a.x, a.x_stride, geo.H, a.tokens) || !token_map(&my, a.y, a.y_stride, geo.H, a.tokens) ||
        !token_map(&mz, a.z, a.z_stride, geo.H, a.tokens) || !state_map(&ms, a.states, dots ? 3 * rows : rows))
        return cudaErrorInvalidValue;
    mw = mx;
    if (dots && !token_map(&mw, a.w, a.w_stride, geo.H, a.tokens)) return cudaErrorInvalidValue;
    AttendTcArgs p{geo, a.log_decay, a.decay, (__nv_bfloat16 *)a.out, a.c_state, a.c_intra, a.dot, a.dot_state,
                   a.tokens * geo.H, (int)rows, geo.nblocks * geo.H};
    if (dots != a.state_t) return cudaErrorInvalidValue;  // what the backward asks for: dq, dk with dots, dv without
    auto k = !a.rev ? lin_attend_tc_kernel<false, true, true>
             : dots ? lin_attend_tc_kernel<true, true, true>
                    : lin_attend_tc_kernel<true, false, false>;
    static std::atomic<uint64_t> allowed[4];
    KDA_TRY(allow_smem(k, AT_SMEM, allowed[a.rev * 2 + dots]));
    return l.whole(k, min(p.items, sm_count()), AT_THREADS, AT_SMEM, p, mx, my, mz, ms, mw);
}

cudaError_t read_linear_error(int *out, bool reset) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_lin_error, sizeof(int));
    if (e != cudaSuccess) return e;
    *out = v;
    if (reset && v) {
        const int z = 0;
        e = cudaMemcpyToSymbol(g_lin_error, &z, sizeof(int));
    }
    return e;
}

}  // namespace kda
