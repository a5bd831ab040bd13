// Attention with a sliding window and sinks on the tensor cores of sm_103a, bf16:
// tcgen05.mma, TMEM and TMA. The formulas stand in kda_window.cu.
//
// The kernels are persistent, one CTA per SM; roles are warps that meet at
// mbarriers, and every role walks the same items and steps. Every wait is
// bounded: one that runs out sets the device error word and the CTA's abort flag,
// every role leaves its loop, and the CTA ends normally. A waiter of a barrier waits
// for each of its phases in turn, since a wait knows a phase by its parity alone. One
// does not: the forward's rows wait for PV only when they rescale O, and skip phases.
// There the order of the products stands in: S of step n, which they have waited
// for, was issued behind PV of step n - 2, whose commit arrives before its own, and PV
// of step n - 1 is the last one issued until their weights of step n are there: the
// barrier is in its phase n - 1 or has just ended it. Another order of the products
// would want a wait for every phase.
#include <cuda.h>
#include <math_constants.h>

#include "kda_tc_roles.cuh"
#include "kda_window_tc.cuh"

namespace kda {
namespace {

__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// The same value in every lane, and known as such to the compiler: a role's loop counters and descriptors then
// stay in the registers that the tensor core's instructions take.
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// MMAs, and the commits behind them, by the lane that holds `e` (see elected), without a branch around them.
__device__ __forceinline__ uint32_t elected() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_ss_if(uint32_t e, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(e)
        : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t e, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(e)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t e, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(e)
        : "memory");
}

// Rows first .. 127 of a K-major (or, the same layout, MN-major) tile of D
// channels and 128 rows become zeros. A whole warp; the tile has arrived.
template <int D> __device__ __forceinline__ void zero_rows(unsigned char *tile, int first, int rows) {
    for (int i = threadIdx.x & 31; i < (rows - first) * (D / 8); i += 32) {
        const int r = first + i / (D / 8), c = i % (D / 8);
        *reinterpret_cast<uint4 *>(tile + kmajor_chunk(r, c, 128)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async();
    __syncwarp();
}

// Stores 64 bf16 (32 words) of each of a warp's 32 rows, lane l's being those of row l.
// A lane that stored its own row would touch a line of its own with every store
// (4000 cycles for a tile of 128 x 128); four lanes exchange their 32-byte pieces
// first, so that they store 128 bytes of one row at a time. Rows from `rows` on are
// left out.
__device__ __forceinline__ void store_rows(__nv_bfloat16 *first, int64_t stride, int rows, uint32_t (&w)[4][8]) {
    const int lane = threadIdx.x & 31;
    const bool odd = lane & 1, high = lane & 2;
#pragma unroll
    for (int a = 0; a < 4; a += 2)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[a][e] : w[a + 1][e], 1);
            if (odd) w[a][e] = got;
            else w[a + 1][e] = got;
        }
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[a][e] : w[a + 2][e], 2);
            if (high) w[a][e] = got;
            else w[a + 2][e] = got;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (lane & ~3) + i;
        if (row < rows) st_v8(first + row * stride + 16 * (lane & 3), w[i]);
    }
}

// ================================================================ forward
// An item is 256 queries of one head, two contexts w of 128 rows. A context goes
// through its keys 64 at a time (first, where there are far pairs, the sinks alone,
// their number rounded up to 16), with two score buffers in turn:
//   S = Q_w K^T (TMEM), P = 2^{c S - m} as bf16 over S's own columns, O_w += P V (TMEM).
// The MMAs of a context go S(0), S(1), PV(0), S(2), PV(1), S(3) ..., so the scores
// of a step are there when the softmax of the one before is through, and the
// softmax never waits for the tensor core (with one buffer of 128 keys it waited
// for PV and the next S: 175 us for 4 x 4096 tokens x 16 heads, window 1024).
// S of step n being complete says that PV of step n - 2 is. The softmax rescales O
// only when a row's maximum has grown by more than 2^8 since the last time, and
// then waits for PV of the step before: the weights are taken against the older
// maximum until then, up to 2^8, which fp32 sums and bf16 weights carry as well.
// That case takes 128 us as calls one after the other (940 TFLOP/s, 48 % of the measured
// rate of a large product), 65,531 packed tokens of 32 heads over 8 key heads, window
// 2048, 1.47 ms with the write into the cache (1.17 PFLOP/s, 60 %): bound by the rows, a
// step's softmax in turn with its products, and O of an item, which they store while the
// next one's scores wait.
//
// warp 0: TMA, 128 keys a tile; 1, 2: MMA of the contexts (and zeros behind a
// sequence's end); 4-7, 8-11: the rows of the contexts, a thread each.
constexpr int FW_THREADS = 384;
template <int D> struct Fw {
    static constexpr int TILE = 128 * D * 2;
    static constexpr int ATOM = 128 * 128;               // 64 channels of 128 rows
    static constexpr int STAGES = D == 128 ? 5 : 8;      // K and V in turn
    static constexpr int KV = 2 * TILE;
    static constexpr int BAR = KV + STAGES * TILE;
    // S, P: of context w and buffer b at 2 w + b; PV, OF (the last PV), OE: of context w
    static constexpr int B_QF = 0, B_QE = 1, B_SF = 2, B_PF = 6, B_PV = 10, B_OF = 12, B_OE = 14, B_KF = 16,
                         B_KE = B_KF + STAGES, COUNT = B_KE + STAGES;
    static constexpr int SMEM = BAR + COUNT * 8 + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory of a block");
};

struct FwArgs {
    WinGeom geo;
    __nv_bfloat16 *o;
    float *lse;
    float scale, c2;  // c2: scale in powers of two
    int items;
};

struct FwItem {
    int start, len, f, rows, h, hk;  // f: the 256 queries' first one in its sequence
    int far, kw;                     // whether there is a tile of the sinks, and its keys
    int nf0, tiles;                  // the first near tile of 128 keys; tiles, the sinks' one counted
    __device__ __forceinline__ FwItem(const WinGeom &g, int it) {
        const int t = g.by_hq.div(it);
        h = it - t * g.hq;
        hk = h / g.group;
        const WinTile x = win_tile(g, t);
        start = x.start, len = x.len, f = x.first;
        rows = min(kWinTile, len - f);
        const int last = f + rows - 1;
        far = g.sinks > 0 && last >= g.window;
        kw = far ? (min(g.sinks, last - g.window + 1) + 15) & ~15 : 0;
        nf0 = max(0, f - g.window + 1) >> 7;
        tiles = rows > 0 ? far + (f >> 7) - nf0 + 1 + (rows > 128) : 0;
    }
    __device__ __forceinline__ int key0(int tile) const { return tile < far ? 0 : (nf0 + tile - far) * 128; }
    __device__ __forceinline__ int keys(int tile) const { return tile < far ? kw : 128; }
};
// A context's tiles among the item's: the sinks' one if it sees any behind its window, then near ones.
struct FwContext {
    int i0, first, last;  // its first query; its near tiles
    bool far;
    int tiles;
    __device__ __forceinline__ FwContext(const WinGeom &g, const FwItem &x, int w) {
        i0 = x.f + 128 * w;
        far = x.far && min(i0 + 127, x.len - 1) >= g.window;
        first = x.far + (max(0, i0 - g.window + 1) >> 7) - x.nf0;
        last = x.far + (i0 >> 7) - x.nf0;
        tiles = x.rows > 128 * w ? far + last - first + 1 : 0;
    }
    __device__ __forceinline__ int tile(int n) const { return far ? (n == 0 ? 0 : first + n - 1) : first + n; }
};

template <int D>
__global__ void __launch_bounds__(FW_THREADS, 1)
win_forward_tc_kernel(FwArgs p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mk16,
                      const __grid_constant__ CUtensorMap mv16) {
    using F = Fw<D>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + F::BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(bar + F::COUNT);
    const Abort ab{reinterpret_cast<volatile int *>(tm + 1)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WinGeom &geo = p.geo;
    if (tid == 0) {
        *ab.flag = 0;
        for (int i = 0; i < F::COUNT; ++i)
            mbar_init(bar + i, (i >= F::B_PF && i < F::B_PV) || (i >= F::B_OE && i < F::B_KF) ? 4
                               : i == F::B_QE || i >= F::B_KE                                 ? 2
                                                                                              : 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;  // S of context 0, two of 64 columns | of context 1 | O_0 | O_1
    const uint32_t bars = smem_u32(bar);
    auto wait = [&](int b, int phase) { return ab.wait_warp(bars + 8 * b, phase & 1); };
    bool ok = true;

    if (warp == 0) {
        // A whole warp waits, one lane copies: with one lane in a wait and the others past it the warp is woken by
        // the wait's time limit alone, microseconds late.
        int s = 0, round = 1, q = 0;  // the next stage and its phase, items so far
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            if (x.tiles == 0) continue;
            if (!(ok = wait(F::B_QE, ++q))) break;
            if (lane == 0) {
                const int contexts = x.rows > 128 ? 2 : 1;
                mbar_arrive_expect_tx(bar + F::B_QF, contexts * F::TILE);
                for (int w = 0; w < contexts; ++w)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(sm + w * F::TILE + c * F::ATOM, &mq, bar + F::B_QF, 64 * c, x.h, x.start + x.f + 128 * w);
            }
            __syncwarp();
            for (int j = 0; j < 2 * x.tiles; ++j) {  // K and V of a tile
                if (!(ok = wait(F::B_KE + s, round))) break;
                if (lane == 0) {
                    const int tile = j >> 1, row = x.start + x.key0(tile);
                    const bool is_v = j & 1;
                    unsigned char *d = sm + F::KV + s * F::TILE;
                    uint64_t *full = bar + F::B_KF + s;
                    mbar_arrive_expect_tx(full, x.keys(tile) * D * 2);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        if (tile >= x.far) tma_load_3d(d + c * F::ATOM, is_v ? &mv : &mk, full, 64 * c, x.hk, row);
                        else
                            for (int r = 0; r < x.kw; r += 16)
                                tma_load_3d(d + c * F::ATOM + r * 128, is_v ? &mv16 : &mk16, full, 64 * c, x.hk, row + r);
                    }
                }
                __syncwarp();
                if (++s == F::STAGES) s = 0, round ^= 1;
            }
        }
    } else if (warp < 3) {
        // A context's products. One thread issues them and is held up until the tensor core takes them, so what it
        // does in between is time without a product of this context: hence two warps, and as few steps in their
        // loops as can be.
        const int w = uni(warp - 1);
        const uint32_t e = elected();
        const uint32_t base = uni(tmem), kv = uni(smem_u32(sm + F::KV)), bb = uni(bars);
        const uint32_t ts = base + 128 * w, to = base + 256 + 128 * w;
        constexpr uint32_t I_O = idesc_bf16(128, D, false, true), I_S = idesc_bf16(128, 64, false, false);
        const uint64_t qd = desc_k(kv - F::KV + w * F::TILE), kd = desc_k(kv), vd = desc_mn(kv, F::ATOM);
        int s = 0, round = 0;            // the next stage and its phase
        int q = 0, oi = 0, pn[2] = {0, 0};  // items so far, phases of O and of the halves' P
        auto on = [&](int b, int phase) { return ab.wait_warp(bb + 8 * b, phase & 1); };
        auto next = [&]() {
            if (++s == F::STAGES) s = 0, round ^= 1;
        };
        // the scores of a half of the tile whose K is in stage s
        auto scores = [&](int u, uint32_t idesc) {
            const uint64_t b = kd + ((s * F::TILE + u * 8192) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_ss_if(e, ts + 64 * u, qd + step_k(ks, F::ATOM), b + step_k(ks, F::ATOM), idesc, ks > 0);
            commit_if(e, bb + 8 * (F::B_SF + 2 * w + u));
        };
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            if (x.tiles == 0) continue;
            const FwContext y(geo, x, w);
            const int tiles = uni(x.tiles), mine = uni(y.tiles), kw = uni(x.kw), far = uni(y.far), others = uni(x.far) - far,
                      lead = uni(y.first) - uni(x.far),  // near tiles in front that the other context alone has use for
                      len = uni(x.len), behind = uni(x.len - x.key0(y.first));  // tokens; from its first near tile on
            const int far0 = far ? min(kw, 64) : 64, far1 = far ? kw - 64 : 64;  // keys of its first tile's halves
            if (!(ok = on(F::B_QF, q++))) break;
            // K and V of tiles that it has none for
            auto pass = [&](int count) {
                for (int i = 0; i < 2 * count && ok; ++i) {
                    if (!(ok = on(F::B_KF + s, round))) break;
                    commit_if(e, bb + 8 * (F::B_KE + s));
                    next();
                }
            };
            if (mine == 0) {
                commit_if(e, bb + 8 * F::B_QE);
                pass(tiles);
                continue;
            }
            pass(others + (far ? 0 : lead));
            // K of the first tile
            if (!ok || !(ok = on(F::B_KF + s, round))) break;
            tc_fence_after();
            scores(0, far ? idesc_bf16(128, far0, false, false) : I_S);
            if (far1 > 0) scores(1, far ? idesc_bf16(128, far1, false, false) : I_S);
            commit_if(e, bb + 8 * (F::B_KE + s));
            next();
            if (mine == 1) commit_if(e, bb + 8 * F::B_QE);
            for (int n = 0; n < mine; ++n) {
                const bool sinks = far && n == 0, more = n + 1 < mine;
                const int sv = s;
                if (!(ok = on(F::B_KF + s, round))) break;
                const int rows = sinks ? len : behind - 128 * (n - far);  // up to the sequence's end
                if (rows < (sinks ? kw : 128)) zero_rows<D>(sm + F::KV + sv * F::TILE, rows, sinks ? kw : 128);
                next();
                const uint64_t vb = vd + ((sv * F::TILE) >> 4);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int keys = !sinks ? 64 : u ? far1 : far0;
                    if (keys > 0) {
                        if (!(ok = on(F::B_PF + 2 * w + u, pn[u]++))) break;
                        if (n == 0 && u == 0 && !(ok = on(F::B_OE + w, ++oi))) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_ts_if(keys > 16 * ks ? e : 0u, to, ts + 64 * u + ks * 8, vb + ((u * 8192) >> 4) + step_mn(ks),
                                      I_O, n > 0 || u > 0 || ks > 0);
                        commit_if(e, bb + 8 * (F::B_PV + w));
                    }
                    if (u == 1) {
                        commit_if(e, bb + 8 * (F::B_KE + sv));
                        if (!more) commit_if(e, bb + 8 * (F::B_OF + w));
                    }
                    if (more) {
                        if (u == 0) {
                            if (sinks) pass(lead);
                            if (!ok || !(ok = on(F::B_KF + s, round))) break;
                            tc_fence_after();
                        }
                        scores(u, I_S);
                    }
                }
                if (!ok) break;
                if (more) {
                    commit_if(e, bb + 8 * (F::B_KE + s));
                    next();
                    if (n + 2 == mine) commit_if(e, bb + 8 * F::B_QE);  // the last scores are on their way
                }
            }
            if (!ok) break;
            pass(tiles - others - lead - mine);
        }
    } else if (warp >= 4) {
        const int w = (warp - 4) >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, ts0 = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
        int sn[2] = {0, 0}, of = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            const FwContext y(geo, x, w);
            if (y.tiles == 0) continue;
            const int i = y.i0 + row;
            float m = -CUDART_INF_F;
            F2 l = f2(0.f, 0.f), l1 = l;
#pragma unroll 1
            for (int h = 0; h < 2 * y.tiles; ++h) {
                const int u = h & 1;
                const bool far = y.far && h < 2;
                if (far && 64 * u >= x.kw) continue;
                const uint32_t ts = ts0 + 64 * u;
                if (!(ok = wait(F::B_SF + 2 * w + u, u ? sn[1] : sn[0]))) break;
                if (u) ++sn[1];
                else ++sn[0];
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(ts, s[0]);
                tmem_ld32(ts + 32, s[1]);
                tmem_wait_ld();
                constexpr uint32_t NONE = 0xff800000u;  // -inf
                const int k0 = (far ? 0 : x.key0(y.tile(h >> 1))) + 64 * u;
                if (far || k0 + 63 > y.i0) {  // some row does not see the last keys (the sinks' columns may be stale)
                    const int hi = (far ? min(geo.sinks, i - geo.window + 1) - 1 : i) - k0;
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c >> 5][c & 31] = c > hi ? NONE : s[c >> 5][c & 31];
                }
                if (!far && k0 < y.i0 + 128 - geo.window) {  // or the first ones
                    const int lo = i - geo.window + 1 - k0;
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c >> 5][c & 31] = c < lo ? NONE : s[c >> 5][c & 31];
                }
                float t[4] = {m, m, m, m};
#pragma unroll
                for (int c = 0; c < 64; c += 8)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        t[v] = max3(t[v], __uint_as_float(s[c >> 5][(c & 31) + v]), __uint_as_float(s[c >> 5][(c & 31) + v + 4]));
                const float top = fmaxf(max3(t[0], t[1], t[2]), t[3]);
                const bool grow = (top - m) * p.c2 > 8.f;  // also when the row sees its first number
                if (h > 0 && __any_sync(0xffffffffu, grow)) {
                    // PV of the step before the last one is complete, so this waits for that of the last one and no
                    // other phase
                    if (!(ok = wait(F::B_PV + w, sn[0] + sn[1]))) break;
                    tc_fence_after();
                    const float f = grow ? exp2_approx((m - top) * p.c2) : 1.f;
                    const F2 ff = f2(f, f);
                    l = l * ff, l1 = l1 * ff;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a, b;
                            f2_get(pair_w(o[e], o[e + 1]) * ff, a, b);
                            o[e] = __float_as_uint(a), o[e + 1] = __float_as_uint(b);
                        }
                        tmem_st32(to + c, o);
                    }
                }
                if (grow) m = top;
                const float off = m == -CUDART_INF_F ? 0.f : -m * p.c2;
                const F2 c2 = f2(p.c2, p.c2), off2 = f2(off, off);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float u0, v0, u1, v1;
                        f2_get(fma2(pair_w(s[c][e], s[c][e + 1]), c2, off2), u0, v0);
                        f2_get(fma2(pair_w(s[c][e + 2], s[c][e + 3]), c2, off2), u1, v1);
                        const F2 a = f2(exp2_approx(u0), exp2_approx(v0)), b = f2(exp2_approx(u1), exp2_approx(v1));
                        l = l + a, l1 = l1 + b;
                        o[e / 2] = pack2(a), o[e / 2 + 1] = pack2(b);
                    }
                    tmem_st16(ts + 16 * c, o);  // over columns that have been read
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar + F::B_PF + 2 * w + u);
            }
            if (!ok) break;
            if (!(ok = wait(F::B_OF + w, of++))) break;
            tc_fence_after();
            const float sum = f2_sum(l + l1), f = 1.f / sum;
            const bool there = i < x.len;
            const int64_t at = (int64_t)(x.start + i) * geo.hq + x.h;
            const F2 ff = f2(f, f);
            const int r0 = y.i0 + (warp & 3) * 32;  // the warp's first row
            __nv_bfloat16 *dst = p.o + ((int64_t)(x.start + r0) * geo.hq + x.h) * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
                uint32_t o[2][32], r[4][8];
                tmem_ld32(to + c, o[0]);
                tmem_ld32(to + c + 32, o[1]);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        r[u][e] = pack2(pair_w(o[u >> 1][16 * (u & 1) + 2 * e], o[u >> 1][16 * (u & 1) + 2 * e + 1]) * ff);
                store_rows(dst + c, (int64_t)geo.hq * D, x.len - r0, r);
            }
            tc_fence_before();
            warp_arrive(bar + F::B_OE + w);
            if (there && p.lse) p.lse[at] = fmaf(m, p.scale, logf(sum));
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

// ================================================================ backward: D
// D_i = sum_j p_ij dp_ij / sum_j p_ij, from both products of rows again, and not
// do . o from the stored o: ds = p (dp - D) is far smaller than dp where one weight is
// close to one, as sinks' are, and the rounding of a bf16 o would be seen in dq and dk (1e-2 of
// them at a weight of 0.8, 2e-1 at 0.999). The weights' sum takes out the rounding of lse,
// so that the ds of a row add up to nothing.
//
// An item is 256 queries of one head, two contexts of 128 as in the forward; a step is
// 128 keys (or the sinks), whose K and V both contexts use, so that one's products run
// while the other's rows are at their weights. The rows also write lse by head, in powers
// of two: a tile of queries is a stretch of memory then. 4 x 4096 x 16, window 1024:
// 124 us. A context's step of 3160 cycles (d = 128) is a chain: 1100 until the rows have
// read S and dP, 350 until the next products are issued, 1650 of products, the other
// context's among them; d = 64 takes 2250, all of them the rows', whose instructions
// wait for one another. Two threads to a row changed nothing; steps of 64 keys, read
// sooner, took 140 to 160 us, since their products take as long as those of 128.
//
// warp 0: TMA; 1, 2: MMA of the contexts; 4-7, 8-11: their rows, a thread each.
template <int D> struct Bd {
    static constexpr int TILE = 128 * D * 2, ATOM = 128 * 128;
    static constexpr int STAGES = D == 128 ? 3 : 8;                    // K and V in turn
    static constexpr int RING = 4 * TILE, BAR = RING + STAGES * TILE;  // in front of it Q, Q, dO, dO
    // QF, OF, QE: the item's Q and dO; of context w: PF, L (a step's S and dP there, in registers)
    static constexpr int B_QF = 0, B_OF = 1, B_QE = 2, B_PF = 3, B_L = 5, B_KF = 7, B_KE = B_KF + STAGES, COUNT = B_KE + STAGES;
    static constexpr int SMEM = BAR + COUNT * 8 + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory of a block");
};

struct BdArgs {
    WinGeom geo;
    const float *lse;     // [tokens][hq]
    float *lse2, *delta;  // [hq][tokens]: lse in powers of two, D
    float c2;
    int items;
};

template <int D>
__global__ void __launch_bounds__(FW_THREADS, 1)
win_delta_tc_kernel(BdArgs p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                    const __grid_constant__ CUtensorMap mk16, const __grid_constant__ CUtensorMap mv16) {
    using B = Bd<D>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + B::BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(bar + B::COUNT);
    const Abort ab{reinterpret_cast<volatile int *>(tm + 1)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WinGeom &geo = p.geo;
    let_next_start();
    if (tid == 0) {
        *ab.flag = 0;
        for (int i = 0; i < B::COUNT; ++i)
            mbar_init(bar + i, i >= B::B_L && i < B::B_KF ? 4 : i == B::B_QE || i >= B::B_KE ? 2 : 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;  // S and dP of context 0 | of context 1
    const uint32_t bars = smem_u32(bar);
    auto wait = [&](int b, int phase) { return ab.wait_warp(bars + 8 * b, phase & 1); };
    bool ok = true;

    if (warp == 0) {
        int s = 0, round = 1, q = 0;  // the next stage and its phase, items so far
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            if (x.tiles == 0) continue;
            if (!(ok = wait(B::B_QE, ++q))) break;
            const int contexts = x.rows > 128 ? 2 : 1;
            auto queries = [&](int at, const CUtensorMap *m, int full) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar + full, contexts * B::TILE);
                    for (int w = 0; w < contexts; ++w)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(sm + (at + w) * B::TILE + c * B::ATOM, m, bar + full, 64 * c, x.h, x.start + x.f + 128 * w);
                }
                __syncwarp();
            };
            queries(0, &mq, B::B_QF);
            for (int j = 0; j < 2 * x.tiles; ++j) {  // K and V of a tile
                if (!(ok = wait(B::B_KE + s, round))) break;
                if (lane == 0) {
                    const int tile = j >> 1, row = x.start + x.key0(tile);
                    const bool is_v = j & 1;
                    unsigned char *d = sm + B::RING + s * B::TILE;
                    uint64_t *full = bar + B::B_KF + s;
                    mbar_arrive_expect_tx(full, x.keys(tile) * D * 2);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        if (tile >= x.far) tma_load_3d(d + c * B::ATOM, is_v ? &mv : &mk, full, 64 * c, x.hk, row);
                        else
                            for (int r = 0; r < x.kw; r += 16)
                                tma_load_3d(d + c * B::ATOM + r * 128, is_v ? &mv16 : &mk16, full, 64 * c, x.hk, row + r);
                    }
                }
                __syncwarp();
                if (j == 0) queries(2, &mo, B::B_OF);
                if (++s == B::STAGES) s = 0, round ^= 1;
            }
            if (ok && lane == 0 && it + gridDim.x < p.items) {  // the next item's, into L2
                const FwItem y(geo, it + gridDim.x);
                for (int w = 0; w < (y.tiles == 0 ? 0 : y.rows > 128 ? 2 : 1); ++w)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        tma_prefetch_3d(&mq, 64 * c, y.h, y.start + y.f + 128 * w);
                        tma_prefetch_3d(&mo, 64 * c, y.h, y.start + y.f + 128 * w);
                    }
            }
            __syncwarp();
        }
    } else if (warp < 3) {
        const int w = uni(warp - 1);
        const uint32_t e = elected(), base = uni(tmem) + 256 * w, sb = uni(smem_u32(sm)), bb = uni(bars);
        constexpr uint32_t I_S = idesc_bf16(128, 128, false, false);
        const uint64_t qd = desc_k(sb + w * B::TILE), od = desc_k(sb + (2 + w) * B::TILE), kd = desc_k(sb + B::RING);
        auto on = [&](int b, int phase) { return ab.wait_warp(bb + 8 * b, phase & 1); };
        int s = 0, round = 0, q = 0, n = 0;  // the next stage and its phase; items, steps of this context so far
        auto next = [&]() {
            if (++s == B::STAGES) s = 0, round ^= 1;
        };
        // S and dP of a tile, one behind the other: what this warp does in between is time without a product
        auto step = [&](uint32_t idesc) {
            const int sk = s;
            if (!(ok = on(B::B_KF + s, round))) return;
            next();
            const int sv = s;
            if (!(ok = on(B::B_KF + s, round))) return;
            next();
            const uint64_t kb = kd + ((sk * B::TILE) >> 4), vb = kd + ((sv * B::TILE) >> 4);
            if (!(ok = on(B::B_L + w, ++n))) return;  // the step before is in registers
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_ss_if(e, base, qd + step_k(ks, B::ATOM), kb + step_k(ks, B::ATOM), idesc, ks > 0);
            commit_if(e, bb + 8 * (B::B_KE + sk));
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_ss_if(e, base + 128, od + step_k(ks, B::ATOM), vb + step_k(ks, B::ATOM), idesc, ks > 0);
            commit_if(e, bb + 8 * (B::B_PF + w));
            commit_if(e, bb + 8 * (B::B_KE + sv));
        };
        auto pass = [&](int tiles) {  // that the other context alone has use for
            for (int i = 0; i < 2 * tiles && ok; ++i) {
                if (!(ok = on(B::B_KF + s, round))) break;
                commit_if(e, bb + 8 * (B::B_KE + s));
                next();
            }
        };
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            if (x.tiles == 0) continue;
            const FwContext y(geo, x, w);
            const int mine = uni(y.tiles), far = mine > 0 ? uni(y.far) : 0, near = mine - far, others = uni(x.far) - far,
                      lead = mine > 0 ? uni(y.first - x.far) : 0, behind = uni(x.tiles) - mine - others - lead;
            const uint32_t i0 = far ? idesc_bf16(128, uni(x.kw), false, false) : I_S;
            if (!(ok = on(B::B_QF, q) && on(B::B_OF, q))) break;
            ++q;
            pass(others);
            if (ok && far) step(i0);
            pass(lead);
            for (int j = 0; j < near && ok; ++j) step(I_S);
            pass(behind);
            if (!ok) break;
            commit_if(e, bb + 8 * B::B_QE);
        }
    } else if (warp >= 4) {
        const int w = (warp - 4) >> 2, row = tid & 127;
        const uint32_t ts = tmem + ((uint32_t)(warp & 3) << 21) + 256 * w, td = ts + 128;
        const F2 c2 = f2(p.c2, p.c2);
        int n = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            const FwContext y(geo, x, w);
            if (y.tiles == 0) continue;
            const int i = y.i0 + row;
            const bool there = i < x.len;
            const float lse2 = there ? p.lse[(int64_t)(x.start + i) * geo.hq + x.h] * 1.4426950408889634f : CUDART_INF_F;
            const F2 l2 = f2(-lse2, -lse2);
            F2 sum = f2(0.f, 0.f), sum1 = sum, all = sum, all1 = sum;
            int key0 = (x.nf0 + y.first - x.far) * 128;  // of the next near tile
            for (int j = 0; j < y.tiles; ++j) {
                const bool far = y.far && j == 0;
                if (!(ok = wait(B::B_PF + w, n++))) break;
                tc_fence_after();
                const int halves = far && x.kw <= 64 ? 1 : 2;
#pragma unroll 1
                for (int u = 0; u < halves; ++u) {
                    uint32_t v[2][32], d[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_ld32(ts + 64 * u + 32 * c, v[c]);
                        tmem_ld32(td + 64 * u + 32 * c, d[c]);
                    }
                    tmem_wait_ld();
                    if (u + 1 == halves) {
                        tc_fence_before();
                        warp_arrive(bar + B::B_L + w);
                    }
                    const int k0 = (far ? 0 : key0) + 64 * u;
                    constexpr uint32_t NONE = 0xff800000u;  // -inf
                    // what a row does not see has no weight, whatever its dP is (the sinks' columns may be stale)
                    if (far || k0 + 63 > y.i0) {
                        const int hi = (far ? min(geo.sinks, i - geo.window + 1) - 1 : i) - k0;
#pragma unroll
                        for (int c = 0; c < 64; ++c) {
                            v[c >> 5][c & 31] = c > hi ? NONE : v[c >> 5][c & 31];
                            d[c >> 5][c & 31] = c > hi ? 0u : d[c >> 5][c & 31];
                        }
                    }
                    if (!far && k0 < y.i0 + 128 - geo.window) {
                        const int lo = i - geo.window + 1 - k0;
#pragma unroll
                        for (int c = 0; c < 64; ++c) {
                            v[c >> 5][c & 31] = c < lo ? NONE : v[c >> 5][c & 31];
                            d[c >> 5][c & 31] = c < lo ? 0u : d[c >> 5][c & 31];
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            float a, b;
                            f2_get(fma2(pair_w(v[c][e], v[c][e + 1]), c2, l2), a, b);
                            const F2 w0 = f2(exp2_approx(a), exp2_approx(b));
                            f2_get(fma2(pair_w(v[c][e + 2], v[c][e + 3]), c2, l2), a, b);
                            const F2 w1 = f2(exp2_approx(a), exp2_approx(b));
                            sum = fma2(w0, pair_w(d[c][e], d[c][e + 1]), sum);
                            sum1 = fma2(w1, pair_w(d[c][e + 2], d[c][e + 3]), sum1);
                            all = all + w0, all1 = all1 + w1;
                        }
                }
                if (!far) key0 += 128;
            }
            if (!ok) break;
            if (there) {
                const int64_t at = (int64_t)x.h * geo.tokens + x.start + i;
                p.delta[at] = f2_sum(sum + sum1) / f2_sum(all + all1);
                p.lse2[at] = lse2;
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

// ================================================================ backward: dk, dv
// An item is 128 keys of one key head; a step is 128 queries of one of its query
// heads. Transposed scores, so that keys are the rows:
//   S^T = K Q^T,  dP^T = V dO^T                      (TMEM)
//   P^T = 2^{c S^T - lse}, to shared memory;  dS^T = P^T (dP^T - D), over dP^T   (bf16)
//   dV += P^T dO,  dK += dS^T Q                      (TMEM, all steps of the item)
// so each tile of Q and dO serves as an operand both ways round and nothing is
// transposed in memory. One warp issues S(n+1), as soon as S(n) is in registers, and
// dV(n), another dK(n) and dP(n+1): S of a step is there when dS of the one before
// is made (with P^T over S^T it had to wait for dV, and a step took 2800 cycles of
// which P and dS are 1850 and the four products 2060). 4 x 4096 x 16, window 1024:
// 244 us, the tensor cores busy half of it; 2900 cycles a step, 4700 more an item. S(n+1)
// held back behind dP(n), or four more warps a half, changed nothing.
// Queries behind the sequence's end count as zeros with an infinite lse.
// The far pairs are items of their own: the sinks against kWinFarQueries queries,
// whose sums are parts that win_far_sum_kernel adds up.
//
// warp 0: TMA; 1: MMA of S and dV; 2: of dP and dK; 3: lse and D of the queries;
// 4-11: P and dS, two threads a key, 64 queries each (the halves of a bf16 row of dS
// lie in the front of their 64 columns, so that no thread writes over what another
// one reads).
constexpr int BW_THREADS = 384;
template <int D> struct Bw {
    static constexpr int TILE = 128 * D * 2, ATOM = 128 * 128;
    static constexpr int QS = 2, OS = 2;                  // stages of Q and dO
    static constexpr int RING_Q = 2 * TILE, RING_O = RING_Q + QS * TILE;
    static constexpr int P = RING_O + OS * TILE;          // P^T, 128 keys of 128 queries
    static constexpr int VEC = P + 2 * ATOM;              // 128 of lse, of two steps, and 128 of D
    static constexpr int BAR = VEC + 1536;
    static constexpr int B_KF = 0, B_KE = 1, B_SF = 2, B_SL = 3, B_PR = 4, B_PE = 5, B_DF = 6, B_DR = 7, B_AF = 8, B_AE = 9,
                         B_QF = 10, B_QE = B_QF + QS, B_OF = B_QE + QS, B_OE = B_OF + OS, B_LF = B_OE + OS,
                         B_XF = B_LF + 2, B_LE = B_LF + 3, B_XE = B_LF + 5, COUNT = B_LF + 6;  // LF, LE: of two buffers
    static constexpr int SMEM = BAR + COUNT * 8 + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory of a block");
};

struct BwArgs {
    WinGeom geo;
    __nv_bfloat16 *dq, *dk, *dv;
    const float *lse2, *delta;  // [hq][tokens]: lse in powers of two, D
    float *part, *near;         // gradients of the sinks, see win_far_sum_kernel
    float scale, c2;
    int fars, items;            // items of far pairs come first
};

struct DkvItem {
    int seq, start, len, first, j0, hk, q0, nq, steps;  // q0: the first tile of 128 queries, nq: their number
    bool far;
    __device__ __forceinline__ DkvItem(const WinGeom &g, int it, int fars) {
        far = it < fars;
        if (!far) it -= fars;
        const int t = g.by_hk.div(it);
        hk = it - t * g.hk;
        const WinTile x = win_tile(g, far ? t : t >> 1);
        seq = x.seq, start = x.start, len = x.len, first = x.first;
        if (far) {
            j0 = 0;
            const int end = min(len, x.first + kWinFarQueries), from = max(x.first, g.window);
            q0 = from >> 7;
            nq = x.first % kWinFarQueries == 0 && from < end ? ((end - 1) >> 7) - q0 + 1 : 0;
        } else {
            j0 = x.first + (t & 1) * 128;
            q0 = j0 >> 7;
            nq = j0 < len ? (int)min((int64_t)len - 1, (int64_t)j0 + 126 + g.window) / 128 - q0 + 1 : 0;
        }
        steps = nq * g.group;
    }
};
struct DkvStep {
    int h, qt;
    __device__ __forceinline__ DkvStep(const WinGeom &g, const DkvItem &x) : h(x.hk * g.group), qt(x.q0) {}
    __device__ __forceinline__ void next(const DkvItem &x) {
        if (++qt == x.q0 + x.nq) qt = x.q0, ++h;
    }
};

template <int D>
__global__ void __launch_bounds__(BW_THREADS, 1)
win_dkv_tc_kernel(BwArgs p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    using B = Bw<D>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + B::BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(bar + B::COUNT);
    const Abort ab{reinterpret_cast<volatile int *>(tm + 1)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WinGeom &geo = p.geo;
    if (tid == 0) {
        *ab.flag = 0;
        for (int i = 0; i < B::COUNT; ++i)
            mbar_init(bar + i, i == B::B_SL || i == B::B_PR || i == B::B_DR || i == B::B_AE || i >= B::B_LE ? 8
                               : i == B::B_KE || i == B::B_AF || (i >= B::B_OE && i < B::B_OE + B::OS) ? 2
                                                                                                       : 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    await_previous();
    let_next_start();  // after the wait: the next kernel reads what this one waited for
    const uint32_t tmem = *tm, t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;
    const uint32_t bars = smem_u32(bar);
    auto wait = [&](int b, int phase) { return ab.wait_warp(bars + 8 * b, phase & 1); };
    bool ok = true;

    if (warp == 0) {
        int n = 0, k = 0;  // steps, items so far
        auto tile = [&](unsigned char *d, const CUtensorMap *m, int full, int h, int row) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c) tma_load_3d(d + c * B::ATOM, m, bar + full, 64 * c, h, row);
        };
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const DkvItem x(geo, it, p.fars);
            if (x.steps == 0) continue;
            if (!(ok = wait(B::B_KE, k + 1))) break;
            ++k;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar + B::B_KF, 2 * B::TILE);
                tile(sm, &mk, B::B_KF, x.hk, x.start + x.j0);
                tile(sm + B::TILE, &mv, B::B_KF, x.hk, x.start + x.j0);
                if (it + gridDim.x < p.items) {  // the next item's, into L2
                    const DkvItem y(geo, it + gridDim.x, p.fars);
                    if (y.steps > 0)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            tma_prefetch_3d(&mk, 64 * c, y.hk, y.start + y.j0);
                            tma_prefetch_3d(&mv, 64 * c, y.hk, y.start + y.j0);
                        }
                }
            }
            __syncwarp();
            DkvStep st(geo, x);
            for (int j = 0; j < x.steps; ++j, ++n, st.next(x)) {
                const int qs = n % B::QS, os = n % B::OS, row = x.start + st.qt * 128;
                if (!(ok = wait(B::B_QE + qs, n / B::QS + 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar + B::B_QF + qs, B::TILE);
                    tile(sm + B::RING_Q + qs * B::TILE, &mq, B::B_QF + qs, st.h, row);
                }
                __syncwarp();
                if (!(ok = wait(B::B_OE + os, n / B::OS + 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar + B::B_OF + os, B::TILE);
                    tile(sm + B::RING_O + os * B::TILE, &mo, B::B_OF + os, st.h, row);
                }
                __syncwarp();
            }
        }
    } else if (warp < 3) {
        // first: S, a step ahead, and dV; second: dK, and dP a step ahead
        const int w = uni(warp - 1);
        const uint32_t e = elected(), base = uni(tmem), sb = uni(smem_u32(sm)), bb = uni(bars);
        constexpr uint32_t I_S = idesc_bf16(128, 128, false, false), I_G = idesc_bf16(128, D, false, true);
        const uint32_t t_p = base + 128 * w, t_g = base + 256 + 128 * w;
        const uint64_t ad = desc_k(sb + w * B::TILE), pd = desc_k(sb + B::P);
        const uint64_t rk = desc_k(sb + (w ? B::RING_O : B::RING_Q)), rm = desc_mn(sb + (w ? B::RING_Q : B::RING_O), B::ATOM);
        auto on = [&](int b, int phase) { return ab.wait_warp(bb + 8 * b, phase & 1); };
        // Two stages a ring, step n's in n & 1. Rows behind the sequence's end may hold anything.
        auto arrived = [&](int full, int ring, int n, int rows) {
            if (!(ok = on(full + (n & 1), n >> 1))) return;
            if (rows < 128) zero_rows<D>(sm + ring + (n & 1) * B::TILE, rows, 128);
            tc_fence_after();
        };
        auto product = [&](int n) {
            const uint64_t b = rk + (((n & 1) * B::TILE) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_ss_if(e, t_p, ad + step_k(ks, B::ATOM), b + step_k(ks, B::ATOM), I_S, ks > 0);
            commit_if(e, bb + 8 * (w ? B::B_DF : B::B_SF));
            if (w) commit_if(e, bb + 8 * (B::B_OE + (n & 1)));
        };
        int k = 0, n = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const DkvItem x(geo, it, p.fars);
            const int steps = uni(x.steps), nq = uni(x.nq), rows0 = uni(x.len - x.q0 * 128);
            if (steps == 0) continue;
            if (!(ok = on(B::B_KF, k))) break;
            int qt = 0;  // of the step ahead
            auto ahead = [&](int n) {
                arrived(w ? B::B_OF : B::B_QF, w ? B::RING_O : B::RING_Q, n, rows0 - 128 * qt);
                // the step's lse, or D, is there before its product is, for those who wait for that
                if (ok && (ok = w ? on(B::B_XF, n) : on(B::B_LF + (n & 1), n >> 1))) product(n);
            };
            ahead(n);
            if (!ok) break;
            if (steps == 1) commit_if(e, bb + 8 * B::B_KE);
            for (int j = 0; j < steps; ++j, ++n) {
                const int rows = rows0 - 128 * qt;
                if (++qt == nq) qt = 0;
                const bool more = j + 1 < steps;
                if (w == 0) {
                    if (more) {
                        if (!(ok = on(B::B_SL, n))) break;
                        ahead(n + 1);
                        if (!ok) break;
                        if (j + 2 == steps) commit_if(e, bb + 8 * B::B_KE);
                    }
                    arrived(B::B_OF, B::RING_O, n, rows);
                    if (!ok || !(ok = on(B::B_PR, n))) break;
                } else {
                    if (!(ok = on(B::B_QF + (n & 1), n >> 1) && on(B::B_DR, n))) break;
                }
                if (j == 0 && !(ok = on(B::B_AE, k + 1))) break;
                tc_fence_after();
                const uint64_t b = rm + (((n & 1) * B::TILE) >> 4);
                if (w == 0) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ss_if(e, t_g, pd + step_k(ks, B::ATOM), b + step_mn(ks), I_G, j > 0 || ks > 0);
                    commit_if(e, bb + 8 * B::B_PE);
                    commit_if(e, bb + 8 * (B::B_OE + (n & 1)));
                } else {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ts_if(e, t_g, t_p + (ks >> 2) * 64 + (ks & 3) * 8, b + step_mn(ks), I_G, j > 0 || ks > 0);
                    commit_if(e, bb + 8 * (B::B_QE + (n & 1)));  // S has used Q long before
                    if (more) {
                        ahead(n + 1);
                        if (!ok) break;
                        if (j + 2 == steps) commit_if(e, bb + 8 * B::B_KE);
                    }
                }
                if (!more) commit_if(e, bb + 8 * B::B_AF);
            }
            ++k;
        }
    } else if (warp == 3) {
        // four queries a lane; the next step's are on their way while this one's wait to be let in
        int n = 0;
        float *vec = reinterpret_cast<float *>(sm + B::VEC);
        float l[4], d[4];
        auto load = [&](const DkvItem &x, const DkvStep &st) {
            const int i0 = st.qt * 128 + 4 * lane;
            const int64_t at = (int64_t)st.h * geo.tokens + x.start + i0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool there = i0 + e < x.len;
                l[e] = there ? p.lse2[at + e] : CUDART_INF_F;  // of kernels that ran a moment ago: not read-only
                d[e] = there ? p.delta[at + e] : 0.f;
            }
        };
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const DkvItem x(geo, it, p.fars);
            if (x.steps == 0) continue;
            DkvStep st(geo, x);
            load(x, st);
            for (int j = 0; j < x.steps; ++j, ++n) {
                const float4 lv = make_float4(-l[0], -l[1], -l[2], -l[3]), dv = make_float4(-d[0], -d[1], -d[2], -d[3]);
                st.next(x);
                if (j + 1 < x.steps) load(x, st);
                if (!(ok = wait(B::B_LE + (n & 1), (n >> 1) + 1))) break;
                reinterpret_cast<float4 *>(vec)[32 * (n & 1) + lane] = lv;
                warp_arrive(bar + B::B_LF + (n & 1));
                if (!(ok = wait(B::B_XE, n + 1))) break;
                reinterpret_cast<float4 *>(vec + 256)[lane] = dv;
                warp_arrive(bar + B::B_XF);
            }
        }
    } else {
        const int half = (warp - 4) >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, ts = t_s + lanes + 64 * half, td = t_dp + lanes + 64 * half;
        const float *vec = reinterpret_cast<const float *>(sm + B::VEC) + 64 * half;
        unsigned char *pt = sm + B::P + half * B::ATOM + (row >> 3) * 1024 + (row & 7) * 128;  // see kmajor_chunk
        const F2 c2 = f2(p.c2, p.c2);
        int n = 0, k = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const DkvItem x(geo, it, p.fars);
            if (x.steps == 0) continue;
            const int j = x.j0 + row;  // this thread's key
            DkvStep st(geo, x);
#pragma unroll 1
            for (int u = 0; u < x.steps; ++u, ++n, st.next(x)) {
                const int i0 = st.qt * 128;
                const int d0 = j - i0 - 64 * half;  // the half's column of the key's own token
                float pr[64];
                if (!(ok = wait(B::B_SF, n))) break;  // and lse
                tc_fence_after();
                uint32_t v[2][32];
                tmem_ld32(ts, v[0]);
                tmem_ld32(ts + 32, v[1]);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(bar + B::B_SL);
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(vec + 128 * (n & 1) + c);
                    const uint32_t *y = v[c >> 5] + (c & 31);
                    float a, b;
                    f2_get(fma2(pair_w(y[0], y[1]), c2, F2{l.x}), a, b);
                    pr[c] = exp2_approx(a), pr[c + 1] = exp2_approx(b);
                    f2_get(fma2(pair_w(y[2], y[3]), c2, F2{l.y}), a, b);
                    pr[c + 2] = exp2_approx(a), pr[c + 3] = exp2_approx(b);
                }
                // far: the queries behind the window see the sinks; near: from the key's own token to the window's end
                const bool edge = x.far ? true : i0 < x.j0 + 127;
                if (edge) {
                    const int lo = !x.far ? d0 : j < geo.sinks ? d0 + geo.window : 64;
#pragma unroll
                    for (int c = 0; c < 64; ++c) pr[c] = c < lo ? 0.f : pr[c];
                }
                if (!x.far && i0 + 127 - x.j0 >= geo.window) {
                    const int hi = d0 + geo.window - 1;
#pragma unroll
                    for (int c = 0; c < 64; ++c) pr[c] = c > hi ? 0.f : pr[c];
                }
                if (!(ok = wait(B::B_PE, n + 1))) break;  // dV of the step before has read P
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4 *>(pt + ((c ^ (row & 7)) << 4)) =
                        make_uint4(pack2(pr[8 * c], pr[8 * c + 1]), pack2(pr[8 * c + 2], pr[8 * c + 3]),
                                   pack2(pr[8 * c + 4], pr[8 * c + 5]), pack2(pr[8 * c + 6], pr[8 * c + 7]));
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {  // LE first: no warp then comes to LE of the next step before all have come to this one's
                    mbar_arrive(bar + B::B_LE + (n & 1));
                    mbar_arrive(bar + B::B_PR);
                }
                // a token that sees itself alone has no ds
                if (i0 == 0 && half == 0) pr[0] = 0.f;
                if (geo.window == 1 && geo.sinks == 0) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) pr[e] = 0.f;
                }
                if (!(ok = wait(B::B_DF, n))) break;  // and D
                tc_fence_after();
                tmem_ld32(td, v[0]);
                tmem_ld32(td + 32, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 d = *reinterpret_cast<const ulonglong2 *>(vec + 256 + 32 * c + e);
                        const float *w = pr + 32 * c + e;
                        o[e / 2] = pack2((pair_w(v[c][e], v[c][e + 1]) + F2{d.x}) * f2(w[0], w[1]));
                        o[e / 2 + 1] = pack2((pair_w(v[c][e + 2], v[c][e + 3]) + F2{d.y}) * f2(w[2], w[3]));
                    }
                    tmem_st16(td + 16 * c, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar + B::B_XE);
                    mbar_arrive(bar + B::B_DR);
                }
            }
            if (!ok) break;
            if (!(ok = wait(B::B_AF, k++))) break;
            tc_fence_after();
            // half 0: dv, half 1: dk. Of sinks that far queries see too, in fp32, for the sum of both.
            const bool there = j < x.len && (!x.far || j < geo.sinks),
                       sink = x.far || (j < geo.sinks && x.len > geo.window);
            const uint32_t src = (half ? t_dk : t_dv) + lanes;
            const float f = half ? p.scale : 1.f;
            __nv_bfloat16 *dst = (half ? p.dk : p.dv) + ((int64_t)(x.start + x.j0 + (warp & 3) * 32) * geo.hk + x.hk) * D;
            float *sum = nullptr;
            if (sink && there) {
                const int64_t r = x.far ? win_far_row(geo, x.seq, x.start, x.first, kWinFarQueries) : win_near_row(geo, x.seq);
                sum = (x.far ? p.part : p.near) + (((r + j) * geo.hk + x.hk) * 2 + (half ? 0 : 1)) * D;
            }
            const F2 ff = f2(f, f);
            const int r0 = x.j0 + (warp & 3) * 32;  // the warp's first row
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
                uint32_t v[2][32], r[4][8];
                tmem_ld32(src + c, v[0]);
                tmem_ld32(src + c + 32, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const F2 g = pair_w(v[u >> 1][16 * (u & 1) + 2 * e], v[u >> 1][16 * (u & 1) + 2 * e + 1]) * ff;
                        if (sum) *reinterpret_cast<unsigned long long *>(sum + c + 16 * u + 2 * e) = g.v;
                        r[u][e] = pack2(g);
                    }
                // a sink's row is written here too, and again when its sums are added up
                if (!x.far) store_rows(dst + c, (int64_t)geo.hk * D, x.len - r0, r);
            }
            tc_fence_before();
            warp_arrive(bar + B::B_AE);
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

// ================================================================ backward: dq
// An item is 128 queries of one head; a step is 128 keys (or the sinks, as in the
// forward):
//   S = Q K^T (two of it),  dP = dO V^T,  dS = P (dP - D) over S (bf16),  dQ += dS K
// One warp issues S(n+1), dQ(n), another dP(n+1), as soon as dP(n) is in registers:
// dS of a step is made while the tensor core does dQ of the step before and S and
// dP of the one behind. K is kept for two steps (S and dQ), V for one. 174 us for the
// same gradients, 2000 cycles a step of which the products are 1545.
//
// warp 0: TMA; 1: MMA of S and dQ; 2: of dP; 4-11: dS, two threads a query, 64 keys each.
template <int D> struct Bq {
    static constexpr int TILE = 128 * D * 2, ATOM = 128 * 128;
    static constexpr int KS = 3, VS = 2;                  // stages of K and V
    static constexpr int RING_K = 2 * TILE, RING_V = RING_K + KS * TILE, BAR = RING_V + VS * TILE;
    // QF, QE: the item's Q and dO; SF: of two buffers; DF, DL: dP there, in registers; DR: of two buffers
    static constexpr int B_QF = 0, B_QE = 1, B_SF = 2, B_DF = 4, B_DL = 5, B_DR = 6, B_AF = 8, B_AE = 9, B_KF = 10,
                         B_KE = B_KF + KS, B_VF = B_KE + KS, B_VE = B_VF + VS, COUNT = B_VE + VS;
    static constexpr int SMEM = BAR + COUNT * 8 + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory of a block");
};

template <int D>
__global__ void __launch_bounds__(BW_THREADS, 1)
win_dq_tc_kernel(BwArgs p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                 const __grid_constant__ CUtensorMap mk16, const __grid_constant__ CUtensorMap mv16) {
    using B = Bq<D>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + B::BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(bar + B::COUNT);
    const Abort ab{reinterpret_cast<volatile int *>(tm + 1)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WinGeom &geo = p.geo;
    if (tid == 0) {
        *ab.flag = 0;
        for (int i = 0; i < B::COUNT; ++i) mbar_init(bar + i, (i >= B::B_DL && i < B::B_AF) || i == B::B_AE ? 8 : i == B::B_QE ? 2 : 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm, t_dp = tmem + 256, t_dq = tmem + 384;  // S, S, dP, dQ
    bool ok = true;
    // A warp may be through with dS of a step before another is with the step before: dP of it waits for
    // nobody's dS. So there are two barriers of dS, in turn.
    auto made = [](int n) { return B::B_DR + (n & 1); };
    struct Item {
        int start, len, i0, h, hk, far, kw, kt0, steps;
        __device__ __forceinline__ Item(const WinGeom &g, int it) {
            const int t = g.by_hq.div(it);
            h = it - t * g.hq;
            hk = h / g.group;
            const WinTile x = win_tile(g, t >> 1);
            start = x.start, len = x.len, i0 = x.first + (t & 1) * 128;
            const int last = min(i0 + 128, len) - 1;
            far = g.sinks > 0 && last >= g.window;
            kw = far ? (min(g.sinks, last - g.window + 1) + 15) & ~15 : 0;
            kt0 = max(0, i0 - g.window + 1) >> 7;
            steps = i0 < len ? far + (i0 >> 7) - kt0 + 1 : 0;
        }
        __device__ __forceinline__ bool is_far(int j) const { return j < far; }
        __device__ __forceinline__ int key0(int j) const { return is_far(j) ? 0 : (kt0 + j - far) * 128; }
        __device__ __forceinline__ int keys(int j) const { return is_far(j) ? kw : 128; }
    };

    const uint32_t bars = smem_u32(bar);
    auto wait = [&](int b, int phase) { return ab.wait_warp(bars + 8 * b, phase & 1); };

    if (warp == 0) {
        int n = 0, k = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const Item x(geo, it);
            if (x.steps == 0) continue;
            if (!(ok = wait(B::B_QE, k + 1))) break;
            ++k;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar + B::B_QF, 2 * B::TILE);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    tma_load_3d(sm + c * B::ATOM, &mq, bar + B::B_QF, 64 * c, x.h, x.start + x.i0);
                    tma_load_3d(sm + B::TILE + c * B::ATOM, &mo, bar + B::B_QF, 64 * c, x.h, x.start + x.i0);
                }
                if (it + gridDim.x < p.items) {  // the next item's, into L2
                    const Item y(geo, it + gridDim.x);
                    if (y.steps > 0)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            tma_prefetch_3d(&mq, 64 * c, y.h, y.start + y.i0);
                            tma_prefetch_3d(&mo, 64 * c, y.h, y.start + y.i0);
                        }
                }
            }
            __syncwarp();
            auto keys = [&](const CUtensorMap *whole, const CUtensorMap *few, unsigned char *d, int full, int j) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar + full, x.keys(j) * D * 2);
                    const int row = x.start + x.key0(j);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        if (!x.is_far(j)) tma_load_3d(d + c * B::ATOM, whole, bar + full, 64 * c, x.hk, row);
                        else
                            for (int r = 0; r < x.kw; r += 16)
                                tma_load_3d(d + c * B::ATOM + r * 128, few, bar + full, 64 * c, x.hk, row + r);
                    }
                }
                __syncwarp();
            };
            for (int j = 0; j < x.steps; ++j, ++n) {
                const int ks = n % B::KS, vs = n % B::VS;
                if (!(ok = wait(B::B_KE + ks, n / B::KS + 1))) break;
                keys(&mk, &mk16, sm + B::RING_K + ks * B::TILE, B::B_KF + ks, j);
                if (!(ok = wait(B::B_VE + vs, n / B::VS + 1))) break;
                keys(&mv, &mv16, sm + B::RING_V + vs * B::TILE, B::B_VF + vs, j);
            }
        }
    } else if (warp < 3) {
        // the first: S a step ahead and dQ; the second: dP. Both see every phase of the keys' ring that they read.
        const int w = uni(warp - 1);
        const uint32_t e = elected(), base = uni(tmem), sb = uni(smem_u32(sm)), bb = uni(bars);
        constexpr uint32_t I_G = idesc_bf16(128, D, false, true), I_S = idesc_bf16(128, 128, false, false);
        const uint64_t ad = desc_k(sb + w * B::TILE), kd = desc_k(sb + (w ? B::RING_V : B::RING_K)),
                       km = desc_mn(sb + B::RING_K, B::ATOM);
        auto on = [&](int b, int phase) { return ab.wait_warp(bb + 8 * b, phase & 1); };
        int n = 0, k = 0, s = 0, round = 0;  // s: the stage of step n + 1's K, or V
        auto product = [&](uint32_t d, uint32_t idesc, int full) {
            const uint64_t b = kd + ((s * B::TILE) >> 4);
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_ss_if(e, d, ad + step_k(ks, B::ATOM), b + step_k(ks, B::ATOM), idesc, ks > 0);
            commit_if(e, bb + 8 * full);
        };
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const Item x(geo, it);
            const int steps = uni(x.steps), far = uni(x.far), kw = uni(x.kw), len = uni(x.len), behind = len - uni(x.kt0) * 128;
            if (steps == 0) continue;
            if (!(ok = on(B::B_QF, k))) break;
            const uint32_t i0 = far ? idesc_bf16(128, kw, false, false) : I_S;  // of the first step
            if (w == 0) {
                // keys behind the sequence's end are masked, but their rows of K meet the zeros of dS
                auto scores = [&](int j) {
                    if (!(ok = on(B::B_KF + s, round))) return;
                    const int rows = j < far ? len : behind - 128 * (j - far), keys = j < far ? kw : 128;
                    if (rows < keys) zero_rows<D>(sm + B::RING_K + s * B::TILE, rows, keys);
                    product(base + 128 * ((n + (j > 0)) & 1), j == 0 ? i0 : I_S, B::B_SF + ((n + (j > 0)) & 1));
                    if (j + 1 == steps) commit_if(e, bb + 8 * B::B_QE);  // Q has been used for the last time
                    if (++s == B::KS) s = 0, round ^= 1;
                };
                int sd = s;  // the stage of step n's K
                scores(0);
                for (int j = 0; j < steps && ok; ++j, ++n) {
                    if (j + 1 < steps) {
                        scores(j + 1);
                        if (!ok) break;
                    }
                    if (!(ok = on(made(n), n >> 1))) break;
                    if (j == 0 && !(ok = on(B::B_AE, k + 1))) break;
                    tc_fence_after();
                    const uint32_t a = base + 128 * (n & 1);
                    const uint64_t b = km + ((sd * B::TILE) >> 4);
                    const int keys = j < far ? kw : 128;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ts_if(keys > 16 * ks ? e : 0u, base + 384, a + (ks >> 2) * 64 + (ks & 3) * 8, b + step_mn(ks), I_G,
                                  j > 0 || ks > 0);
                    commit_if(e, bb + 8 * (B::B_KE + sd));
                    if (++sd == B::KS) sd = 0;
                    if (j + 1 == steps) commit_if(e, bb + 8 * B::B_AF);
                }
            } else {
                for (int j = 0; j < steps; ++j, ++n) {
                    if (!(ok = on(B::B_VF + s, round))) break;
                    if (n > 0 && !(ok = on(B::B_DL, n - 1))) break;  // dP of the step before is in registers
                    product(base + 256, j == 0 ? i0 : I_S, B::B_DF);
                    commit_if(e, bb + 8 * (B::B_VE + s));
                    if (j + 1 == steps) commit_if(e, bb + 8 * B::B_QE);
                    if (++s == B::VS) s = 0, round ^= 1;
                }
            }
            ++k;
        }
    } else if (warp >= 4) {
        const int half = (warp - 4) >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, td = t_dp + lanes + 64 * half;
        int n = 0, k = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const Item x(geo, it);
            if (x.steps == 0) continue;
            const int i = x.i0 + row;
            const bool there = i < x.len;
            const int64_t at = (int64_t)x.h * geo.tokens + x.start + i;
            const float lse2 = there ? p.lse2[at] : CUDART_INF_F, delta = there ? p.delta[at] : 0.f;
            const bool single = i == 0 || (geo.window == 1 && geo.sinks == 0);  // sees itself alone
            const F2 c2 = f2(p.c2, p.c2), l2 = f2(-lse2, -lse2), d2 = f2(-delta, -delta);
            for (int j = 0; j < x.steps; ++j, ++n) {
                const bool far = x.is_far(j);
                const int k0 = x.key0(j) + 64 * half, chunks = x.keys(j) - 64 * half;  // none of a few sinks' for the second half
                const int hi = (far ? min(geo.sinks, i - geo.window + 1) - 1 - 64 * half : single ? -1 : i - k0),
                          lo = far ? 0 : i - geo.window + 1 - k0;
                const uint32_t ts = tmem + 128 * (n & 1) + lanes + 64 * half;
                if (!(ok = wait(B::B_SF + (n & 1), n >> 1) && wait(B::B_DF, n))) break;
                tc_fence_after();
                uint32_t v[2][32], d[2][32];
                if (chunks > 0) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tmem_ld32(ts + 32 * u, v[u]);
                        tmem_ld32(td + 32 * u, d[u]);
                    }
                    tmem_wait_ld();
                }
                tc_fence_before();
                warp_arrive(bar + B::B_DL);
                if (chunks > 0) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a, b;
                            f2_get(fma2(pair_w(v[u][e], v[u][e + 1]), c2, l2), a, b);
                            f2_get((pair_w(d[u][e], d[u][e + 1]) + d2) * f2(exp2_approx(a), exp2_approx(b)), a, b);
                            v[u][e] = __float_as_uint(a), v[u][e + 1] = __float_as_uint(b);
                        }
                    if (far || x.key0(j) + 127 > x.i0) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) v[c >> 5][c & 31] = c > hi ? 0u : v[c >> 5][c & 31];
                    }
                    if (!far && x.key0(j) < x.i0 + 128 - geo.window) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) v[c >> 5][c & 31] = c < lo ? 0u : v[c >> 5][c & 31];
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = pack2(pair_w(v[u][2 * e], v[u][2 * e + 1]));
                        tmem_st16(ts + 16 * u, o);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                warp_arrive(bar + made(n));
            }
            if (!ok) break;
            if (!(ok = wait(B::B_AF, k++))) break;
            tc_fence_after();
            const F2 sc = f2(p.scale, p.scale);
            const int r0 = x.i0 + (warp & 3) * 32;  // the warp's first row
            if (D == 128 || half == 0) {  // 64 channels
                uint32_t v[2][32], r[4][8];
                tmem_ld32(t_dq + lanes + 64 * half, v[0]);
                tmem_ld32(t_dq + lanes + 64 * half + 32, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        r[u][e] = pack2(pair_w(v[u >> 1][16 * (u & 1) + 2 * e], v[u >> 1][16 * (u & 1) + 2 * e + 1]) * sc);
                store_rows(p.dq + ((int64_t)(x.start + r0) * geo.hq + x.h) * D + 64 * half, (int64_t)geo.hq * D, x.len - r0, r);
            }
            tc_fence_before();
            warp_arrive(bar + B::B_AE);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    settle(ab);
    await_previous();  // whoever comes next waits for both kernels
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ================================================================ host side
// [tokens][H][D] bf16 with a token stride, boxes of 64 channels x 1 head x `rows` tokens.
template <int D> bool token_map(CUtensorMap *m, const void *ptr, int64_t stride, int H, int64_t tokens, int rows) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {D, (cuuint64_t)H, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {D * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D> cudaError_t forward(const WinGeom &geo, const WinArgs &a, cudaStream_t s) {
    CUtensorMap mq, mk, mv, mk16, mv16;
    if (!token_map<D>(&mq, a.q, a.q_stride, a.hq, geo.tokens, 128) ||
        !token_map<D>(&mk, a.k, a.k_stride, a.hk, geo.tokens, 128) ||
        !token_map<D>(&mv, a.v, a.v_stride, a.hk, geo.tokens, 128) ||
        !token_map<D>(&mk16, a.k, a.k_stride, a.hk, geo.tokens, 16) ||
        !token_map<D>(&mv16, a.v, a.v_stride, a.hk, geo.tokens, 16))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(win_forward_tc_kernel<D>, Fw<D>::SMEM, allowed);
    if (e != cudaSuccess) return e;
    const FwArgs p{geo, (__nv_bfloat16 *)a.o, a.lse, a.scale, a.scale * 1.4426950408889634f, geo.ntiles * geo.hq};
    win_forward_tc_kernel<D><<<p.items < sm_count() ? p.items : sm_count(), FW_THREADS, Fw<D>::SMEM, s>>>(p, mq, mk, mv, mk16,
                                                                                                       mv16);
    return cudaGetLastError();
}

template <int D>
cudaError_t backward(const WinGeom &geo, const WinArgs &a, float *lse2, float *delta, float *part, float *near, Launches &l) {
    CUtensorMap mq, mk, mv, mo, mk16, mv16;
    if (!token_map<D>(&mq, a.q, a.q_stride, a.hq, geo.tokens, 128) ||
        !token_map<D>(&mk, a.k, a.k_stride, a.hk, geo.tokens, 128) ||
        !token_map<D>(&mv, a.v, a.v_stride, a.hk, geo.tokens, 128) ||
        !token_map<D>(&mo, a.d_o, (int64_t)a.hq * D, a.hq, geo.tokens, 128) ||
        !token_map<D>(&mk16, a.k, a.k_stride, a.hk, geo.tokens, 16) ||
        !token_map<D>(&mv16, a.v, a.v_stride, a.hk, geo.tokens, 16))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed[3];
    cudaError_t e = allow_smem(win_dkv_tc_kernel<D>, Bw<D>::SMEM, allowed[0]);
    if (e == cudaSuccess) e = allow_smem(win_dq_tc_kernel<D>, Bq<D>::SMEM, allowed[1]);
    if (e == cudaSuccess) e = allow_smem(win_delta_tc_kernel<D>, Bd<D>::SMEM, allowed[2]);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    const float c2 = a.scale * 1.4426950408889634f;
    const BdArgs b{geo, a.lse, lse2, delta, c2, geo.ntiles * geo.hq};
    e = l.next(win_delta_tc_kernel<D>, b.items < sms ? b.items : sms, FW_THREADS, Bd<D>::SMEM, b, mq, mk, mv, mo, mk16, mv16);
    if (e != cudaSuccess) return e;
    const int fars = geo.sinks > 0 && geo.window < geo.T ? geo.ntiles * geo.hk : 0;
    BwArgs p{geo, (__nv_bfloat16 *)a.dq, (__nv_bfloat16 *)a.dk, (__nv_bfloat16 *)a.dv, lse2, delta, part, near,
             a.scale, c2, fars, fars + geo.ntiles * 2 * geo.hk};
    e = l.next(win_dkv_tc_kernel<D>, p.items < sms ? p.items : sms, BW_THREADS, Bw<D>::SMEM, p, mq, mk, mv, mo);
    if (e != cudaSuccess) return e;
    p.items = geo.ntiles * 2 * geo.hq;
    return l.next(win_dq_tc_kernel<D>, p.items < sms ? p.items : sms, BW_THREADS, Bq<D>::SMEM, p, mq, mk, mv, mo, mk16, mv16);
}

}  // namespace

cudaError_t launch_window_backward_tc(const WinGeom &geo, const WinArgs &a, float *lse2, float *delta, float *part,
                                      float *near, Launches &l) {
    return a.d == 128 ? backward<128>(geo, a, lse2, delta, part, near, l) : backward<64>(geo, a, lse2, delta, part, near, l);
}

cudaError_t launch_window_forward_tc(const WinGeom &geo, const WinArgs &a, cudaStream_t s) {
    return a.d == 128 ? forward<128>(geo, a, s) : forward<64>(geo, a, s);
}

cudaError_t read_window_error(int *out, bool reset) { return read_tc_error(out, reset); }

}  // namespace kda
