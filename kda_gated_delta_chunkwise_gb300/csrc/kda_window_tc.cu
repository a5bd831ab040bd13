// Attention with a sliding window and sinks on the tensor cores of sm_103a, bf16:
// tcgen05.mma, TMEM and TMA. The formulas stand in kda_window.cu.
//
// The kernels are persistent, one CTA per SM; roles are warps that meet at
// mbarriers, and every role walks the same items and steps. Every wait is
// bounded: one that runs out sets the device error word and the CTA's abort flag,
// every role leaves its loop, and the CTA ends normally. Every waiter of a barrier
// waits for each of its phases in turn.
#include <cuda.h>
#include <math_constants.h>

#include "kda_tc_roles.cuh"
#include "kda_window_tc.cuh"

namespace kda {
namespace {

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

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

// ================================================================ forward
// An item is 256 queries of one head, two contexts w of 128 rows: while one
// context's softmax runs, the tensor core works for the other. A step is a tile of
// 128 keys (the first one, where there are far pairs: the sinks alone, their
// number rounded up to 16). For context w:
//   S_w = Q_w K^T (TMEM), P_w = 2^{c S - m} as bf16 over S_w's own columns,
//   O_w += P_w V (TMEM).
// The MMAs of a context go S, PV, S, PV ..., so that S of a step being complete
// says that PV of the step before is, and the softmax may rescale O. It does so
// only when a row's maximum has grown by more than 2^8 since the last time: the
// weights are taken against the older maximum until then, up to 2^8, which fp32
// sums and bf16 weights carry as well.
//
// warp 0: TMA; 1: MMA (and zeros behind a sequence's end); 4-7, 8-11: the rows of
// the contexts, a thread each.
constexpr int FW_THREADS = 384;
template <int D> struct Fw {
    static constexpr int TILE = 128 * D * 2;
    static constexpr int ATOM = 128 * 128;               // 64 channels of 128 rows
    static constexpr int STAGES = D == 128 ? 5 : 8;      // K and V in turn
    static constexpr int KV = 2 * TILE;
    static constexpr int BAR = KV + STAGES * TILE;
    static constexpr int B_QF = 0, B_QE = 1, B_SF = 2, B_PF = 4, B_OF = 6, B_OE = 8, B_KF = 10, B_KE = B_KF + STAGES,
                         COUNT = B_KE + STAGES;
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
    int start, len, f, rows, h, hk;  // f: the tile's first token in its sequence
    int far, kw;                     // whether there is a step of the sinks, and its keys
    int kt0, steps;                  // first near tile of 128 keys
    int nf[2], diag[2];              // near tiles of the contexts
    bool far_of[2];
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
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            nf[w] = max(0, f + 128 * w - g.window + 1) >> 7;
            diag[w] = (f >> 7) + w;
            far_of[w] = far && rows > 128 * w && min(last, f + 128 * w + 127) >= g.window;
        }
        kt0 = nf[0];
        steps = rows > 0 ? far + diag[rows > 128] - kt0 + 1 : 0;
    }
    __device__ __forceinline__ bool is_far(int j) const { return j < far; }
    __device__ __forceinline__ int tile(int j) const { return kt0 + j - far; }
    __device__ __forceinline__ bool uses(int w, int j) const {
        if (rows <= 128 * w) return false;
        if (is_far(j)) return far_of[w];
        const int kt = tile(j);
        return kt >= nf[w] && kt <= diag[w];
    }
    __device__ __forceinline__ int key0(int j) const { return is_far(j) ? 0 : tile(j) * 128; }
    __device__ __forceinline__ int keys(int j) const { return is_far(j) ? kw : 128; }
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
            mbar_init(bar + i, (i >= F::B_PF && i < F::B_OF) || (i >= F::B_OE && i < F::B_KF) ? 4 : 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tm;  // S_0 | S_1 | O_0 | O_1
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&mq);
            prefetch_tmap(&mk);
            prefetch_tmap(&mv);
            int n = 0, q = 0;  // stages, items so far
            for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
                const FwItem x(geo, it);
                if (x.steps == 0) continue;
                auto keys = [&](const CUtensorMap *whole, const CUtensorMap *few, int j) {
                    const int s = n % F::STAGES;
                    if (!(ok = ab.wait(bar + F::B_KE + s, ((n / F::STAGES) & 1) ^ 1))) return;
                    ++n;
                    unsigned char *d = sm + F::KV + s * F::TILE;
                    uint64_t *full = bar + F::B_KF + s;
                    mbar_arrive_expect_tx(full, x.keys(j) * D * 2);
                    const int row = x.start + x.key0(j);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        if (!x.is_far(j)) tma_load_3d(d + c * F::ATOM, whole, full, 64 * c, x.hk, row);
                        else
                            for (int r = 0; r < x.kw; r += 16)
                                tma_load_3d(d + c * F::ATOM + r * 128, few, full, 64 * c, x.hk, row + r);
                    }
                };
                if (!(ok = ab.wait(bar + F::B_QE, (q & 1) ^ 1))) break;
                ++q;
                const int contexts = x.rows > 128 ? 2 : 1;
                mbar_arrive_expect_tx(bar + F::B_QF, contexts * F::TILE);
                for (int w = 0; w < contexts; ++w)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(sm + w * F::TILE + c * F::ATOM, &mq, bar + F::B_QF, 64 * c, x.h,
                                    x.start + x.f + 128 * w);
                for (int j = 0; j < x.steps && ok; ++j) {
                    keys(&mk, &mk16, j);
                    if (ok) keys(&mv, &mv16, j);
                }
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t I_O = idesc_bf16(128, D, false, true);
        int n = 0, q = 0;                  // stages, items so far
        int pv[2] = {0, 0}, oi[2] = {0, 0};  // softmax steps, items of the contexts
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            if (x.steps == 0) continue;
            if (!(ok = __all_sync(0xffffffffu, ab.wait(bar + F::B_QF, q & 1)))) break;
            ++q;
            // scores of step j, whose K is in stage s
            auto scores = [&](int w, int j, int s) {
                if (!x.uses(w, j)) return;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t d = tmem + 128 * w, idesc = idesc_bf16(128, x.keys(j), false, false);
                    const uint64_t a = desc_k(smem_u32(sm + w * F::TILE)), b = desc_k(smem_u32(sm + F::KV + s * F::TILE));
                    mma_ss<false>(d, a, b, idesc);
#pragma unroll
                    for (int ks = 1; ks < D / 16; ++ks)
                        mma_ss<true>(d, a + step_k(ks, F::ATOM), b + step_k(ks, F::ATOM), idesc);
                    umma_commit(bar + F::B_SF + w);
                }
                __syncwarp();
            };
            auto arrived = [&](int i) {  // stage of the i-th tile
                return __all_sync(0xffffffffu, ab.wait(bar + F::B_KF + i % F::STAGES, (i / F::STAGES) & 1));
            };
            auto release = [&](int i) {
                if (lane == 0) umma_commit(bar + F::B_KE + i % F::STAGES);
                __syncwarp();
            };
            if (!(ok = arrived(n))) break;
            scores(0, 0, n % F::STAGES);
            scores(1, 0, n % F::STAGES);
            release(n);
            bool first[2] = {true, true};
            int last[2] = {-1, -1};
            for (int j = 0; j < x.steps; ++j)
                for (int w = 0; w < 2; ++w)
                    if (x.uses(w, j)) last[w] = j;
            if (x.steps == 1 && lane == 0) umma_commit(bar + F::B_QE);
            for (int j = 0; j < x.steps && ok; ++j) {
                const int iv = n + 2 * j + 1, ik = iv + 1;  // this step's V, the next one's K
                const bool more = j + 1 < x.steps;
                if (!(ok = arrived(iv))) break;
                unsigned char *v = sm + F::KV + (iv % F::STAGES) * F::TILE;
                const int behind = x.len - x.key0(j);  // rows of V past the sequence's end may hold anything
                if (behind < x.keys(j)) zero_rows<D>(v, behind, x.keys(j));
                if (more && !(ok = arrived(ik))) break;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (x.uses(w, j)) {
                        ok = __all_sync(0xffffffffu, ab.wait(bar + F::B_PF + w, pv[w] & 1));
                        if (!ok) break;
                        ++pv[w];
                        if (first[w] && !(ok = __all_sync(0xffffffffu, ab.wait(bar + F::B_OE + w, (oi[w] & 1) ^ 1)))) break;
                        tc_fence_after();
                        if (lane == 0) {
                            const uint32_t o = tmem + 256 + 128 * w, pt = tmem + 128 * w;
                            const uint64_t b = desc_mn(smem_u32(v), F::ATOM);
                            if (first[w]) umma_bf16_ts<false>(o, pt, b, I_O);
                            else umma_bf16_ts<true>(o, pt, b, I_O);
                            if (x.is_far(j)) {
                                for (int ks = 1; ks < x.kw / 16; ++ks) umma_bf16_ts<true>(o, pt + ks * 8, b + step_mn(ks), I_O);
                            } else {
#pragma unroll
                                for (int ks = 1; ks < 8; ++ks) umma_bf16_ts<true>(o, pt + ks * 8, b + step_mn(ks), I_O);
                            }
                            if (j == last[w]) umma_commit(bar + F::B_OF + w);
                        }
                        __syncwarp();
                        if (j == last[w]) ++oi[w];
                        first[w] = false;
                    }
                    if (more) scores(w, j + 1, ik % F::STAGES);
                }
                if (!ok) break;
                release(iv);
                if (more) release(ik);
                if (j + 2 == x.steps && lane == 0) umma_commit(bar + F::B_QE);  // the last scores are on their way
                __syncwarp();
            }
            n += 2 * x.steps;
        }
    } else if (warp >= 4) {
        const int w = (warp - 4) >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, ts = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
        int sf = 0, of = 0;
        for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
            const FwItem x(geo, it);
            if (x.rows <= 128 * w) continue;
            const int i = x.f + 128 * w + row;
            float m = -CUDART_INF_F;
            F2 l = f2(0.f, 0.f);
            bool first = true;
            for (int j = 0; j < x.steps && ok; ++j) {
                if (!x.uses(w, j)) continue;
                ok = __all_sync(0xffffffffu, ab.wait(bar + F::B_SF + w, sf & 1));
                if (!ok) break;
                ++sf;
                tc_fence_after();
                const bool far = x.is_far(j);
                const int k0 = x.key0(j), chunks = far ? (x.kw + 31) >> 5 : 4;
                // columns lo .. hi are seen; the whole tile by every row of the context: no masks
                const int hi = far ? min(geo.sinks, i - geo.window + 1) - 1 : i - k0, lo = far ? 0 : i - geo.window + 1 - k0;
                const bool masked = far || k0 + 127 > x.f + 128 * w || k0 < x.f + 128 * w + 127 - geo.window + 1;
                auto mask = [&](uint32_t (&s)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        s[e] = c + e < lo || c + e > hi ? 0xff800000u : s[e];
                };
                float top = -CUDART_INF_F;
                uint32_t s[32];
                for (int c = 0; c < chunks; ++c) {
                    tmem_ld32(ts + 32 * c, s);
                    tmem_wait_ld();
                    if (masked) mask(s, 32 * c);
                    float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
                    for (int e = 2; e < 32; e += 2)
                        a = fmaxf(a, __uint_as_float(s[e])), b = fmaxf(b, __uint_as_float(s[e + 1]));
                    top = max3(top, a, b);
                }
                const bool grow = (top - m) * p.c2 > 8.f;  // also the first number that a row sees
                if (!first && __any_sync(0xffffffffu, grow)) {
                    const float f = grow ? exp2_approx((m - top) * p.c2) : 1.f;
                    const F2 ff = f2(f, f);
                    l = l * ff;
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
                first = false;
                const float off = m == -CUDART_INF_F ? 0.f : -m * p.c2;
                const F2 c2 = f2(p.c2, p.c2), off2 = f2(off, off);
                for (int c = 0; c < chunks; ++c) {
                    tmem_ld32(ts + 32 * c, s);
                    tmem_wait_ld();
                    if (masked) mask(s, 32 * c);
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, b;
                        f2_get(fma2(pair_w(s[e], s[e + 1]), c2, off2), a, b);
                        a = exp2_approx(a), b = exp2_approx(b);
                        l = fma2(f2(a, b), f2(1.f, 1.f), l);
                        o[e / 2] = pack2(a, b);
                    }
                    tmem_st16(ts + 16 * c, o);  // over columns that have been read
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar + F::B_PF + w);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, ab.wait(bar + F::B_OF + w, of & 1));
            if (!ok) break;
            ++of;
            tc_fence_after();
            const float sum = f2_sum(l), f = 1.f / sum;
            const bool there = i < x.len;
            const int64_t at = (int64_t)(x.start + i) * geo.hq + x.h;
            const F2 ff = f2(f, f);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t r[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[e] = pack2(pair_w(o[16 * u + 2 * e], o[16 * u + 2 * e + 1]) * ff);
                    if (there) st_v8(p.o + at * D + c + 16 * u, r);
                }
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

}  // namespace

cudaError_t launch_window_forward_tc(const WinGeom &geo, const WinArgs &a, cudaStream_t s) {
    return a.d == 128 ? forward<128>(geo, a, s) : forward<64>(geo, a, s);
}

cudaError_t read_window_error(int *out, bool reset) { return read_tc_error(out, reset); }

}  // namespace kda
