// The cache of window attention: writing the keys and values of packed prompts
// into their slots, and one token per sequence against its slot.
//
// A slot holds the sinks and then a ring of the last `window` tokens, entry by
// entry [entries][hk][d]. With the new token written, the tokens that it sees
// are exactly the first min(position + 1, entries) entries, and a softmax does not
// mind their order, so a step is an attention over a stretch of memory.
//
// The step is bound by memory: every entry of a key head is read once for all
// its query heads. One warp takes 16 entries (fp32: 8) at a time, 8 KB of keys and
// values, from a ring of its own that cp.async fills two steps ahead (128 KB in
// flight on an SM; straight into registers, a step's values were waited for in
// every step: 451 us for 256 sequences of 32 heads, 8 key heads and 2052 entries).
// They go into the fragments of mma.sync, 16 query heads (or what there are) as the
// rows of the product: a contraction does not mind the order of its index, so a
// lane reads 16 bytes of consecutive channels and the query's fragments are read
// the same way; for the values' product a lane holds the entries and channels that
// its fragments want, two entries' halves joined by a byte permutation. That case takes
// 304 us (7.1 TB/s). fp32 calls of up to eight query heads to a key head go another way
// (see FourHeads): 256 sequences of 3000 entries, four heads to each of four key heads 450
// us (7.0 TB/s), by split tf32 780; eight to one 153 and 219. More heads to a key head stay
// with split tf32: sixteen to each of two 451 us (3.5 TB/s). Few sequences are cut over the
// CTAs of a cluster, whose sums are joined through distributed shared memory in rank
// order.
#include <math_constants.h>

#include <type_traits>

#include "kda_rows.cuh"
#include "kda_tc_ptx.cuh"
#include "kda_window.cuh"

namespace kda {
namespace {

// ================================================================ prompts into the cache
// A stretch of the tokens that are kept, of all prompts one after the other, to each
// block. Every block reads all offsets once, since nothing may be written if any is bad,
// and adds up on the way what each prompt keeps. (A block to each eight tokens that a
// prompt might keep, which read all offsets too, took 1388 us for 4096 prompts of 16 tokens
// and slots of 2052, now 31; 256 of 64, eight heads, 65 and 27; 16 of 4096 46 and 48.)
constexpr int CT = 256, CTOK = 8, CFLIGHT = 4;  // CTOK: tokens of a stretch come in eights; CFLIGHT: pieces on their way
__global__ void __launch_bounds__(CT)
win_cache_write_kernel(WinCacheArgs p, int row16, int es) {  // row16: 16-byte pieces of a token's heads
    __shared__ int bad, missing, first_prompt, first_token;
    __shared__ int64_t sums[CT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        bad = (p.cu_seqlens[0] != 0 || p.cu_seqlens[p.N] != p.T) ? 1 : 0;
        missing = 0;
    }
    __syncthreads();
    bool fresh;
    // a warp's prompts, and the tokens that they keep
    const int each = (p.N + CT - 1) / CT * 32, n0 = min(p.N, warp * each), n1 = min(p.N, n0 + each);
    int64_t mine = 0;
    bool down = false, none = false;
#pragma unroll 4
    for (int n = n0 + lane; n < n1; n += 32) {
        const int64_t len = (int64_t)p.cu_seqlens[n + 1] - p.cu_seqlens[n];
        down |= len < 0;
        if (blockIdx.x == 0) none |= slot_of(p.slots, n, fresh) >= p.pool;
        mine += min(len, (int64_t)p.entries);
    }
    if (down) atomicOr(&bad, 1);
    if (none) atomicOr(&missing, 1);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    if (bad || missing) {
        if (tid == 0 && blockIdx.x == 0 && p.status) atomicOr(p.status, bad ? KDA_DEV_BAD_CU_SEQLENS : KDA_DEV_BAD_SLOT);
        if (bad) return;
    }
    int64_t before = 0, all = 0;  // of the warps in front; of all
#pragma unroll
    for (int w = 0; w < CT / 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    // this block's stretch, and where it starts
    const int64_t per = ((all + CTOK - 1) / CTOK + gridDim.x - 1) / gridDim.x * CTOK;
    int64_t at = blockIdx.x * per;
    const int64_t end = min(all, at + per);
    if (at >= end) return;
    if (before <= at && at < before + mine) {  // in one of this warp's prompts
        for (int n = n0 + lane;; n += 32) {
            const int kept = n < n1 ? min(p.cu_seqlens[n + 1] - p.cu_seqlens[n], p.entries) : 0;
            int64_t upto = before + kept;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, off) - before;
                if (lane >= off) upto += y;
            }
            if (upto - kept <= at && at < upto) first_prompt = n, first_token = (int)(at - (upto - kept));
            before = __shfl_sync(0xffffffffu, upto, 31);
            if (at < before) break;
        }
    }
    __syncthreads();
    const int window = p.entries - p.sinks;
    for (int n = first_prompt, skip = first_token; at < end; ++n, skip = 0) {
        const int start = p.cu_seqlens[n], len = p.cu_seqlens[n + 1] - start;
        const int first = min(p.sinks, len), second = max(first, len - window), kept = first + len - second;
        const int upto_here = (int)min((int64_t)kept, skip + end - at);
        at += upto_here - skip;
        const int64_t slot = slot_of(p.slots, n, fresh);
        if (slot >= p.pool) continue;
        for (int x0 = skip; x0 < upto_here; x0 += 32) {
            const int pieces = min(32, upto_here - x0) * row16;
            for (int i0 = tid; i0 < pieces; i0 += CFLIGHT * CT) {
                uint4 k[CFLIGHT], v[CFLIGHT];
#pragma unroll
                for (int u = 0; u < CFLIGHT; ++u) {
                    const int i = i0 + u * CT, x = x0 + i / row16, c = i % row16 * (16 / es);
                    if (i >= pieces) continue;
                    const int64_t token = start + (x < first ? x : second + x - first);
                    k[u] = *reinterpret_cast<const uint4 *>((const char *)p.k + (token * p.k_stride + c) * es);
                    v[u] = *reinterpret_cast<const uint4 *>((const char *)p.v + (token * p.v_stride + c) * es);
                }
#pragma unroll
                for (int u = 0; u < CFLIGHT; ++u) {
                    const int i = i0 + u * CT, x = x0 + i / row16, c = i % row16 * (16 / es), token = x < first ? x : second + x - first;
                    if (i >= pieces) continue;
                    const int64_t entry = slot * p.entries + (token < p.sinks ? token : p.sinks + (token - p.sinks) % window);
                    const int64_t dst = (entry * p.hk * p.d + c) * es;
                    *reinterpret_cast<uint4 *>((char *)p.k_cache + dst) = k[u];
                    *reinterpret_cast<uint4 *>((char *)p.v_cache + dst) = v[u];
                }
            }
        }
    }
}

// ================================================================ one token
constexpr int DT = 128, DW = DT / 32, HEADS = 16;

__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d += the fp32 product of four values of a with two of b, each in two tf32 parts
__device__ __forceinline__ void mma_fp32(float (&d)[4], const float (&a)[4], float x0, float x1) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = tf32(a[i]);
        lo[i] = tf32(a[i] - __uint_as_float(hi[i]));
    }
    const uint32_t h0 = tf32(x0), h1 = tf32(x1);
    mma_tf32(d, lo, h0, h1);
    mma_tf32(d, hi, tf32(x0 - __uint_as_float(h0)), tf32(x1 - __uint_as_float(h1)));
    mma_tf32(d, hi, h0, h1);
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// What a type's fragments look like. Channels: a chunk is 16 bytes, CH channels; a
// lane's K chunks are 4 CH apart (t within), its V chunks 8 CH apart (g within).
template <typename T, int D> struct Shape {
    static constexpr int CH = 16 / sizeof(T);
    static constexpr int KEYS = sizeof(T) == 2 ? 16 : 8;  // entries a step
    static constexpr int NB = KEYS / 8;                   // their 8-column blocks
    static constexpr int KC = D / (4 * CH);               // chunks of a lane and key
    static constexpr int VC = D / (8 * CH);               // chunks of a lane and value row
    static constexpr int VR = sizeof(T) == 2 ? 4 : 2;     // value rows of a lane
    // the value row u of lane t within the step
    static __device__ __forceinline__ int v_row(int t, int u) { return 2 * t + (u & 1) + (u >> 1) * 8; }
    // The ring: a stage is the step's keys, then its values, entry by entry, 16-byte pieces exchanged so that the
    // eight lanes that read at a time (two rows of keys, four of values) meet eight different banks of 16 bytes.
    static constexpr int ROW = D * sizeof(T), STAGE = 2 * KEYS * ROW, STAGES = 3;
    static __device__ __forceinline__ int k_at(int row, int piece) { return row * ROW + ((piece ^ ((row & 1) << 2)) << 4); }
    static __device__ __forceinline__ int v_at(int row, int piece) { return (KEYS + row) * ROW + ((piece ^ (row & 7)) << 4); }
};

// fp32 and up to eight query heads to a key head: fp32 products, four heads at a
// time. A row is 16 bytes in each of D / 4 lanes; the sums of a step's eight entries
// and four heads are shared out among the lanes while they are added up, one to a lane.
template <int D> struct FourHeads {
    static constexpr int L = D / 4, R = 32 / L, ROWS = 8 / R;  // lanes of a row, rows at a time, times
    F2 q[4][2], acc[4][2];
    float m, l;  // of head lane % 4; l: of this lane's entries
    __device__ __forceinline__ void load(const float *src, int heads, int lane) {
        m = -CUDART_INF_F, l = 0.f;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float4 x = h < heads ? *reinterpret_cast<const float4 *>(src + h * D + lane % L * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            q[h][0] = f2(x.x, x.y), q[h][1] = f2(x.z, x.w);
            acc[h][0] = acc[h][1] = f2(0.f, 0.f);
        }
    }
    // the entries' keys at k(row), values at v(row); `there` entries; c2: the scale in powers of two
    template <typename K, typename V> __device__ __forceinline__ void step(K k, V v, int there, float c2, int lane) {
        const int sub = lane / L;
        float s[4 * ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float4 x = k(i * R + sub);
#pragma unroll
            for (int h = 0; h < 4; ++h) s[4 * i + h] = f2_sum(fma2(f2(x.z, x.w), q[h][1], f2(x.x, x.y) * q[h][0]));
        }
#pragma unroll
        for (int n = 2 * ROWS, bit = L / 2; bit > 0; n >>= 1, bit >>= 1) {
            const bool up = lane & bit;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = up ? s[i] : s[i + n], keep = up ? s[i + n] : s[i];
                s[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
            }
        }
        const float x = lane % L / 4 * R + sub < there ? s[0] * c2 : -CUDART_INF_F;  // of that entry
        float top = fmaxf(m, x);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float scale = exp2_approx(m - top), w = exp2_approx(x - top);
        l = fmaf(l, scale, w);
        if (__any_sync(0xffffffffu, top != m)) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float f = __shfl_sync(0xffffffffu, scale, h);
                acc[h][0] = acc[h][0] * f2(f, f), acc[h][1] = acc[h][1] * f2(f, f);
            }
        }
        m = top;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float4 y = v(i * R + sub);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float f = __shfl_sync(0xffffffffu, w, sub * L + 4 * i + h);
                acc[h][0] = fma2(f2(f, f), f2(y.x, y.y), acc[h][0]);
                acc[h][1] = fma2(f2(f, f), f2(y.z, y.w), acc[h][1]);
            }
        }
    }
    // the warp's sums: [4][D], and of each head its maximum and sum
    __device__ __forceinline__ void store(float *part, float *stat, int heads, int lane) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (lane < 4 && lane < heads) stat[2 * lane] = m, stat[2 * lane + 1] = l;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            float a[4];
            f2_get(acc[h][0], a[0], a[1]);
            f2_get(acc[h][1], a[2], a[3]);
            if (R == 2) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] += __shfl_xor_sync(0xffffffffu, a[e], 16);
            }
            if (h < heads && lane < L) *reinterpret_cast<float4 *>(part + h * D + lane * 4) = make_float4(a[0], a[1], a[2], a[3]);
        }
    }
};

// QUADS: of fp32, fours of query heads that go the way above; 0: mma.sync
template <typename T, int D, int QUADS>
__global__ void __launch_bounds__(DT, 2)
win_decode_kernel(WinCacheArgs p, int cl) {
    using S = Shape<T, D>;
    constexpr int CH = S::CH, KEYS = S::KEYS, NB = S::NB, KC = S::KC, VC = S::VC, VR = S::VR;
    extern __shared__ __align__(16) float sm[];
    float *part = sm;                            // [DW][HEADS][D]: the warps' sums, in the rings' place
    float *own = part + DW * HEADS * D;          // [HEADS][D]: the CTA's
    float *stat = own + HEADS * D;               // [DW][HEADS][2]: the warps' maximum and sum
    float *own_stat = stat + DW * HEADS * 2;     // [HEADS][2]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % cl, nh = blockIdx.x / cl, n = nh / p.hk, hk = nh - n * p.hk, group = p.hq / p.hk;
    bool fresh;
    const int64_t slot = slot_of(p.slots, n, fresh);
    const int pos = p.positions[n];
    if (slot >= p.pool || pos < 0) {  // the same in the whole cluster
        if (tid == 0 && rank == 0 && p.status) atomicOr(p.status, slot >= p.pool ? KDA_DEV_BAD_SLOT : KDA_DEV_BAD_POSITION);
        return;
    }
    const int window = p.entries - p.sinks;
    const int fill = pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % window;  // the new token's entry
    const int count = pos < p.entries ? pos + 1 : p.entries;
    const T *knew = (const T *)p.k + n * p.k_stride + hk * D, *vnew = (const T *)p.v + n * p.v_stride + hk * D;
    const int64_t step = (int64_t)p.hk * D, base = (slot * p.entries * p.hk + hk) * D;
    T *kc = (T *)p.k_cache + base, *vc = (T *)p.v_cache + base;
    // the new row is read where it came from, by whoever has its entry, so writing it races with nobody
    if (rank == 0 && tid < 2 * (D / CH)) {
        const int c = tid % (D / CH) * CH;
        const bool is_k = tid < D / CH;
        *reinterpret_cast<uint4 *>((is_k ? kc : vc) + fill * step + c) =
            *reinterpret_cast<const uint4 *>((is_k ? knew : vnew) + c);
    }
    const int tiles = (count + KEYS - 1) / KEYS, per = (tiles + cl - 1) / cl;
    const int tile0 = rank * per, tile1 = min(tiles, tile0 + per);
    const float c2 = p.scale * 1.4426950408889634f;  // scores in powers of two

    for (int h0 = 0; h0 < group; h0 += HEADS) {
        const int heads = min(HEADS, group - h0);
        const T *q = (const T *)p.q + n * p.q_stride + (int64_t)(hk * group + h0) * D;
        FourHeads<D> four[QUADS > 0 ? QUADS : 1];
        uint4 qf[2][KC];  // rows g and g + 8
        if constexpr (QUADS > 0) {
#pragma unroll
            for (int u = 0; u < QUADS; ++u) four[u].load((const float *)q + 4 * u * D, heads - 4 * u, lane);
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int j = 0; j < KC; ++j)
                    qf[r][j] = g + r * 8 < heads ? *reinterpret_cast<const uint4 *>(q + (g + r * 8) * D + 4 * CH * j + CH * t)
                                                 : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        float acc[D / 8][4], m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        unsigned char *ring = reinterpret_cast<unsigned char *>(sm) + warp * S::STAGES * S::STAGE;
        const uint32_t ring_s = tc::smem_u32(ring);
        auto fetch = [&](int tile, int stage) {  // one group of copies, empty past the last step
            if (tile < tile1) {
                constexpr int PIECES = D / CH;
#pragma unroll
                for (int i = 0; i < KEYS * PIECES / 32; ++i) {
                    const int r = (i * 32 + lane) / PIECES, piece = (i * 32 + lane) % PIECES, e = tile * KEYS + r;
                    const bool there = e < count;
                    const int64_t at = (there ? e : 0) * step + piece * CH;
                    const uint32_t dst = ring_s + stage * S::STAGE;
                    copy16(dst + S::k_at(r, piece), e == fill ? knew + piece * CH : kc + at, there);
                    copy16(dst + S::v_at(r, piece), e == fill ? vnew + piece * CH : vc + at, there);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int tile = tile0 + warp, stage = 0;
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i) fetch(tile + i * DW, i);
        for (; tile < tile1; tile += DW) {
            __syncwarp();  // the stage that is filled now has been read by every lane
            fetch(tile + (S::STAGES - 1) * DW, stage == 0 ? S::STAGES - 1 : stage - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 1) : "memory");
            __syncwarp();
            const unsigned char *buf = ring + stage * S::STAGE;
            stage = stage == S::STAGES - 1 ? 0 : stage + 1;
            if constexpr (QUADS > 0) {
                const int piece = lane % FourHeads<D>::L;
                auto k = [&](int row) { return *reinterpret_cast<const float4 *>(buf + S::k_at(row, piece)); };
                auto v = [&](int row) { return *reinterpret_cast<const float4 *>(buf + S::v_at(row, piece)); };
#pragma unroll
                for (int u = 0; u < QUADS; ++u) four[u].step(k, v, count - tile * KEYS, c2, lane);
            } else {
                uint4 vf[VR][VC];
                float s[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.f;
#pragma unroll
                    for (int j = 0; j < KC; ++j) {
                        const uint4 x = qf[0][j], y = qf[1][j];
                        const uint4 k = *reinterpret_cast<const uint4 *>(buf + S::k_at(b * 8 + g, 4 * j + t));
                        if constexpr (sizeof(T) == 2) {
                            mma_bf16(s[b], x.x, y.x, x.y, y.y, k.x, k.y);
                            mma_bf16(s[b], x.z, y.z, x.w, y.w, k.z, k.w);
                        } else {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            const float a0[4] = {__uint_as_float(x.x), __uint_as_float(y.x), __uint_as_float(x.y), __uint_as_float(y.y)};
                            const float a1[4] = {__uint_as_float(x.z), __uint_as_float(y.z), __uint_as_float(x.w), __uint_as_float(y.w)};
                            mma_fp32(d, a0, __uint_as_float(k.x), __uint_as_float(k.y));
                            mma_fp32(d, a1, __uint_as_float(k.z), __uint_as_float(k.w));
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[b][e] += d[e];
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < VR; ++u)
#pragma unroll
                    for (int i = 0; i < VC; ++i)
                        vf[u][i] = *reinterpret_cast<const uint4 *>(buf + S::v_at(S::v_row(t, u), 8 * i + g));
                float top[2] = {m[0], m[1]};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[b][e] = tile * KEYS + b * 8 + 2 * t + (e & 1) < count ? s[b][e] * c2 : -CUDART_INF_F;
                        top[e >> 1] = fmaxf(top[e >> 1], s[b][e]);
                    }
                }
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // a step has an entry at least, so the maximum is a number
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                    keep[e] = exp2_approx(m[e] - top[e]);
                    l[e] *= keep[e];
                }
                if (__any_sync(0xffffffffu, top[0] != m[0] || top[1] != m[1])) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][e] *= keep[e >> 1];
                    }
                }
                m[0] = top[0], m[1] = top[1];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[b][e] = exp2_approx(s[b][e] - m[e >> 1]);
                        l[e >> 1] += s[b][e];
                    }
                }
                if constexpr (sizeof(T) == 2) {
                    // the weights are rounded to bf16, as the values are: by 2^-8 of each at most and independently of
                    // one another, so that their sum is off by no more than the result's own rounding
                    const uint32_t a0 = pack(s[0][0], s[0][1]), a1 = pack(s[0][2], s[0][3]), a2 = pack(s[NB - 1][0], s[NB - 1][1]),
                                   a3 = pack(s[NB - 1][2], s[NB - 1][3]);
#pragma unroll
                    for (int i = 0; i < VC; ++i) {
                        const uint32_t w[4][4] = {{vf[0][i].x, vf[0][i].y, vf[0][i].z, vf[0][i].w},
                                                  {vf[1][i].x, vf[1][i].y, vf[1][i].z, vf[1][i].w},
                                                  {vf[VR - 2][i].x, vf[VR - 2][i].y, vf[VR - 2][i].z, vf[VR - 2][i].w},
                                                  {vf[VR - 1][i].x, vf[VR - 1][i].y, vf[VR - 1][i].z, vf[VR - 1][i].w}};
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            const uint32_t sel = b & 1 ? 0x7632 : 0x5410;
                            mma_bf16(acc[i * 8 + b], a0, a1, a2, a3, __byte_perm(w[0][b / 2], w[1][b / 2], sel),
                                     __byte_perm(w[2][b / 2], w[3][b / 2], sel));
                        }
                    }
                } else {
                    const float a[4] = {s[0][0], s[0][2], s[0][1], s[0][3]};
#pragma unroll
                    for (int i = 0; i < VC; ++i) {
                        const float w[2][4] = {{__uint_as_float(vf[0][i].x), __uint_as_float(vf[0][i].y),
                                                __uint_as_float(vf[0][i].z), __uint_as_float(vf[0][i].w)},
                                               {__uint_as_float(vf[1][i].x), __uint_as_float(vf[1][i].y),
                                                __uint_as_float(vf[1][i].z), __uint_as_float(vf[1][i].w)}};
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_fp32(d, a, w[0][b], w[1][b]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i * 4 + b][e] += d[e];
                        }
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the rings have been read
        if constexpr (QUADS > 0) {
#pragma unroll
            for (int u = 0; u < QUADS; ++u)
                four[u].store(part + (warp * HEADS + 4 * u) * D, stat + (warp * HEADS + 4 * u) * 2, heads - 4 * u, lane);
        } else {
            // the warps' sums: lane (g, t) has, of rows g and g + 8, channels 8 CH i + CH (2 t + e) + b
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                const int r = g + e * 8;
                if (r >= heads) continue;
                if (t == 0) stat[(warp * HEADS + r) * 2] = m[e], stat[(warp * HEADS + r) * 2 + 1] = l[e];
                float *dst = part + (warp * HEADS + r) * D;
#pragma unroll
                for (int i = 0; i < VC; ++i) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
#pragma unroll
                        for (int b = 0; b < CH; b += 4)
                            *reinterpret_cast<float4 *>(dst + 8 * CH * i + CH * (2 * t + u) + b) =
                                make_float4(acc[i * CH + b][2 * e + u], acc[i * CH + b + 1][2 * e + u],
                                            acc[i * CH + b + 2][2 * e + u], acc[i * CH + b + 3][2 * e + u]);
                    }
                }
            }
        }
        __syncthreads();
        for (int x = tid; x < heads * D; x += DT) {
            const int r = x / D;
            float top = -CUDART_INF_F, a = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < DW; ++w) top = fmaxf(top, stat[(w * HEADS + r) * 2]);
#pragma unroll
            for (int w = 0; w < DW; ++w) {
                const float mw = stat[(w * HEADS + r) * 2], f = mw == -CUDART_INF_F ? 0.f : exp2_approx(mw - top);
                a += f * part[(w * HEADS) * D + x];
                sum += f * stat[(w * HEADS + r) * 2 + 1];
            }
            if (cl == 1) {
                ((T *)p.o)[((int64_t)n * p.hq + hk * group + h0) * D + x] = from_f32<T>(a / sum);
            } else {
                own[x] = a;
                if (x % D == 0) own_stat[2 * r] = top, own_stat[2 * r + 1] = sum;
            }
        }
        if (cl > 1) {
            tc::cluster_sync();
            const uint32_t so = tc::smem_u32(own), ss = tc::smem_u32(own_stat);
            auto remote = [](uint32_t addr, int r) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::mapa(addr, r)) : "memory");
                return v;
            };
            const int share = (heads * D + cl - 1) / cl;
            for (int x = rank * share + tid; x < min(heads * D, (rank + 1) * share); x += DT) {
                const int r = x / D;
                float top = -CUDART_INF_F, a = 0.f, sum = 0.f;
                for (int k = 0; k < cl; ++k) top = fmaxf(top, remote(ss + r * 8, k));
                for (int k = 0; k < cl; ++k) {
                    const float mk = remote(ss + r * 8, k), f = mk == -CUDART_INF_F ? 0.f : exp2_approx(mk - top);
                    a += f * remote(so + x * 4, k);
                    sum += f * remote(ss + r * 8 + 4, k);
                }
                ((T *)p.o)[((int64_t)n * p.hq + hk * group + h0) * D + x] = from_f32<T>(a / sum);
            }
            tc::cluster_sync();
        } else {
            __syncthreads();
        }
    }
}

template <typename T, int D, int QUADS> cudaError_t decode(const WinCacheArgs &a, cudaStream_t s) {
    constexpr size_t sums = (DW * HEADS * D + HEADS * D + DW * HEADS * 2 + HEADS * 2) * sizeof(float);
    constexpr size_t rings = DW * Shape<T, D>::STAGES * Shape<T, D>::STAGE, smem = sums > rings ? sums : rings;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(win_decode_kernel<T, D, QUADS>, smem, allowed);
    if (e != cudaSuccess) return e;
    // CTAs of a cluster: as many as still run all at once (two on an SM, less what does not come out even with the
    // clusters' places: 75 sequences of one head in clusters of four, 300 CTAs, took 25.8 us, in pairs 19.5; 64 in
    // clusters of four 20.2, of two 21.9), and a step for every warp. A second round costs more than longer
    // stretches: 100 in clusters of four 38.8, in pairs 31.8.
    const int64_t work = (int64_t)a.N * a.hk;
    int cl = 1;
    while (cl < 8 && work * cl * 2 <= 256 && a.entries >= cl * 2 * DW * Shape<T, D>::KEYS) cl *= 2;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cl;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(work * cl));
    c.blockDim = dim3(DT);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, win_decode_kernel<T, D, QUADS>, a, cl);
}

}  // namespace

cudaError_t launch_window_cache_write(const WinCacheArgs &a, cudaStream_t s) {
    const int es = a.dt == KDA_BF16 ? 2 : 4;
    const int64_t kept = (int64_t)a.N * a.entries < a.T ? (int64_t)a.N * a.entries : a.T, blocks = (kept + CTOK - 1) / CTOK;  // at most
    constexpr int MOST = 152 * 2048 / CT;  // all that run at once
    win_cache_write_kernel<<<blocks < 1 ? 1 : blocks < MOST ? (unsigned)blocks : MOST, CT, 0, s>>>(a, a.hk * a.d * es / 16, es);
    return cudaGetLastError();
}

cudaError_t launch_window_decode(const WinCacheArgs &a, cudaStream_t s) {
    const int group = a.hq / a.hk;
    auto of = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (a.dt == KDA_BF16) return decode<__nv_bfloat16, D, 0>(a, s);
        return group <= 4 ? decode<float, D, 1>(a, s) : group <= 8 ? decode<float, D, 2>(a, s) : decode<float, D, 0>(a, s);
    };
    return a.d == 128 ? of(std::integral_constant<int, 128>{}) : of(std::integral_constant<int, 64>{});
}

}  // namespace kda
