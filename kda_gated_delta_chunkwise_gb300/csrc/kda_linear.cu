// Linear attention with a decay: S_t = e^{g_t} S_{t-1} + k_t v_t^T,
// o_t = scale S_t^T q_t, and its gradients, for any supported type and size.
//
// A sequence is cut into blocks. With L_i the sum of the log decays of a
// block's tokens up to i and S the state before the block,
//   o_i = scale (e^{L_i} S^T q_i + sum_{j <= i} e^{L_i - L_j} (q_i . k_j) v_j)
//   S'  = e^{L_end} S + sum_j e^{L_end - L_j} k_j v_j^T.
// Every exponent is a sum of log decays over a stretch of tokens, so it is <= 0
// and nothing overflows however strong the decay. Three launches:
//   lin_state_kernel   every block's own sum over j, all blocks at once;
//   lin_scan_kernel    joins them along each sequence, one pass, elementwise;
//   lin_attend_kernel  every block's outputs, all blocks at once.
// A block of the general kernels is 64 tokens, one CTA; where the shapes allow
// it the tensor-core kernels (kda_linear_tc.cu) take the place of the first and
// the last.
// Backward, with G the gradient of the state after a token
// (G_t = scale q_t do_t^T + e^{g_{t+1}} G_{t+1}): dq_t = scale S_t do_t,
// dk_t = G_t v_t, dv_t = G_t^T k_t. These are three more attentions of the
// same form: dq with (do, v, k) for (q, k, v) and S transposed, dk with
// (v, do, q) and dv with (k, q, do) in reverse time with G for S; so the same
// three kernels run them, both directions (all three attentions) in one launch. The gradient of a log decay is everything that
// passes over the step into its token,
//   dg_t = sum_{i >= t > j} M_ij + sum_{i >= t} q_i.dq_i(S part)
//        + sum_{j < t} k_j.dk_j(G part) + e^{L_end} <S, G>    (inside a block)
//        = X + sum_{i >= t} (q_i.dq_i - k_i.dk_i),
//   X = e^{L_end} <S, G> + sum_j k_j.dk_j(G part),
// so it needs the row dots that the dq and dk passes have at hand.
//
// The products run on mma.sync tf32 (scores of bf16 inputs: bf16, exact). bf16
// values are exact in tf32; an fp32 operand is split in two tf32 parts (22 bits)
// where its error would reach an fp32 output, and kept as one part (11 bits,
// against the 8 of the bf16 output) where it would not. Accumulators, states and sums are fp32.
#include <math_constants.h>

#include <algorithm>

#include "kda_linear.cuh"
#include "kda_linear_tc.cuh"

namespace kda {
namespace {

constexpr int NT = 256;  // threads of the three main kernels
constexpr int CH = kLinChunk;

// The segment length where the state is carried along inside (lin_roll_tc): a
// function of the sequence's own length and the heads, so that a sequence gives
// the same bits alone and in any batch. A segment costs its 128-token chunks and
// about two more (its first state, its share of the scan), so short ones pay for
// being many; long ones leave a small batch on few of the 152 SMs, so one
// sequence is cut into at least 64 (or into the shortest). bf16, d = 128:
//   4 x 4096 tokens x 16 heads: 512 136 us, 1024 123, 2048 117;
//   1 x 16384 x 2: 512 41, 1024 61; 1 x 65536 x 1: 1024 68, 2048 105;
//   16 sequences of 20011 tokens in all x 16: 512 172, by this rule 171-175.
constexpr int kLeastSegment = 512;
__host__ __device__ constexpr int segment_tokens(int64_t len, int H) {
    int n = len <= 2048 ? kLeastSegment : len <= 16384 ? 1024 : len <= 65536 ? 2048 : kLongestSegment;
    while (n > kLeastSegment && (int64_t)n * 64 > len * H) n /= 2;
    return n;
}

// ---------------------------------------------------------------- packed batches: the table of blocks
// sb = 0: segments of segment_tokens(length).
constexpr int kPrepThreads = 1024;
__global__ void __launch_bounds__(kPrepThreads)
lin_blocks_kernel(const int32_t *cu, int N, int T_total, int H, int sb, int nblocks, int4 *blocks,
                  int32_t *seq_block, int32_t *place, int32_t *status, int32_t *user_status) {
    constexpr int kBuckets = 66;
    __shared__ int bad;
    __shared__ int wsum[kPrepThreads / 32], count[kBuckets];
    auto bucket = [](int len) { return min((len + 63) / 64, kBuckets - 1); };
    if (threadIdx.x < kBuckets) count[threadIdx.x] = 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = (cu[0] != 0 || cu[N] != T_total) ? 1 : 0;
    __syncthreads();
    for (int i = tid; i < N; i += kPrepThreads)
        if (cu[i + 1] < cu[i] || cu[i] < 0 || cu[i + 1] > T_total) atomicOr(&bad, 1);
    __syncthreads();
    const bool b = bad != 0;
    if (tid == 0) {
        *status = b ? KDA_DEV_BAD_CU_SEQLENS : KDA_DEV_OK;
        if (user_status) *user_status = *status;
        seq_block[0] = 0;
    }
    int base = 0;
    for (int i0 = 0; i0 < N; i0 += kPrepThreads) {
        const int i = i0 + tid;
        int x = 0;
        if (i < N && !b) {
            const int len = cu[i + 1] - cu[i], per = sb ? sb : segment_tokens(len, H);
            x = (len + per - 1) / per;
        }
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
        if (i < N) seq_block[i + 1] = before + x;
        base = all;
        __syncthreads();
    }
    __threadfence_block();
    __syncthreads();
    auto entry = [&](int j) {
        if (j >= base) return make_int4(0, 0, 0, 0);
        int lo = 0, hi = N - 1;  // the last sequence whose first block is <= j
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (seq_block[m] <= j) lo = m;
            else hi = m - 1;
        }
        const int per = sb ? sb : segment_tokens(cu[lo + 1] - cu[lo], H);
        const int start = cu[lo] + (j - seq_block[lo]) * per;
        return make_int4(lo, start, min(per, cu[lo + 1] - start), 0);
    };
    if (!place) {
        for (int j = tid; j < nblocks; j += kPrepThreads) blocks[j] = entry(j);
        return;
    }
    // Segments of unequal lengths, longest first (to 64 tokens): dealt out in
    // turn they end at about the same time (16 sequences, 20011 tokens in all,
    // 16 heads: 180-211 us in the order of the batch, 171-175 so).
    // Where one stands among its equals is left to chance and changes no result.
    for (int j = tid; j < nblocks; j += kPrepThreads) atomicAdd(count + bucket(entry(j).z), 1);
    __syncthreads();
    if (tid == 0) {
        int at = 0;
        for (int k = kBuckets - 1; k >= 0; --k) {
            const int n = count[k];
            count[k] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int j = tid; j < nblocks; j += kPrepThreads) {
        const int4 e = entry(j);
        const int at = atomicAdd(count + bucket(e.z), 1);
        blocks[at] = e;
        place[j] = at;
    }
}

// ---------------------------------------------------------------- warp products
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
// acc[m][n] (16 x 8 tiles at rows r0 + 16 m, columns c0 + 8 n) += sum_k a(r, k) b(k, c).
// SA, SB: the operand is split in two tf32 parts (the product of the two low
// parts, 2^-22 of the whole, is left out). The tensor core cuts its sums off
// where a CUDA core rounds them, which over K / 8 steps in one accumulator cost
// 1.7e-6 to 4e-6 in the results; so with a split operand each step's products
// are summed from zero and added to the accumulator in fp32.
// TA, TB: the operand is exact in tf32 as it is (a bf16 value).
template <int K, int MT, int NT8, bool SA, bool SB, bool TA, bool TB, typename FA, typename FB>
__device__ __forceinline__ void product(float (&acc)[MT][NT8][4], FA a, FB b, int r0, int c0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 2
    for (int k = 0; k < K; k += 8) {
        uint32_t ah[MT][4], al[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = r0 + 16 * m + g;
            const float x[4] = {a(r, k + t), a(r + 8, k + t), a(r, k + t + 4), a(r + 8, k + t + 4)};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                ah[m][u] = TA ? __float_as_uint(x[u]) : tf32(x[u]);
                if (SA) al[m][u] = tf32(x[u] - __uint_as_float(ah[m][u]));
            }
        }
#pragma unroll
        for (int n = 0; n < NT8; ++n) {
            const float x0 = b(k + t, c0 + 8 * n + g), x1 = b(k + t + 4, c0 + 8 * n + g);
            const uint32_t h0 = TB ? __float_as_uint(x0) : tf32(x0), h1 = TB ? __float_as_uint(x1) : tf32(x1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (!SA && !SB) {
                    mma_tf32(acc[m][n], ah[m], h0, h1);
                    continue;
                }
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                if (SA) mma_tf32(d, al[m], h0, h1);
                if (SB) mma_tf32(d, ah[m], tf32(x0 - __uint_as_float(h0)), tf32(x1 - __uint_as_float(h1)));
                mma_tf32(d, ah[m], h0, h1);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][n][e] += d[e];
            }
        }
    }
}

// acc[n] += x_r . y_c over K channels, both [row][K] in shared memory with leading
// dimension ld: bf16 products, exact, 16 channels an instruction and two a load
// (as tf32 the same scores took a load and a conversion an element).
template <int K, int NT8>
__device__ __forceinline__ void row_products(float (&acc)[1][NT8][4], const __nv_bfloat16 *x, const __nv_bfloat16 *y,
                                             int ld, int r0, int c0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    auto two = [&](const __nv_bfloat16 *p, int row, int k) {
        return *reinterpret_cast<const uint32_t *>(p + row * ld + k + 2 * t);
    };
#pragma unroll 2
    for (int k = 0; k < K; k += 16) {
        const uint32_t a[4] = {two(x, r0 + g, k), two(x, r0 + g + 8, k), two(x, r0 + g, k + 8), two(x, r0 + g + 8, k + 8)};
#pragma unroll
        for (int n = 0; n < NT8; ++n) {
            float(&d)[4] = acc[0][n];
            asm volatile(
                "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                "{%0,%1,%2,%3};"
                : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(two(y, c0 + 8 * n + g, k)),
                  "r"(two(y, c0 + 8 * n + g, k + 8)));
        }
    }
}

// Global to shared memory without waiting (joined by loads_done); `bytes` short
// of the size: the rest is zero.
template <int SIZE> __device__ __forceinline__ void load_async(void *dst, const void *src, int bytes) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void loads_done() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
}
// Rows of a [64][D] tile into shared memory; rows past `rows` are zero.
template <typename T, int D>
__device__ __forceinline__ void load_tile(T *dst, int ld, const T *src, int64_t stride, int rows) {
    constexpr int V = 16 / sizeof(T), PER = D / V;
    for (int i = threadIdx.x; i < CH * PER; i += NT) {
        const int r = i / PER, c = (i % PER) * V;
        load_async<16>(dst + r * ld + c, src + min(r, rows - 1) * stride + c, r < rows ? 16 : 0);
    }
}
// Leading dimensions that keep the fragment reads free of bank conflicts:
// rows across lanes (A, or B stored [n][k]) and rows along k (B stored [k][n]).
template <typename T> __host__ __device__ constexpr int ld_rows(int d) { return sizeof(T) == 2 ? d + 8 : d + 4; }
template <typename T> __host__ __device__ constexpr int ld_cols(int d) { return d + 8; }

// ---------------------------------------------------------------- a block's own state
// out[block][head] = sum_s w_s x_s y_s^T over the block's tokens: forward
// w_s = e^{L_end - L_s} with (x, y) = (k, v); reverse w_s = e^{L_s} with
// (q, do). Also e^{L_end} of the block (forward). Bound by latency at the sizes
// that this path is for: a load of the tiles and the decays (all in flight at
// once), one 64-token product, one store. 2 x 999 tokens x 4 heads, fp32, 64 x 128,
// both directions: 256 CTAs, 11 us on cold caches.
template <typename T> struct StateArgs {
    LinGeom geo;
    const T *x, *y;
    int64_t x_stride, y_stride;
    const float *log_decay;
    int decay;
    float *out, *total, *total_rev;  // the block's decay_total as the forward and as the reverse scan use it, nullable
};
template <typename T, int DK, int DV, bool REV> __device__ __forceinline__ void block_state(const StateArgs<T> &p) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int WM = DK / 32, WN = NT / 32 / WM, COLS = DV / WN, N8 = COLS / 8;
    constexpr int LDX = ld_cols<T>(DK), LDY = ld_cols<T>(DV);
    extern __shared__ __align__(16) unsigned char smem[];
    T *xs = reinterpret_cast<T *>(smem);
    T *ys = xs + CH * LDX;
    float2 *a = reinterpret_cast<float2 *>(ys + CH * LDY);
    __shared__ long long scan[NT / 32];
    __shared__ DecayEvents events;
    __shared__ float w[CH];
    const LinGeom &geo = p.geo;
    const int b = blockIdx.x / geo.H, h = blockIdx.x % geo.H;
    const LinBlock blk = lin_block<true>(geo, b);
    if (blk.len <= 0) return;
    load_tile<T, DK>(xs, LDX, p.x + blk.start * p.x_stride + h * DK, p.x_stride, blk.len);
    load_tile<T, DV>(ys, LDY, p.y + blk.start * p.y_stride + h * DV, p.y_stride, blk.len);
    const long long sum =
        decay_prefix<NT>(p.log_decay, p.decay, blk.start, geo.H, h, blk.len, blk.len, a, scan, &events);
    const float2 end = a[blk.len];
    if (threadIdx.x == 0) {
        const int64_t at = (int64_t)b * geo.H + h;
        const float total = decay_total(sum);
        if (p.total) p.total[at] = events.nan_before(blk.len - 1) ? CUDART_NAN_F : total;
        if (p.total_rev) p.total_rev[at] = events.nan_after(-1) ? CUDART_NAN_F : total;
    }
    if (threadIdx.x < CH) {
        const int s = min((int)threadIdx.x, blk.len - 1);
        w[threadIdx.x] = REV ? decay_ratio(a[s + 1], make_float2(0.f, 0.f)) : decay_ratio(end, a[s + 1]);
    }
    loads_done();
    const int warp = threadIdx.x >> 5, r0 = (warp % WM) * 32, c0 = (warp / WM) * COLS;
    float acc[2][N8][4] = {};
    product<CH, 2, N8, true, F32, false, !F32>(
        acc, [&](int r, int k) { return to_f32(xs[k * LDX + r]) * w[k]; },
        [&](int k, int c) { return to_f32(ys[k * LDY + c]); }, r0, c0);
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float *dst = p.out + ((int64_t)b * geo.H + h) * DK * DV;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < N8; ++n) {
            const int r = r0 + 16 * m + g, c = c0 + 8 * n + 2 * t;
            *reinterpret_cast<float2 *>(dst + r * DV + c) = make_float2(acc[m][n][0], acc[m][n][1]);
            *reinterpret_cast<float2 *>(dst + (r + 8) * DV + c) = make_float2(acc[m][n][2], acc[m][n][3]);
        }
}

// The backward needs both directions and neither fills the GPU: one launch.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(NT) lin_state_kernel(const StateArgs<T> fwd, const StateArgs<T> rev) {
    after_previous();
    if (blockIdx.y == 0) block_state<T, DK, DV, false>(fwd);
    else block_state<T, DK, DV, true>(rev);
}

// ---------------------------------------------------------------- joining the blocks
// In place, along each (sequence, head): forward, every block's own sum gives
// way to the state before the block, S <- e^{L_end} S + c own, and the last S
// is the final state; reverse, to the gradient of the state after the block.
// Elementwise over the state: one float4 per thread, the blocks in turn, four
// loads ahead, with the errors of its sums (ScanElements). Bound by memory, or by the latency of a turn where the sequences
// are few and long: 4 x 4096 tokens x 16 heads in segments of 1024, 8-10 us;
// 131072 x 32 in segments of 4096 (67 MB each way), 18 us, 7.5 TB/s (L2 helps).
struct ScanArgs {
    float *states;
    const float *s0;  // nullable
    float *sT;        // nullable
    float c;
    const float *total;  // every block's decay_total
};
template <bool REV>
__device__ __forceinline__ void scan_blocks(const LinGeom &geo, const ScanArgs &q, int size4) {
    const float c = q.c;
    const float *total = q.total;
    if (geo.status && *geo.status != KDA_DEV_OK) return;
    const int per = size4 / NT;
    const int64_t nh = blockIdx.x / per;
    const int n = (int)(nh / geo.H), h = (int)(nh % geo.H);
    const int64_t e = (int64_t)(blockIdx.x % per) * NT + threadIdx.x;
    int first, last;
    lin_seq_blocks<true>(geo, n, first, last);
    ScanElements S(q.s0 ? reinterpret_cast<const float4 *>(q.s0)[nh * size4 + e] : make_float4(0.f, 0.f, 0.f, 0.f));
    float4 *p = reinterpret_cast<float4 *>(q.states);
    const int count = last - first;
    constexpr int AHEAD = 4;
    float4 own[AHEAD];
    float f[AHEAD];
    auto at = [&](int i) {
        const int b = REV ? last - 1 - i : first + i;
        return (int64_t)(geo.place ? geo.place[b] : b) * geo.H + h;
    };
    for (int i0 = 0; i0 < count; i0 += AHEAD) {
        float4 *dst[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i0 + u < count) {
                dst[u] = p + at(i0 + u) * size4 + e;
                own[u] = *dst[u];
                f[u] = total[at(i0 + u)];
            }
        if (S.finite(own, f, count - i0)) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (i0 + u < count) {
                    *dst[u] = S.value();
                    S.step(f[u], c, own[u]);
                }
        } else {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (i0 + u < count) {
                    *dst[u] = S.value();
                    S.step_any(f[u], c, own[u]);
                }
        }
    }
    if (q.sT) reinterpret_cast<float4 *>(q.sT)[nh * size4 + e] = S.value();
}

// The backward's two directions do not depend on each other: one launch (blockIdx.y).
__global__ void __launch_bounds__(NT)
lin_scan_kernel(const LinGeom geo, const ScanArgs fwd, const ScanArgs rev, int size4) {
    after_previous();
    if (blockIdx.y == 0) {
        if (fwd.states) scan_blocks<false>(geo, fwd, size4);
    } else {
        scan_blocks<true>(geo, rev, size4);
    }
}

// ---------------------------------------------------------------- outputs
struct AttendArgs {
    LinGeom geo;
    const void *x, *y, *z;  // the query, key and value roles
    int64_t x_stride, y_stride, z_stride;
    const float *log_decay;
    int decay;
    const float *states;    // [block][head][d_k][d_v]: before the block, or (reverse) its gradient after it
    void *out;              // [tokens][H][DO]
    float c_state, c_intra;
    // row dots with `w` (the role tensor of the output's own operand), or null
    const void *w;
    int64_t w_stride;
    float *dot, *dot_state;  // [tokens][H]: w_i . out_i before rounding, and of its state part
};

// out_i = c_state f_i x_i S + c_intra sum_j D_ij (x_i . y_j) z_j over the
// tokens j <= i of the block (reverse: j >= i); S is [DC][DO], or stored
// [DO][DC] and read transposed (ST).
// EXACT: the fp32 operands P and S are split too, for the row dots.
// Bound by latency and, in fp32, by the three products of every split operand.
// Everything a block reads is in flight at once; P takes the place of x and y,
// which leaves room for two CTAs on an SM. 2 x 999 tokens x 4 heads, fp32, 64 x 128:
// the backward's three passes took 85 us as launches of their own, with loads
// and products in turn; the whole backward went from 102 to 63 us (66 since the
// scan carries its rounding along).
// In bf16 bound by instructions (8 x 2048 tokens x 16 heads, 64 x 64: 72 % of the
// issue slots, mostly loads of single values and conversions): 154 us for the
// whole forward, 137 with the scores as bf16 products and no conversions of
// values that are exact as they are.
template <typename T, int DC, int DO> constexpr size_t attend_smem() {
    return 2 * CH * ld_rows<T>(DC) * sizeof(T) + CH * (DO + 8) * 4 + CH * ld_cols<T>(DO) * sizeof(T) + (CH + 1) * 8;
}
template <typename T, int DC, int DO, bool REV, bool ST, bool EXACT>
__device__ __forceinline__ void attend_block(const AttendArgs &p) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int LDX = ld_rows<T>(DC), LDZ = ld_cols<T>(DO), LDS = DO + 8, LDP = CH + 4, N8 = DO / 16;
    static_assert(CH * LDP * 4 <= 2 * CH * LDX * (int)sizeof(T), "P takes the place of x and y");
    extern __shared__ __align__(16) unsigned char smem[];
    T *xs = reinterpret_cast<T *>(smem);
    T *ys = xs + CH * LDX;
    float *ps = reinterpret_cast<float *>(smem);
    float *ss = reinterpret_cast<float *>(ys + CH * LDX);  // a 64-row piece of the state
    T *zs = reinterpret_cast<T *>(ss + CH * LDS);
    float2 *a = reinterpret_cast<float2 *>(zs + CH * LDZ);
    __shared__ long long scan[NT / 32];
    __shared__ DecayEvents events;
    __shared__ float dots[2][2][CH];
    const LinGeom &geo = p.geo;
    const int h = blockIdx.x % geo.H, b = blockIdx.x / geo.H;
    const LinBlock blk = lin_block<true>(geo, b);
    const int len = blk.len;
    if (len <= 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int r0 = (warp & 3) * 16, half = warp >> 2, c0 = half * (DO / 2), s0 = half * 32;
    const int64_t tok = blk.start;
    const float *S = p.states + ((int64_t)b * geo.H + h) * DC * DO;
    auto load_state = [&](int k0) {
        if (!ST) {
            for (int i = threadIdx.x; i < CH * DO / 4; i += NT) {
                const int r = i / (DO / 4), c = (i % (DO / 4)) * 4;
                load_async<16>(ss + r * LDS + c, S + (int64_t)(k0 + r) * DO + c, 16);
            }
        } else {
            for (int i = threadIdx.x; i < CH * DO; i += NT) {
                const int r = i % CH, c = i / CH;
                load_async<4>(ss + r * LDS + c, S + (int64_t)c * DC + k0 + r, 4);
            }
        }
    };
    load_tile<T, DC>(xs, LDX, (const T *)p.x + tok * p.x_stride + h * DC, p.x_stride, len);
    load_state(0);
    load_tile<T, DC>(ys, LDX, (const T *)p.y + tok * p.y_stride + h * DC, p.y_stride, len);
    load_tile<T, DO>(zs, LDZ, (const T *)p.z + tok * p.z_stride + h * DO, p.z_stride, len);
    decay_prefix<NT>(p.log_decay, p.decay, blk.start, geo.H, h, len, len, a, scan, &events);
    loads_done();

    // the state part, 64 rows of the contraction at a time, and the scores
    float acc[1][N8][4] = {}, sc[1][4][4] = {};
    auto state_part = [&](int k0) {
        product<CH, 1, N8, F32, EXACT, !F32, false>(
            acc, [&](int r, int k) { return to_f32(xs[r * LDX + k0 + k]); },
            [&](int k, int c) { return ss[k * LDS + c]; }, r0, c0);
    };
    state_part(0);
    if (DC > CH) {
        __syncthreads();
        load_state(CH);
    }
    if constexpr (F32)
        product<DC, 1, 4, true, true, false, false>(
            sc, [&](int r, int k) { return xs[r * LDX + k]; }, [&](int k, int c) { return ys[c * LDX + k]; }, r0, s0);
    else
        row_products<DC, 4>(sc, xs, ys, LDX, r0, s0);
    if (DC > CH) {
        loads_done();
        state_part(CH);
    }
    __syncthreads();  // x and y are read: P may take their place
    auto row_dots = [&](float *dst) {  // w_i . acc_i over this warp's columns
        float d[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = r0 + g + 8 * e;
            if (r < len) {
                const T *w = (const T *)p.w + (tok + r) * p.w_stride + h * DO;
#pragma unroll
                for (int n = 0; n < N8; ++n) {
                    const int c = c0 + 8 * n + 2 * t;
                    d[e] += to_f32(w[c]) * acc[0][n][2 * e] + to_f32(w[c + 1]) * acc[0][n][2 * e + 1];
                }
            }
            d[e] += __shfl_xor_sync(0xffffffffu, d[e], 1);
            d[e] += __shfl_xor_sync(0xffffffffu, d[e], 2);
            if (t == 0) dst[r] = d[e];
        }
    };
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = min(r0 + g + 8 * e, len - 1);
        float f = p.c_state * (REV ? decay_ratio(a[len], a[i + 1]) : decay_ratio(a[i + 1], make_float2(0.f, 0.f)));
        if (REV ? events.nan_after(i) : events.nan_before(i)) f = CUDART_NAN_F;
#pragma unroll
        for (int n = 0; n < N8; ++n) {
            acc[0][n][2 * e] = f == 0.f ? 0.f : acc[0][n][2 * e] * f;  // a reset, whatever the state held
            acc[0][n][2 * e + 1] = f == 0.f ? 0.f : acc[0][n][2 * e + 1] * f;
        }
    }
    if (p.dot_state) row_dots(dots[0][half]);

    // the block's own tokens
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = r0 + g + 8 * (e >> 1), j = s0 + 8 * n + 2 * t + (e & 1);
            float v = 0.f;  // chosen, not multiplied: what lies past the end may be anything
            if (i < len && j < len && (REV ? j >= i : j <= i))
                v = p.c_intra * sc[0][n][e] * (REV ? decay_ratio(a[j + 1], a[i + 1]) : decay_ratio(a[i + 1], a[j + 1]));
            ps[i * LDP + j] = v;
        }
    __syncthreads();
    product<CH, 1, N8, EXACT, F32, false, !F32>(
        acc, [&](int r, int k) { return ps[r * LDP + k]; },
        [&](int k, int c) { return to_f32(zs[k * LDZ + c]); }, r0, c0);
    if (p.dot) row_dots(dots[1][half]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = r0 + g + 8 * e;
        if (r >= len) continue;
        T *o = (T *)p.out + ((tok + r) * geo.H + h) * DO;
#pragma unroll
        for (int n = 0; n < N8; ++n) {
            const int c = c0 + 8 * n + 2 * t;
            if (F32)
                *reinterpret_cast<float2 *>(o + c) = make_float2(acc[0][n][2 * e], acc[0][n][2 * e + 1]);
            else
                *reinterpret_cast<__nv_bfloat162 *>(o + c) =
                    __floats2bfloat162_rn(acc[0][n][2 * e], acc[0][n][2 * e + 1]);
        }
    }
    if (p.dot) {
        __syncthreads();
        if ((int)threadIdx.x < len) {
            const int64_t i = (tok + threadIdx.x) * geo.H + h;
            p.dot[i] = dots[1][0][threadIdx.x] + dots[1][1][threadIdx.x];
            if (p.dot_state) p.dot_state[i] = dots[0][0][threadIdx.x] + dots[0][1][threadIdx.x];
        }
    }
}

template <typename T, int DK, int DV> __global__ void __launch_bounds__(NT) lin_attend_kernel(const AttendArgs p) {
    after_previous();
    attend_block<T, DK, DV, false, false, sizeof(T) == 4>(p);
}
// The backward's three passes, each too small for the GPU, in one launch, the
// longest first. EXACT: for the row dots.
template <typename T, int DK, int DV, bool EXACT>
__global__ void __launch_bounds__(NT)
lin_attend_back_kernel(const AttendArgs dk, const AttendArgs dq, const AttendArgs dv) {
    after_previous();
    if (blockIdx.y == 0) attend_block<T, DV, DK, true, true, EXACT>(dk);
    else if (blockIdx.y == 1) attend_block<T, DV, DK, false, true, EXACT>(dq);
    else attend_block<T, DK, DV, true, false, sizeof(T) == 4>(dv);
}

// ---------------------------------------------------------------- gradient of the log decay
// Per block and head: dg_t = X + sum_{i >= t} (qdq_i - kdk_i), with
// X = e^{L_end} <S, G> + sum_j kdk_state_j. A reset (log decay at or below the
// clamp) passes nothing on: its gradient is zero, not the sum's rounding.
__global__ void __launch_bounds__(NT)
lin_decay_grad_kernel(LinGeom geo, const float *log_decay, int decay, const float *states,
                      const float *grads, const float *inner,
                      const float *total, int size4,
                      const float *qdq, const float *kdk,
                      const float *kdk_state, int64_t dot_stride, float *dg,
                      float *block_sum) {
    after_previous();
    __shared__ float red[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / geo.H, h = blockIdx.x % geo.H;
    const LinBlock blk = lin_block<true>(geo, b);
    const int64_t bh = (int64_t)b * geo.H + h;
    auto block_add = [&](float v) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        __syncthreads();
        if (lane == 0) red[warp] = v;
        __syncthreads();
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) s += red[w];
        return s;
    };
    if (blk.len <= 0) {
        if (block_sum && tid == 0) block_sum[bh] = 0.f;
        return;
    }
    float x = 0.f;
    if (inner) {  // <S, G> already summed up to kScanPartials pieces
        if (tid < kScanPartials) x = inner[bh * kScanPartials + tid];
    } else {
        const float4 *S = reinterpret_cast<const float4 *>(states) + bh * size4;
        const float4 *G = reinterpret_cast<const float4 *>(grads) + bh * size4;
        for (int i = tid; i < size4; i += NT) {
            const float4 s = S[i], g = G[i];
            x += s.x * g.x + s.y * g.y + s.z * g.z + s.w * g.w;
        }
    }
    x = decay_times(total[bh], x);
    for (int i = tid; i < blk.len; i += NT) {
        const int64_t at = (int64_t)(blk.start + i) * geo.H + h;
        x += kdk_state[at] + (dot_stride ? kdk_state[at + dot_stride] : 0.f);
    }
    float run = block_add(x), sum = 0.f;
    for (int i1 = (blk.len + NT - 1) / NT * NT; i1 > 0; i1 -= NT) {  // from the end, thread tid at i1 - 1 - tid
        const int i = i1 - 1 - tid;
        const int64_t at = (int64_t)(blk.start + i) * geo.H + h;
        float v = 0.f;
        if (i < blk.len) {
            v = qdq[at] - kdk[at];
            if (dot_stride) v += qdq[at + dot_stride] - kdk[at + dot_stride];
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += y;
        }
        __syncthreads();
        if (lane == 31) red[warp] = v;
        __syncthreads();
        float before = run, all = run;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) before += red[w];
            all += red[w];
        }
        if (i < blk.len) {
            const float lg = decay == KDA_DECAY_HEAD ? log_decay[h] : log_decay[at];
            const float d = lg <= kMinLogDecay ? 0.f : before + v;
            if (dg) dg[at] = d;
            sum += d;
        }
        run = all;
    }
    if (block_sum) {
        const float s = block_add(sum);
        if (tid == 0) block_sum[bh] = s;
    }
}

// One decay per head: its gradient is the sum over every token, in block order.
__global__ void __launch_bounds__(NT)
lin_head_sum_kernel(LinGeom geo, const float *block_sum, float *dg) {
    after_previous();
    __shared__ float red[NT];
    if (geo.status && *geo.status != KDA_DEV_OK) return;
    const int h = blockIdx.x;
    float s = 0.f;
    for (int b = threadIdx.x; b < geo.nblocks; b += NT) s += block_sum[(int64_t)b * geo.H + h];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int n = NT / 2; n > 0; n >>= 1) {
        if ((int)threadIdx.x < n) red[threadIdx.x] += red[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[h] = red[0];
}

__global__ void lin_status_kernel(int32_t *status, int value) { *status = value; }

// ---------------------------------------------------------------- host side
size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The block length of the general kernels: one chunk a block gives the most
// blocks at once (257 tokens x 2 heads, fp32, d = 64: the call took 34.5 us in
// blocks of 64, 53.8 in blocks of 256). One length for all, so that a sequence
// gives the same bits in any batch.
constexpr int kGeneralBlock = CH;

int64_t max_blocks(int N, int64_t T, bool packed, int sb) {
    return packed ? T / sb + N : (int64_t)N * ((T + sb - 1) / sb);
}

struct Plan {
    LinGeom geo;
    int4 *blocks;
    int32_t *seq_block, *status, *place;
    float *total, *total_rev, *states, *grads, *qdq, *kdk, *kdk_state, *block_sum;
    __nv_bfloat16 *s_parts, *g_parts;  // tensor-core path: the joined states as bf16 parts
    float *inner;                      // and <S, G> of every block, in pieces
    int64_t part_stride, dot_stride;
    size_t bytes;
};
bool use_tc(kda_dtype_t dt, int dk, int dv) { return dt == KDA_BF16 && dk == 128 && dv == 128; }
// `rolled`: the tensor-core path with the state carried along inside segments
// (the forward, and the backward without the decay's gradient).
Plan make_plan(int N, int64_t T, int H, int dk, int dv, kda_dtype_t dt, bool packed, bool back, bool rolled, void *ws) {
    Plan p{};
    const int64_t tokens = packed ? T : N * T;
    const bool tc = use_tc(dt, dk, dv);
    const int sb = !tc ? kGeneralBlock : !rolled ? kLinMaxBlock : packed ? kLeastSegment : segment_tokens(T, H);
    const int64_t nb = max_blocks(N, T, packed, sb);
    unsigned char *base = static_cast<unsigned char *>(ws);
    size_t at = 0;
    auto take = [&](size_t n) {
        void *r = base ? base + at : nullptr;
        at += up(n);
        return r;
    };
    if (packed) {
        p.status = (int32_t *)take(4);
        p.seq_block = (int32_t *)take(4 * ((size_t)N + 1));
        p.blocks = (int4 *)take(16 * (size_t)nb);
        if (rolled) p.place = (int32_t *)take(4 * (size_t)nb);
    }
    const size_t state = (size_t)nb * H * dk * dv * 4;
    p.total = (float *)take((size_t)nb * H * 4);
    if (back) p.total_rev = (float *)take((size_t)nb * H * 4);
    p.states = (float *)take(state);
    p.part_stride = nb * H * dk * dv;
    if (back && (!tc || rolled)) p.grads = (float *)take(state);
    if (back && tc && !rolled) {
        p.s_parts = (__nv_bfloat16 *)take(state / 2 * 3);
        p.g_parts = (__nv_bfloat16 *)take(state / 2 * 3);
        p.inner = (float *)take((size_t)nb * H * kScanPartials * 4);
    }
    if (back && !rolled) {
        const size_t halves = tc ? 2 : 1;  // row dots come in so many pieces
        p.dot_stride = tc ? tokens * H : 0;
        p.qdq = (float *)take(halves * tokens * H * 4);
        p.kdk = (float *)take(halves * tokens * H * 4);
        p.kdk_state = (float *)take(halves * tokens * H * 4);
        p.block_sum = (float *)take((size_t)nb * H * 4);
    }
    p.bytes = at;
    p.geo = {p.blocks, p.seq_block, p.status, p.place, N, (int)T, H, sb,
             (int)((T + sb - 1) / sb), (int)nb, FastDiv(H),
             FastDiv((uint32_t)std::max<int64_t>(1, (T + sb - 1) / sb))};
    if (!packed) p.geo.blocks = nullptr, p.geo.seq_block = nullptr, p.geo.status = nullptr;
    return p;
}

#define KDA_TRY(x)                              \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

// One direction (`back` false: the forward's) or both.
template <typename T, int DK, int DV>
cudaError_t run_states(const Plan &p, const LinArgs &a, bool back, Launches &l) {
    constexpr size_t smem = CH * (ld_cols<T>(DK) + ld_cols<T>(DV)) * sizeof(T) + (CH + 1) * sizeof(float2);
    auto k = lin_state_kernel<T, DK, DV>;
    static std::atomic<uint64_t> allowed{0};
    KDA_TRY(allow_smem(k, smem, allowed));
    const StateArgs<T> f{p.geo, (const T *)a.k, (const T *)a.v, a.k_stride, a.v_stride, a.log_decay, a.decay, p.states,
                         p.total, p.total_rev};
    const StateArgs<T> r{p.geo, (const T *)a.q, (const T *)a.d_o, a.q_stride, (int64_t)a.H * DV, a.log_decay, a.decay,
                         p.grads, nullptr, nullptr};
    const dim3 grid((unsigned)((int64_t)p.geo.nblocks * p.geo.H), back ? 2 : 1);
    return l.next(k, grid, NT, smem, f, r);
}
// `rev` null: forward alone.
cudaError_t run_scan(const Plan &p, const ScanArgs &fwd, const ScanArgs *rev, int dk, int dv, Launches &l) {
    const int size4 = dk * dv / 4;
    const dim3 grid((unsigned)((int64_t)p.geo.N * p.geo.H * (size4 / NT)), rev ? 2 : 1);
    return l.next(lin_scan_kernel, grid, NT, 0, p.geo, fwd, rev ? *rev : ScanArgs{}, size4);
}

cudaError_t prepare_blocks(const Plan &p, const LinArgs &a, bool rolled, Launches &l) {
    if (!a.cu_seqlens) return cudaSuccess;
    return l.next(lin_blocks_kernel, 1, kPrepThreads, 0, a.cu_seqlens, a.N, a.T, a.H, rolled ? 0 : p.geo.sb, p.geo.nblocks,
             p.blocks, p.seq_block, p.place, p.status, a.status);
}

// bf16, d_k = d_v = 128: the same steps on the tensor cores.
cudaError_t forward_tc(const LinArgs &a, cudaStream_t s) {
    Launches l{s};
    const Plan p = make_plan(a.N, a.T, a.H, 128, 128, a.dt, a.cu_seqlens != nullptr, false, use_tc(a.dt, a.dk, a.dv), a.workspace);
    const int64_t tokens = a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    KDA_TRY(prepare_blocks(p, a, true, l));
    // one segment a sequence and no final state asked for: the first states are all there is
    const bool need_states = a.sT || a.cu_seqlens || p.geo.per_seq > 1;
    if (tokens > 0 && need_states)
        KDA_TRY(launch_state_tc(p.geo, false, a.k, a.k_stride, a.v, a.v_stride, tokens, a.log_decay, a.decay, p.states,
                                p.total, nullptr, l));
    KDA_TRY(run_scan(p, {p.states, a.s0, a.sT, 1.f, p.total}, nullptr, 128, 128, l));
    if (tokens == 0) return cudaSuccess;
    RollTc t{};
    t.geo = p.geo;
    t.x = a.q; t.y = a.k; t.z = a.v;
    t.x_stride = a.q_stride; t.y_stride = a.k_stride; t.z_stride = a.v_stride;
    t.states = p.states; t.tokens = tokens;
    t.log_decay = a.log_decay; t.decay = a.decay;
    t.out = a.o; t.c_state = a.scale; t.c_intra = a.scale; t.c_roll = 1.f;
    return launch_roll_tc(t, l);
}

// Backward without the decay's gradient: three passes with the state carried along.
cudaError_t backward_rolled_tc(const LinArgs &a, cudaStream_t s) {
    Launches l{s};
    constexpr bool rolled = true;
    const Plan p = make_plan(a.N, a.T, a.H, 128, 128, a.dt, a.cu_seqlens != nullptr, true, rolled, a.workspace);
    const int64_t tokens = a.cu_seqlens ? a.T : (int64_t)a.N * a.T, so = (int64_t)a.H * 128;
    KDA_TRY(prepare_blocks(p, a, true, l));
    if (tokens > 0) {
        KDA_TRY(launch_state_tc(p.geo, false, a.k, a.k_stride, a.v, a.v_stride, tokens, a.log_decay, a.decay, p.states,
                                p.total, p.total_rev, l));
        KDA_TRY(launch_state_tc(p.geo, true, a.q, a.q_stride, a.d_o, so, tokens, a.log_decay, a.decay, p.grads,
                                nullptr, nullptr, l));
    }
    const ScanArgs grads{p.grads, a.dsT, a.ds0, a.scale, p.total_rev};
    KDA_TRY(run_scan(p, {p.states, a.s0, nullptr, 1.f, p.total}, &grads, 128, 128, l));
    if (tokens == 0) return cudaSuccess;
    RollTc t{};
    t.geo = p.geo;
    t.tokens = tokens;
    t.log_decay = a.log_decay; t.decay = a.decay;
    t.c_intra = a.scale;
    RollTc u = t;  // dq
    u.state_t = true;
    u.x = a.d_o; u.y = a.v; u.z = a.k;
    u.x_stride = so; u.y_stride = a.v_stride; u.z_stride = a.k_stride;
    u.states = p.states; u.out = a.dq; u.c_state = a.scale; u.c_roll = 1.f;
    KDA_TRY(launch_roll_tc(u, l));
    u = t;  // dk
    u.rev = u.state_t = true;
    u.x = a.v; u.y = a.d_o; u.z = a.q;
    u.x_stride = a.v_stride; u.y_stride = so; u.z_stride = a.q_stride;
    u.states = p.grads; u.out = a.dk_out; u.c_state = 1.f; u.c_roll = a.scale;
    KDA_TRY(launch_roll_tc(u, l));
    u = t;  // dv
    u.rev = true;
    u.x = a.k; u.y = a.q; u.z = a.d_o;
    u.x_stride = a.k_stride; u.y_stride = a.q_stride; u.z_stride = so;
    u.states = p.grads; u.out = a.dv_out; u.c_state = 1.f; u.c_roll = a.scale;
    return launch_roll_tc(u, l);
}

// Backward with the decay's gradient: blocks of kLinMaxBlock, every block's
// states in three bf16 parts, and the row dots.
cudaError_t backward_tc(const LinArgs &a, cudaStream_t s) {
    Launches l{s};
    constexpr bool rolled = false;
    const Plan p = make_plan(a.N, a.T, a.H, 128, 128, a.dt, a.cu_seqlens != nullptr, true, rolled, a.workspace);
    const int64_t tokens = a.cu_seqlens ? a.T : (int64_t)a.N * a.T, so = (int64_t)a.H * 128;
    const bool head = a.decay == KDA_DECAY_HEAD;
    KDA_TRY(prepare_blocks(p, a, false, l));
    if (tokens > 0) {
        KDA_TRY(launch_state_tc(p.geo, false, a.k, a.k_stride, a.v, a.v_stride, tokens, a.log_decay, a.decay, p.states,
                                p.total, p.total_rev, l));
        KDA_TRY(launch_scan_tc(p.geo, false, p.states, p.total, a.s0, nullptr, 1.f, p.s_parts, p.part_stride,
                               nullptr, nullptr, l));
        // the blocks' own sums of the states are done with: those of the gradients take their place
        KDA_TRY(launch_state_tc(p.geo, true, a.q, a.q_stride, a.d_o, so, tokens, a.log_decay, a.decay, p.states,
                                nullptr, nullptr, l));
    }
    KDA_TRY(launch_scan_tc(p.geo, true, p.states, p.total_rev, a.dsT, a.ds0, a.scale, p.g_parts, p.part_stride,
                           p.s_parts, p.inner, l));
    if (tokens == 0)
        return head ? cudaMemsetAsync(a.d_decay, 0, sizeof(float) * a.H, s) : cudaSuccess;
    AttendTc t{};
    t.geo = p.geo;
    t.tokens = tokens;
    t.log_decay = a.log_decay; t.decay = a.decay;
    t.c_intra = a.scale;
    AttendTc u = t;  // dv
    u.rev = true;
    u.x = a.k; u.y = a.q; u.z = a.d_o;
    u.x_stride = a.k_stride; u.y_stride = a.q_stride; u.z_stride = so;
    u.states = p.g_parts; u.out = a.dv_out; u.c_state = 1.f;
    KDA_TRY(launch_attend_tc(u, l));
    u = t;  // dq
    u.state_t = true;
    u.x = a.d_o; u.y = a.v; u.z = a.k; u.w = a.q;
    u.x_stride = so; u.y_stride = a.v_stride; u.z_stride = a.k_stride; u.w_stride = a.q_stride;
    u.states = p.s_parts; u.out = a.dq; u.c_state = a.scale;
    u.dot = p.qdq;
    KDA_TRY(launch_attend_tc(u, l));
    u = t;  // dk
    u.rev = u.state_t = true;
    u.x = a.v; u.y = a.d_o; u.z = a.q; u.w = a.k;
    u.x_stride = a.v_stride; u.y_stride = so; u.z_stride = a.q_stride; u.w_stride = a.k_stride;
    u.states = p.g_parts; u.out = a.dk_out; u.c_state = 1.f;
    u.dot = p.kdk;
    u.dot_state = p.kdk_state;
    KDA_TRY(launch_attend_tc(u, l));
    KDA_TRY(l.next(lin_decay_grad_kernel, (unsigned)((int64_t)p.geo.nblocks * a.H), NT, 0,
              p.geo, a.log_decay, a.decay, nullptr, nullptr, p.inner, p.total, 0, p.qdq, p.kdk, p.kdk_state, p.dot_stride,
        head ? nullptr : a.d_decay, head ? p.block_sum : nullptr));
    if (!head) return cudaSuccess;
    return l.next(lin_head_sum_kernel, a.H, NT, 0, p.geo, p.block_sum, a.d_decay);
}

template <typename T, int DK, int DV> cudaError_t forward(const LinArgs &a, cudaStream_t s) {
    Launches l{s};
    constexpr bool F32 = sizeof(T) == 4;
    const Plan p = make_plan(a.N, a.T, a.H, DK, DV, a.dt, a.cu_seqlens != nullptr, false, use_tc(a.dt, a.dk, a.dv), a.workspace);
    KDA_TRY(prepare_blocks(p, a, false, l));
    if (p.geo.nblocks > 0)
        KDA_TRY((run_states<T, DK, DV>(p, a, false, l)));
    KDA_TRY(run_scan(p, {p.states, a.s0, a.sT, 1.f, p.total}, nullptr, DK, DV, l));
    if (p.geo.nblocks == 0) return cudaSuccess;
    AttendArgs t{};
    t.geo = p.geo;
    t.x = a.q; t.y = a.k; t.z = a.v;
    t.x_stride = a.q_stride; t.y_stride = a.k_stride; t.z_stride = a.v_stride;
    t.log_decay = a.log_decay; t.decay = a.decay; t.states = p.states;
    t.out = a.o; t.c_state = a.scale; t.c_intra = a.scale;
    constexpr size_t smem = attend_smem<T, DK, DV>();
    auto k = lin_attend_kernel<T, DK, DV>;
    static std::atomic<uint64_t> allowed{0};
    KDA_TRY(allow_smem(k, smem, allowed));
    return l.next(k, (unsigned)((int64_t)p.geo.nblocks * a.H), NT, smem, t);
}

template <typename T, int DK, int DV, bool EXACT>
cudaError_t run_attend_back(const AttendArgs &dk, const AttendArgs &dq, const AttendArgs &dv, Launches &l) {
    constexpr size_t smem = std::max(attend_smem<T, DK, DV>(), attend_smem<T, DV, DK>());
    auto k = lin_attend_back_kernel<T, DK, DV, EXACT>;
    static std::atomic<uint64_t> allowed{0};
    KDA_TRY(allow_smem(k, smem, allowed));
    return l.next(k, dim3((unsigned)((int64_t)dk.geo.nblocks * dk.geo.H), 3), NT, smem, dk, dq, dv);
}
template <typename T, int DK, int DV> cudaError_t backward(const LinArgs &a, cudaStream_t s) {
    Launches l{s};
    constexpr bool rolled = false;
    const Plan p = make_plan(a.N, a.T, a.H, DK, DV, a.dt, a.cu_seqlens != nullptr, true, rolled, a.workspace);
    KDA_TRY(prepare_blocks(p, a, false, l));
    const int64_t so = (int64_t)a.H * DV;
    if (p.geo.nblocks > 0) KDA_TRY((run_states<T, DK, DV>(p, a, true, l)));
    const ScanArgs grads{p.grads, a.dsT, a.ds0, a.scale, p.total_rev};
    KDA_TRY(run_scan(p, {p.states, a.s0, nullptr, 1.f, p.total}, &grads, DK, DV, l));
    const bool dots = a.d_decay != nullptr, head = a.decay == KDA_DECAY_HEAD;
    if (p.geo.nblocks == 0) return dots && head ? cudaMemsetAsync(a.d_decay, 0, sizeof(float) * a.H, s) : cudaSuccess;
    AttendArgs t{};
    t.geo = p.geo;
    t.log_decay = a.log_decay; t.decay = a.decay;
    t.c_intra = a.scale;
    AttendArgs dv = t;  // keys attend, in reverse time, to the queries of later tokens
    dv.x = a.k; dv.y = a.q; dv.z = a.d_o;
    dv.x_stride = a.k_stride; dv.y_stride = a.q_stride; dv.z_stride = so;
    dv.states = p.grads; dv.out = a.dv_out; dv.c_state = 1.f;
    AttendArgs dq = t;
    dq.x = a.d_o; dq.y = a.v; dq.z = a.k;
    dq.x_stride = so; dq.y_stride = a.v_stride; dq.z_stride = a.k_stride;
    dq.states = p.states; dq.out = a.dq; dq.c_state = a.scale;
    dq.w = a.q; dq.w_stride = a.q_stride; dq.dot = dots ? p.qdq : nullptr;
    AttendArgs dk = t;
    dk.x = a.v; dk.y = a.d_o; dk.z = a.q;
    dk.x_stride = a.v_stride; dk.y_stride = so; dk.z_stride = a.q_stride;
    dk.states = p.grads; dk.out = a.dk_out; dk.c_state = 1.f;
    dk.w = a.k; dk.w_stride = a.k_stride; dk.dot = dots ? p.kdk : nullptr; dk.dot_state = dots ? p.kdk_state : nullptr;
    if (!dots) return run_attend_back<T, DK, DV, sizeof(T) == 4>(dk, dq, dv, l);
    KDA_TRY((run_attend_back<T, DK, DV, true>(dk, dq, dv, l)));
    KDA_TRY(l.next(lin_decay_grad_kernel, (unsigned)((int64_t)p.geo.nblocks * a.H), NT, 0, p.geo, a.log_decay, a.decay,
              p.states, p.grads, nullptr, p.total, DK * DV / 4, p.qdq, p.kdk, p.kdk_state, p.dot_stride,
              head ? nullptr : a.d_decay, head ? p.block_sum : nullptr));
    if (!head) return cudaSuccess;
    return l.next(lin_head_sum_kernel, a.H, NT, 0, p.geo, p.block_sum, a.d_decay);
}

}  // namespace

size_t linear_workspace_bytes(int N, int64_t T, int H, int dk, int dv, kda_dtype_t dt, bool packed) {
    return make_plan(N, T, H, dk, dv, dt, packed, false, use_tc(dt, dk, dv), nullptr).bytes;
}
size_t linear_backward_workspace_bytes(int N, int64_t T, int H, int dk, int dv, kda_dtype_t dt, bool packed) {
    size_t n = make_plan(N, T, H, dk, dv, dt, packed, true, false, nullptr).bytes;
    if (use_tc(dt, dk, dv)) n = std::max(n, make_plan(N, T, H, dk, dv, dt, packed, true, true, nullptr).bytes);
    return n;
}

#define KDA_LINEAR_DISPATCH(FN)                                                                                 \
    const bool bf = a.dt == KDA_BF16;                                                                           \
    if (a.dk == 128 && a.dv == 128) return FN<float, 128, 128>(a, s);                                           \
    if (a.dk == 64 && a.dv == 64) return bf ? FN<__nv_bfloat16, 64, 64>(a, s) : FN<float, 64, 64>(a, s);        \
    if (a.dk == 128) return bf ? FN<__nv_bfloat16, 128, 64>(a, s) : FN<float, 128, 64>(a, s);                   \
    return bf ? FN<__nv_bfloat16, 64, 128>(a, s) : FN<float, 64, 128>(a, s)

cudaError_t launch_linear(const LinArgs &a, cudaStream_t s) {
    if (use_tc(a.dt, a.dk, a.dv)) return forward_tc(a, s);
    KDA_LINEAR_DISPATCH(forward);
}
cudaError_t launch_linear_backward(const LinArgs &a, cudaStream_t s) {
    if (use_tc(a.dt, a.dk, a.dv)) return a.d_decay ? backward_tc(a, s) : backward_rolled_tc(a, s);
    KDA_LINEAR_DISPATCH(backward);
}

cudaError_t launch_linear_status(int32_t *status, int value, cudaStream_t s) {
    lin_status_kernel<<<1, 1, 0, s>>>(status, value);
    return cudaGetLastError();
}

}  // namespace kda
