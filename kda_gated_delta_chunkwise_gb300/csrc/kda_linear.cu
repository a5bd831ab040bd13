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
//   lin_attend_kernel  every 64-token tile of outputs, all tiles at once.
// Backward, with G the gradient of the state after a token
// (G_t = scale q_t do_t^T + e^{g_{t+1}} G_{t+1}): dq_t = scale S_t do_t,
// dk_t = G_t v_t, dv_t = G_t^T k_t. These are three more attentions of the
// same form: dq with (do, v, k) for (q, k, v) and S transposed, dk with
// (v, do, q) and dv with (k, q, do) in reverse time with G for S; so the same
// three kernels run them. The gradient of a log decay is everything that
// passes over the step into its token,
//   dg_t = sum_{i >= t > j} M_ij + sum_{i >= t} q_i.dq_i(S part)
//        + sum_{j < t} k_j.dk_j(G part) + e^{L_end} <S, G>    (inside a block)
//        = X + sum_{i >= t} (q_i.dq_i - k_i.dk_i),
//   X = e^{L_end} <S, G> + sum_j k_j.dk_j(G part),
// so it needs the row dots that the dq and dk passes have at hand.
//
// The products run on mma.sync tf32. bf16 values are exact in tf32; an fp32
// operand is split in two tf32 parts (22 bits) where its error would reach an
// fp32 output, and kept as one part (11 bits, against the 8 of the bf16 output)
// where it would not. Accumulators, states and sums are fp32.
#include <algorithm>

#include "kda_linear.cuh"
#include "kda_linear_tc.cuh"

namespace kda {
namespace {

constexpr int NT = 256;  // threads of the three main kernels
constexpr int CH = kLinChunk;

// The segment length where the state is carried along inside (lin_roll_tc): a
// function of the sequence's own length, so that a sequence gives the same bits
// alone and in any batch. A segment costs its 128-token chunks and about two
// more (its first state, its share of the scan), so short ones pay for being
// many and long ones leave a small batch on few of the 152 SMs.
constexpr int kLeastSegment = 512;
__host__ __device__ constexpr int segment_tokens(int64_t len) {
    return len <= 2048 ? kLeastSegment : len <= 16384 ? 1024 : len <= 65536 ? 2048 : 4096;
}

// ---------------------------------------------------------------- packed batches: the table of blocks
// sb = 0: segments of segment_tokens(length).
constexpr int kPrepThreads = 1024;
__global__ void __launch_bounds__(kPrepThreads)
lin_blocks_kernel(const int32_t *__restrict__ cu, int N, int T_total, int sb, int nblocks, int4 *blocks,
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
            const int len = cu[i + 1] - cu[i], per = sb ? sb : segment_tokens(len);
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
        const int per = sb ? sb : segment_tokens(cu[lo + 1] - cu[lo]);
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
template <int K, int MT, int NT8, bool SA, bool SB, typename FA, typename FB>
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
                ah[m][u] = tf32(x[u]);
                if (SA) al[m][u] = tf32(x[u] - __uint_as_float(ah[m][u]));
            }
        }
#pragma unroll
        for (int n = 0; n < NT8; ++n) {
            const float x0 = b(k + t, c0 + 8 * n + g), x1 = b(k + t + 4, c0 + 8 * n + g);
            const uint32_t h0 = tf32(x0), h1 = tf32(x1);
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

// Rows of a [64][D] tile into shared memory; rows past `rows` are zero.
template <typename T, int D>
__device__ __forceinline__ void load_tile(T *dst, int ld, const T *src, int64_t stride, int rows) {
    constexpr int V = 16 / sizeof(T), PER = D / V;
    for (int i = threadIdx.x; i < CH * PER; i += NT) {
        const int r = i / PER, c = (i % PER) * V;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) x = __ldg(reinterpret_cast<const uint4 *>(src + r * stride + c));
        *reinterpret_cast<uint4 *>(dst + r * ld + c) = x;
    }
}
// Leading dimensions that keep the fragment reads free of bank conflicts:
// rows across lanes (A, or B stored [n][k]) and rows along k (B stored [k][n]).
template <typename T> __host__ __device__ constexpr int ld_rows(int d) { return sizeof(T) == 2 ? d + 8 : d + 4; }
template <typename T> __host__ __device__ constexpr int ld_cols(int d) { return d + 8; }

// ---------------------------------------------------------------- a block's own state
// out[block][head] = sum_s w_s x_s y_s^T over the block's tokens: forward
// w_s = e^{L_end - L_s} with (x, y) = (k, v); reverse w_s = e^{L_s} with
// (q, do). Also e^{L_end} of the block (forward).
template <typename T, int DK, int DV, bool REV>
__global__ void __launch_bounds__(NT)
lin_state_kernel(LinGeom geo, const T *__restrict__ x, int64_t x_stride, const T *__restrict__ y, int64_t y_stride,
                 const float *__restrict__ log_decay, int decay, float *__restrict__ out, float *__restrict__ total) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int WM = DK / 32, WN = NT / 32 / WM, COLS = DV / WN, N8 = COLS / 8;
    constexpr int LDX = ld_cols<T>(DK), LDY = ld_cols<T>(DV);
    extern __shared__ __align__(16) unsigned char smem[];
    T *xs = reinterpret_cast<T *>(smem);
    T *ys = xs + CH * LDX;
    float2 *a = reinterpret_cast<float2 *>(ys + CH * LDY);
    __shared__ long long scan[NT / 32];
    __shared__ float w[CH];
    const int b = blockIdx.x / geo.H, h = blockIdx.x % geo.H;
    const LinBlock blk = lin_block(geo, b);
    if (blk.len <= 0) return;
    decay_prefix<NT>(log_decay, decay, blk.start, geo.H, h, blk.len, blk.len, a, scan);
    const float2 end = a[blk.len];
    if (total && threadIdx.x == 0) total[(int64_t)b * geo.H + h] = decay_ratio(end, make_float2(0.f, 0.f));
    const int warp = threadIdx.x >> 5, r0 = (warp % WM) * 32, c0 = (warp / WM) * COLS;
    float acc[2][N8][4] = {};
    for (int j0 = 0; j0 < blk.len; j0 += CH) {
        const int rows = min(CH, blk.len - j0);
        const int64_t tok = blk.start + j0;
        __syncthreads();
        load_tile<T, DK>(xs, LDX, x + tok * x_stride + h * DK, x_stride, rows);
        load_tile<T, DV>(ys, LDY, y + tok * y_stride + h * DV, y_stride, rows);
        if (threadIdx.x < CH) {
            const int s = min(j0 + (int)threadIdx.x, blk.len - 1);
            w[threadIdx.x] = REV ? decay_ratio(a[s + 1], make_float2(0.f, 0.f)) : decay_ratio(end, a[s + 1]);
        }
        __syncthreads();
        product<CH, 2, N8, true, F32>(
            acc, [&](int r, int k) { return to_f32(xs[k * LDX + r]) * w[k]; },
            [&](int k, int c) { return to_f32(ys[k * LDY + c]); }, r0, c0);
    }
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float *dst = out + ((int64_t)b * geo.H + h) * DK * DV;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < N8; ++n) {
            const int r = r0 + 16 * m + g, c = c0 + 8 * n + 2 * t;
            *reinterpret_cast<float2 *>(dst + r * DV + c) = make_float2(acc[m][n][0], acc[m][n][1]);
            *reinterpret_cast<float2 *>(dst + (r + 8) * DV + c) = make_float2(acc[m][n][2], acc[m][n][3]);
        }
}

// ---------------------------------------------------------------- joining the blocks
// In place, along each (sequence, head): forward, every block's own sum gives
// way to the state before the block, S <- e^{L_end} S + c own, and the last S
// is the final state; reverse, to the gradient of the state after the block.
// Elementwise over the state: one float4 per thread, the blocks in turn, four
// loads ahead.
template <bool REV>
__global__ void __launch_bounds__(NT)
lin_scan_kernel(LinGeom geo, float *__restrict__ states, const float *__restrict__ total, const float *__restrict__ s0,
                float *__restrict__ sT, float c, int size4) {
    if (geo.status && *geo.status != KDA_DEV_OK) return;
    const int per = size4 / NT;
    const int64_t nh = blockIdx.x / per;
    const int n = (int)(nh / geo.H), h = (int)(nh % geo.H);
    const int64_t e = (int64_t)(blockIdx.x % per) * NT + threadIdx.x;
    int first, last;
    lin_seq_blocks(geo, n, first, last);
    float4 S = s0 ? reinterpret_cast<const float4 *>(s0)[nh * size4 + e] : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 *p = reinterpret_cast<float4 *>(states);
    const int count = last - first;
    constexpr int AHEAD = 4;
    float4 own[AHEAD];
    float f[AHEAD];
    auto at = [&](int i) {
        const int b = REV ? last - 1 - i : first + i;
        return (int64_t)(geo.place ? __ldg(geo.place + b) : b) * geo.H + h;
    };
    for (int i0 = 0; i0 < count; i0 += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i0 + u < count) {
                own[u] = p[at(i0 + u) * size4 + e];
                f[u] = total[at(i0 + u)];
            }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i0 + u < count) {
                p[at(i0 + u) * size4 + e] = S;
                if (f[u] == 0.f) S = make_float4(0.f, 0.f, 0.f, 0.f);  // a reset, whatever the state held
                S.x = f[u] * S.x + c * own[u].x;
                S.y = f[u] * S.y + c * own[u].y;
                S.z = f[u] * S.z + c * own[u].z;
                S.w = f[u] * S.w + c * own[u].w;
            }
    }
    if (sT) reinterpret_cast<float4 *>(sT)[nh * size4 + e] = S;
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
template <typename T, int DC, int DO, bool REV, bool ST, bool EXACT>
__global__ void __launch_bounds__(NT) lin_attend_kernel(AttendArgs p) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int LDX = ld_rows<T>(DC), LDZ = ld_cols<T>(DO), LDS = DO + 8, LDP = CH + 4, N8 = DO / 16;
    extern __shared__ __align__(16) unsigned char smem[];
    T *xs = reinterpret_cast<T *>(smem);
    T *ys = xs + CH * LDX;
    float *ps = reinterpret_cast<float *>(ys + CH * LDX);
    float *ss = ps + CH * LDP;               // a 64-row piece of the state, then the z tile
    T *zs = reinterpret_cast<T *>(ss);
    float2 *a = reinterpret_cast<float2 *>(ss + CH * LDS);
    __shared__ long long scan[NT / 32];
    __shared__ float dots[2][2][CH];
    const LinGeom &geo = p.geo;
    const int tiles = geo.sb / CH;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % geo.H, b = blockIdx.x / tiles / geo.H;
    const LinBlock blk = lin_block(geo, b);
    const int i0 = tile * CH;
    if (i0 >= blk.len) return;
    decay_prefix<NT>(p.log_decay, p.decay, blk.start, geo.H, h, blk.len, blk.len, a, scan);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int r0 = (warp & 3) * 16, half = warp >> 2, c0 = half * (DO / 2);
    const int irows = min(CH, blk.len - i0);
    load_tile<T, DC>(xs, LDX, (const T *)p.x + (int64_t)(blk.start + i0) * p.x_stride + h * DC, p.x_stride, irows);

    // the state part, 64 rows of the contraction at a time
    float acc[1][N8][4] = {};
    const float *S = p.states + ((int64_t)b * geo.H + h) * DC * DO;
    for (int k0 = 0; k0 < DC; k0 += CH) {
        __syncthreads();
        if (!ST) {
            for (int i = threadIdx.x; i < CH * DO / 4; i += NT) {
                const int r = i / (DO / 4), c = (i % (DO / 4)) * 4;
                *reinterpret_cast<float4 *>(ss + r * LDS + c) =
                    __ldg(reinterpret_cast<const float4 *>(S + (int64_t)(k0 + r) * DO + c));
            }
        } else {
            for (int i = threadIdx.x; i < CH * DO; i += NT) {
                const int r = i % CH, c = i / CH;
                ss[r * LDS + c] = __ldg(S + (int64_t)c * DC + k0 + r);
            }
        }
        __syncthreads();
        product<CH, 1, N8, F32, EXACT>(
            acc, [&](int r, int k) { return to_f32(xs[r * LDX + k0 + k]); },
            [&](int k, int c) { return ss[k * LDS + c]; }, r0, c0);
    }
    auto row_dots = [&](float *dst) {  // w_i . acc_i over this warp's columns
        float d[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = r0 + g + 8 * e;
            if (r < irows) {
                const T *w = (const T *)p.w + (int64_t)(blk.start + i0 + r) * p.w_stride + h * DO;
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
        const int i = min(i0 + r0 + g + 8 * e, blk.len - 1);
        const float f = p.c_state * (REV ? decay_ratio(a[blk.len], a[i + 1])
                                         : decay_ratio(a[i + 1], make_float2(0.f, 0.f)));
#pragma unroll
        for (int n = 0; n < N8; ++n) {
            acc[0][n][2 * e] = f == 0.f ? 0.f : acc[0][n][2 * e] * f;  // a reset, whatever the state held
            acc[0][n][2 * e + 1] = f == 0.f ? 0.f : acc[0][n][2 * e + 1] * f;
        }
    }
    if (p.dot_state) row_dots(dots[0][half]);

    // the block's own tokens
    const int jfirst = REV ? i0 : 0, jlast = REV ? blk.len : i0 + CH;
    for (int j0 = jfirst; j0 < jlast; j0 += CH) {
        const int jrows = min(CH, blk.len - j0);
        const int64_t tok = blk.start + j0;
        __syncthreads();
        load_tile<T, DC>(ys, LDX, (const T *)p.y + tok * p.y_stride + h * DC, p.y_stride, jrows);
        load_tile<T, DO>(zs, LDZ, (const T *)p.z + tok * p.z_stride + h * DO, p.z_stride, jrows);
        __syncthreads();
        float sc[1][4][4] = {};
        const int s0 = half * 32;
        product<DC, 1, 4, F32, F32>(
            sc, [&](int r, int k) { return to_f32(xs[r * LDX + k]); },
            [&](int k, int c) { return to_f32(ys[c * LDX + k]); }, r0, s0);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = r0 + g + 8 * (e >> 1), c = s0 + 8 * n + 2 * t + (e & 1);
                const int i = i0 + r, j = j0 + c;
                float v = 0.f;  // chosen, not multiplied: what lies past the end may be anything
                if (i < blk.len && j < blk.len && (REV ? j >= i : j <= i))
                    v = p.c_intra * sc[0][n][e] * (REV ? decay_ratio(a[j + 1], a[i + 1]) : decay_ratio(a[i + 1], a[j + 1]));
                ps[r * LDP + c] = v;
            }
        __syncthreads();
        product<CH, 1, N8, EXACT, F32>(
            acc, [&](int r, int k) { return ps[r * LDP + k]; },
            [&](int k, int c) { return to_f32(zs[k * LDZ + c]); }, r0, c0);
    }
    if (p.dot) row_dots(dots[1][half]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = r0 + g + 8 * e;
        if (r >= irows) continue;
        T *o = (T *)p.out + ((int64_t)(blk.start + i0 + r) * geo.H + h) * DO;
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
        if ((int)threadIdx.x < irows) {
            const int64_t i = (int64_t)(blk.start + i0 + threadIdx.x) * geo.H + h;
            p.dot[i] = dots[1][0][threadIdx.x] + dots[1][1][threadIdx.x];
            if (p.dot_state) p.dot_state[i] = dots[0][0][threadIdx.x] + dots[0][1][threadIdx.x];
        }
    }
}

// ---------------------------------------------------------------- gradient of the log decay
// Per block and head: dg_t = X + sum_{i >= t} (qdq_i - kdk_i), with
// X = e^{L_end} <S, G> + sum_j kdk_state_j. A reset (log decay at or below the
// clamp) passes nothing on: its gradient is zero, not the sum's rounding.
__global__ void __launch_bounds__(NT)
lin_decay_grad_kernel(LinGeom geo, const float *__restrict__ log_decay, int decay, const float *__restrict__ states,
                      const float *__restrict__ grads, const float *__restrict__ inner,
                      const float *__restrict__ total, int size4,
                      const float *__restrict__ qdq, const float *__restrict__ kdk,
                      const float *__restrict__ kdk_state, int64_t dot_stride, float *__restrict__ dg,
                      float *__restrict__ block_sum) {
    __shared__ float red[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / geo.H, h = blockIdx.x % geo.H;
    const LinBlock blk = lin_block(geo, b);
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
        if (tid < kScanPartials) x = __ldg(inner + bh * kScanPartials + tid);
    } else {
        const float4 *S = reinterpret_cast<const float4 *>(states) + bh * size4;
        const float4 *G = reinterpret_cast<const float4 *>(grads) + bh * size4;
        for (int i = tid; i < size4; i += NT) {
            const float4 s = __ldg(S + i), g = __ldg(G + i);
            x += s.x * g.x + s.y * g.y + s.z * g.z + s.w * g.w;
        }
    }
    x *= total[bh];
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
lin_head_sum_kernel(LinGeom geo, const float *__restrict__ block_sum, float *__restrict__ dg) {
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

// ---------------------------------------------------------------- host side
size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The block length of the general kernels, which work on 64-token chunks one
// after the other: one chunk a block gives the most blocks at once (257 tokens
// x 2 heads, fp32, d = 64: 21 us of GPU time in blocks of 64, 40 in blocks of
// 256). One length for all, so that a sequence gives the same bits in any batch.
constexpr int kGeneralBlock = 64;

int64_t max_blocks(int N, int64_t T, bool packed, int sb) {
    return packed ? T / sb + N : (int64_t)N * ((T + sb - 1) / sb);
}

struct Plan {
    LinGeom geo;
    int4 *blocks;
    int32_t *seq_block, *status, *place;
    float *total, *states, *grads, *qdq, *kdk, *kdk_state, *block_sum;
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
    const int sb = !tc ? kGeneralBlock : !rolled ? kLinMaxBlock : packed ? kLeastSegment : segment_tokens(T);
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

template <typename T, int DK, int DV, bool REV>
cudaError_t run_states(const Plan &p, const void *x, int64_t xs, const void *y, int64_t ys, const LinArgs &a,
                       float *out, cudaStream_t s) {
    const size_t fixed = CH * (ld_cols<T>(DK) + ld_cols<T>(DV)) * sizeof(T);
    const size_t smem = fixed + (p.geo.sb + 1) * sizeof(float2);
    auto k = lin_state_kernel<T, DK, DV, REV>;
    static std::atomic<uint64_t> allowed{0};
    KDA_TRY(allow_smem(k, fixed + (kLinMaxBlock + 1) * sizeof(float2), allowed));
    k<<<(unsigned)((int64_t)p.geo.nblocks * p.geo.H), NT, smem, s>>>(p.geo, (const T *)x, xs, (const T *)y, ys,
                                                                     a.log_decay, a.decay, out, REV ? nullptr : p.total);
    return cudaGetLastError();
}
template <bool REV>
cudaError_t run_scan(const Plan &p, float *states, const float *s0, float *sT, float c, int dk, int dv,
                     cudaStream_t s) {
    const int size4 = dk * dv / 4;
    lin_scan_kernel<REV><<<(unsigned)((int64_t)p.geo.N * p.geo.H * (size4 / NT)), NT, 0, s>>>(p.geo, states, p.total,
                                                                                            s0, sT, c, size4);
    return cudaGetLastError();
}
template <typename T, int DC, int DO, bool REV, bool ST, bool EXACT>
cudaError_t run_attend(const AttendArgs &p, cudaStream_t s) {
    const size_t fixed = 2 * CH * ld_rows<T>(DC) * sizeof(T) + CH * (CH + 4) * 4 + CH * (DO + 8) * 4;
    const size_t smem = fixed + (p.geo.sb + 1) * sizeof(float2);
    auto k = lin_attend_kernel<T, DC, DO, REV, ST, EXACT>;
    static std::atomic<uint64_t> allowed{0};
    KDA_TRY(allow_smem(k, fixed + (kLinMaxBlock + 1) * sizeof(float2), allowed));
    k<<<(unsigned)((int64_t)p.geo.nblocks * p.geo.H * (p.geo.sb / CH)), NT, smem, s>>>(p);
    return cudaGetLastError();
}

cudaError_t prepare_blocks(const Plan &p, const LinArgs &a, bool rolled, cudaStream_t s) {
    if (!a.cu_seqlens) return cudaSuccess;
    lin_blocks_kernel<<<1, kPrepThreads, 0, s>>>(a.cu_seqlens, a.N, a.T, rolled ? 0 : p.geo.sb, p.geo.nblocks, p.blocks,
                                                 p.seq_block, p.place, p.status, a.status);
    return cudaGetLastError();
}

// bf16, d_k = d_v = 128: the same steps on the tensor cores.
cudaError_t forward_tc(const LinArgs &a, cudaStream_t s) {
    const Plan p = make_plan(a.N, a.T, a.H, 128, 128, a.dt, a.cu_seqlens != nullptr, false, use_tc(a.dt, a.dk, a.dv), a.workspace);
    const int64_t tokens = a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    KDA_TRY(prepare_blocks(p, a, true, s));
    // one segment a sequence and no final state asked for: the first states are all there is
    const bool need_states = a.sT || a.cu_seqlens || p.geo.per_seq > 1;
    if (tokens > 0 && need_states)
        KDA_TRY(launch_state_tc(p.geo, false, a.k, a.k_stride, a.v, a.v_stride, tokens, a.log_decay, a.decay, p.states,
                                p.total, s));
    KDA_TRY(run_scan<false>(p, p.states, a.s0, a.sT, 1.f, 128, 128, s));
    if (tokens == 0) return cudaSuccess;
    RollTc t{};
    t.geo = p.geo;
    t.x = a.q; t.y = a.k; t.z = a.v;
    t.x_stride = a.q_stride; t.y_stride = a.k_stride; t.z_stride = a.v_stride;
    t.states = p.states; t.tokens = tokens;
    t.log_decay = a.log_decay; t.decay = a.decay;
    t.out = a.o; t.c_state = a.scale; t.c_intra = a.scale; t.c_roll = 1.f;
    return launch_roll_tc(t, s);
}

// Backward without the decay's gradient: three passes with the state carried along.
cudaError_t backward_rolled_tc(const LinArgs &a, cudaStream_t s) {
    constexpr bool rolled = true;
    const Plan p = make_plan(a.N, a.T, a.H, 128, 128, a.dt, a.cu_seqlens != nullptr, true, rolled, a.workspace);
    const int64_t tokens = a.cu_seqlens ? a.T : (int64_t)a.N * a.T, so = (int64_t)a.H * 128;
    KDA_TRY(prepare_blocks(p, a, true, s));
    if (tokens > 0) {
        KDA_TRY(launch_state_tc(p.geo, false, a.k, a.k_stride, a.v, a.v_stride, tokens, a.log_decay, a.decay, p.states,
                                p.total, s));
        KDA_TRY(launch_state_tc(p.geo, true, a.q, a.q_stride, a.d_o, so, tokens, a.log_decay, a.decay, p.grads,
                                nullptr, s));
        KDA_TRY(run_scan<false>(p, p.states, a.s0, nullptr, 1.f, 128, 128, s));
    }
    KDA_TRY(run_scan<true>(p, p.grads, a.dsT, a.ds0, a.scale, 128, 128, s));
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
    KDA_TRY(launch_roll_tc(u, s));
    u = t;  // dk
    u.rev = u.state_t = true;
    u.x = a.v; u.y = a.d_o; u.z = a.q;
    u.x_stride = a.v_stride; u.y_stride = so; u.z_stride = a.q_stride;
    u.states = p.grads; u.out = a.dk_out; u.c_state = 1.f; u.c_roll = a.scale;
    KDA_TRY(launch_roll_tc(u, s));
    u = t;  // dv
    u.rev = true;
    u.x = a.k; u.y = a.q; u.z = a.d_o;
    u.x_stride = a.k_stride; u.y_stride = a.q_stride; u.z_stride = so;
    u.states = p.grads; u.out = a.dv_out; u.c_state = 1.f; u.c_roll = a.scale;
    return launch_roll_tc(u, s);
}

// Backward with the decay's gradient: blocks of kLinMaxBlock, every block's
// states in three bf16 parts, and the row dots.
cudaError_t backward_tc(const LinArgs &a, cudaStream_t s) {
    constexpr bool rolled = false;
    const Plan p = make_plan(a.N, a.T, a.H, 128, 128, a.dt, a.cu_seqlens != nullptr, true, rolled, a.workspace);
    const int64_t tokens = a.cu_seqlens ? a.T : (int64_t)a.N * a.T, so = (int64_t)a.H * 128;
    const bool head = a.decay == KDA_DECAY_HEAD;
    KDA_TRY(prepare_blocks(p, a, false, s));
    if (tokens > 0) {
        KDA_TRY(launch_state_tc(p.geo, false, a.k, a.k_stride, a.v, a.v_stride, tokens, a.log_decay, a.decay, p.states,
                                p.total, s));
        KDA_TRY(launch_scan_tc(p.geo, false, p.states, p.total, a.s0, nullptr, 1.f, p.s_parts, p.part_stride,
                               nullptr, nullptr, s));
        // the blocks' own sums of the states are done with: those of the gradients take their place
        KDA_TRY(launch_state_tc(p.geo, true, a.q, a.q_stride, a.d_o, so, tokens, a.log_decay, a.decay, p.states,
                                nullptr, s));
    }
    KDA_TRY(launch_scan_tc(p.geo, true, p.states, p.total, a.dsT, a.ds0, a.scale, p.g_parts, p.part_stride,
                           p.s_parts, p.inner, s));
    if (tokens == 0)
        return head ? cudaMemsetAsync(a.d_decay, 0, sizeof(float) * a.H, s) : cudaSuccess;
    AttendTc t{};
    t.geo = p.geo;
    t.part_stride = p.part_stride; t.tokens = tokens;
    t.log_decay = a.log_decay; t.decay = a.decay;
    t.c_intra = a.scale;
    AttendTc u = t;  // dv
    u.rev = true;
    u.x = a.k; u.y = a.q; u.z = a.d_o;
    u.x_stride = a.k_stride; u.y_stride = a.q_stride; u.z_stride = so;
    u.states = p.g_parts; u.out = a.dv_out; u.c_state = 1.f;
    KDA_TRY(launch_attend_tc(u, s));
    u = t;  // dq
    u.state_t = true;
    u.x = a.d_o; u.y = a.v; u.z = a.k; u.w = a.q;
    u.x_stride = so; u.y_stride = a.v_stride; u.z_stride = a.k_stride; u.w_stride = a.q_stride;
    u.states = p.s_parts; u.out = a.dq; u.c_state = a.scale;
    u.dot = p.qdq;
    KDA_TRY(launch_attend_tc(u, s));
    u = t;  // dk
    u.rev = u.state_t = true;
    u.x = a.v; u.y = a.d_o; u.z = a.q; u.w = a.k;
    u.x_stride = a.v_stride; u.y_stride = so; u.z_stride = a.q_stride; u.w_stride = a.k_stride;
    u.states = p.g_parts; u.out = a.dk_out; u.c_state = 1.f;
    u.dot = p.kdk;
    u.dot_state = p.kdk_state;
    KDA_TRY(launch_attend_tc(u, s));
    lin_decay_grad_kernel<<<(unsigned)((int64_t)p.geo.nblocks * a.H), NT, 0, s>>>(
        p.geo, a.log_decay, a.decay, nullptr, nullptr, p.inner, p.total, 0, p.qdq, p.kdk, p.kdk_state, p.dot_stride,
        head ? nullptr : a.d_decay, head ? p.block_sum : nullptr);
    KDA_TRY(cudaGetLastError());
    if (!head) return cudaSuccess;
    lin_head_sum_kernel<<<a.H, NT, 0, s>>>(p.geo, p.block_sum, a.d_decay);
    return cudaGetLastError();
}

template <typename T, int DK, int DV> cudaError_t forward(const LinArgs &a, cudaStream_t s) {
    constexpr bool F32 = sizeof(T) == 4;
    const Plan p = make_plan(a.N, a.T, a.H, DK, DV, a.dt, a.cu_seqlens != nullptr, false, use_tc(a.dt, a.dk, a.dv), a.workspace);
    KDA_TRY(prepare_blocks(p, a, false, s));
    if (p.geo.nblocks > 0)
        KDA_TRY((run_states<T, DK, DV, false>(p, a.k, a.k_stride, a.v, a.v_stride, a, p.states, s)));
    KDA_TRY((run_scan<false>(p, p.states, a.s0, a.sT, 1.f, DK, DV, s)));
    if (p.geo.nblocks == 0) return cudaSuccess;
    AttendArgs t{};
    t.geo = p.geo;
    t.x = a.q; t.y = a.k; t.z = a.v;
    t.x_stride = a.q_stride; t.y_stride = a.k_stride; t.z_stride = a.v_stride;
    t.log_decay = a.log_decay; t.decay = a.decay; t.states = p.states;
    t.out = a.o; t.c_state = a.scale; t.c_intra = a.scale;
    return run_attend<T, DK, DV, false, false, F32>(t, s);
}

template <typename T, int DK, int DV> cudaError_t backward(const LinArgs &a, cudaStream_t s) {
    constexpr bool F32 = sizeof(T) == 4, rolled = false;
    const Plan p = make_plan(a.N, a.T, a.H, DK, DV, a.dt, a.cu_seqlens != nullptr, true, rolled, a.workspace);
    KDA_TRY(prepare_blocks(p, a, false, s));
    const int64_t so = (int64_t)a.H * DV;
    if (p.geo.nblocks > 0) {
        KDA_TRY((run_states<T, DK, DV, false>(p, a.k, a.k_stride, a.v, a.v_stride, a, p.states, s)));
        KDA_TRY((run_states<T, DK, DV, true>(p, a.q, a.q_stride, a.d_o, so, a, p.grads, s)));
        KDA_TRY((run_scan<false>(p, p.states, a.s0, nullptr, 1.f, DK, DV, s)));
    }
    KDA_TRY((run_scan<true>(p, p.grads, a.dsT, a.ds0, a.scale, DK, DV, s)));
    if (p.geo.nblocks == 0) return a.d_decay && a.decay == KDA_DECAY_HEAD
                                       ? cudaMemsetAsync(a.d_decay, 0, sizeof(float) * a.H, s) : cudaSuccess;
    const bool dots = a.d_decay != nullptr;
    AttendArgs t{};
    t.geo = p.geo;
    t.log_decay = a.log_decay; t.decay = a.decay;
    t.c_intra = a.scale;
    AttendArgs u = t;  // dv: keys attend, in reverse time, to the queries of later tokens
    u.x = a.k; u.y = a.q; u.z = a.d_o;
    u.x_stride = a.k_stride; u.y_stride = a.q_stride; u.z_stride = so;
    u.states = p.grads; u.out = a.dv_out; u.c_state = 1.f;
    KDA_TRY((run_attend<T, DK, DV, true, false, F32>(u, s)));
    u = t;  // dq
    u.x = a.d_o; u.y = a.v; u.z = a.k;
    u.x_stride = so; u.y_stride = a.v_stride; u.z_stride = a.k_stride;
    u.states = p.states; u.out = a.dq; u.c_state = a.scale;
    u.w = a.q; u.w_stride = a.q_stride; u.dot = dots ? p.qdq : nullptr;
    KDA_TRY((F32 || dots ? run_attend<T, DV, DK, false, true, true>(u, s)
                         : run_attend<T, DV, DK, false, true, F32>(u, s)));
    u = t;  // dk
    u.x = a.v; u.y = a.d_o; u.z = a.q;
    u.x_stride = a.v_stride; u.y_stride = so; u.z_stride = a.q_stride;
    u.states = p.grads; u.out = a.dk_out; u.c_state = 1.f;
    u.w = a.k; u.w_stride = a.k_stride; u.dot = dots ? p.kdk : nullptr; u.dot_state = dots ? p.kdk_state : nullptr;
    KDA_TRY((F32 || dots ? run_attend<T, DV, DK, true, true, true>(u, s)
                         : run_attend<T, DV, DK, true, true, F32>(u, s)));
    if (!dots) return cudaSuccess;
    const bool head = a.decay == KDA_DECAY_HEAD;
    lin_decay_grad_kernel<<<(unsigned)((int64_t)p.geo.nblocks * a.H), NT, 0, s>>>(
        p.geo, a.log_decay, a.decay, p.states, p.grads, nullptr, p.total, DK * DV / 4, p.qdq, p.kdk, p.kdk_state, p.dot_stride,
        head ? nullptr : a.d_decay, head ? p.block_sum : nullptr);
    KDA_TRY(cudaGetLastError());
    if (!head) return cudaSuccess;
    lin_head_sum_kernel<<<a.H, NT, 0, s>>>(p.geo, p.block_sum, a.d_decay);
    return cudaGetLastError();
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

}  // namespace kda
