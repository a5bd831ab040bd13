// One token of linear attention with a decay, the state updated in place:
//   S <- e^g S + k v^T,   o = scale S^T q.
//
// Bound by memory: the state (dk x dv fp32 per head) is read once and written
// once. The columns of a state do not interact, so a head is cut into slices
// of 32 value columns (128-byte row pieces), one CTA each: a single sequence of
// 32 heads runs on 128 CTAs, and a large batch has more, smaller CTAs to keep
// the memory busy with. A thread owns four columns of DK / ROWS rows and issues
// all its 16-byte loads first; the sums over the rows for o go through shared
// memory, in a fixed order. bf16, d = 128, a CTA for 32 columns against one for
// the whole head: 32 heads 2.8 us and 3.4, 512 12.1 and 13.4, 2048 42.1 and 43.9,
// 8192 155.7 and 157.4 (1.08 GB, 6.95 TB/s, 103 % of a copy).
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int NT = 256;
constexpr int COLS = 32;

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(NT)
lin_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, int64_t q_stride,
                  int64_t k_stride, int64_t v_stride, const float *__restrict__ log_decay, int decay, float scale,
                  float *__restrict__ state, const int32_t *__restrict__ slots, int pool_size,
                  int32_t *__restrict__ status, int H, T *__restrict__ o) {
    constexpr int SLICES = DV / COLS, TPR = COLS / 4, ROWS = NT / TPR, PASSES = DK / ROWS;
    static_assert(DK % ROWS == 0, "rows per thread");
    __shared__ float sk[DK], sq[DK];
    __shared__ __align__(16) float red[ROWS][COLS];
    const int64_t nh = blockIdx.x / SLICES;
    const int c0 = (int)(blockIdx.x % SLICES) * COLS, n = (int)(nh / H), h = (int)(nh % H);
    const int tid = threadIdx.x, col = (tid % TPR) * 4, row0 = tid / TPR;
    bool fresh;
    const int64_t slot = slot_of(slots, n, fresh);
    if (slots && slot >= pool_size) {  // uniform over the CTA
        if (tid == 0 && status) atomicOr(status, KDA_DEV_BAD_SLOT);
        return;
    }
    float *S = state + (slot * H + h) * (int64_t)DK * DV + c0 + col;
    float4 s[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
        s[p] = fresh ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : __ldcs(reinterpret_cast<const float4 *>(S + (int64_t)(row0 + p * ROWS) * DV));
    if (tid < DK) {
        sk[tid] = to_f32(k[n * k_stride + h * DK + tid]);
        sq[tid] = to_f32(q[n * q_stride + h * DK + tid]);
    }
    const T *vp = v + n * v_stride + h * DV + c0 + col;
    const float4 vv = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    const float g = decay == KDA_DECAY_NONE ? 0.f : decay == KDA_DECAY_HEAD ? log_decay[h] : log_decay[nh];
    const float a = g <= kMinLogDecay ? 0.f : expf(g);
    if (a == 0.f) {  // a reset leaves nothing, whatever the state held
#pragma unroll
        for (int p = 0; p < PASSES; ++p) s[p] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    float4 po = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int i = row0 + p * ROWS;
        const float kk = sk[i], qq = sq[i];
        s[p].x = a * s[p].x + kk * vv.x;
        s[p].y = a * s[p].y + kk * vv.y;
        s[p].z = a * s[p].z + kk * vv.z;
        s[p].w = a * s[p].w + kk * vv.w;
        __stcs(reinterpret_cast<float4 *>(S + (int64_t)i * DV), s[p]);
        po.x += qq * s[p].x;
        po.y += qq * s[p].y;
        po.z += qq * s[p].z;
        po.w += qq * s[p].w;
    }
    *reinterpret_cast<float4 *>(&red[row0][col]) = po;
    __syncthreads();
    if (tid < COLS) {
        float x = 0.f;
#pragma unroll 8
        for (int r = 0; r < ROWS; ++r) x += red[r][tid];
        o[nh * DV + c0 + tid] = from_f32<T>(scale * x);
    }
}

template <typename T, int DK, int DV>
cudaError_t run(const void *q, const void *k, const void *v, int64_t qs, int64_t ks, int64_t vs, const float *g,
                int decay, float scale, float *state, const int32_t *slots, int pool, int32_t *status, void *o, int N,
                int H, cudaStream_t s) {
    lin_decode_kernel<T, DK, DV><<<(unsigned)((int64_t)N * H * (DV / COLS)), NT, 0, s>>>(
        (const T *)q, (const T *)k, (const T *)v, qs, ks, vs, g, decay, scale, state, slots, pool, status, H, (T *)o);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, kda_dtype_t dt, int64_t qs, int64_t ks,
                                 int64_t vs, const float *g, int decay, float scale, float *state,
                                 const int32_t *slots, int pool, int32_t *status, void *o, int N, int H, int dk, int dv,
                                 cudaStream_t s) {
#define KDA_CASE(K_, V_)                                                                                              \
    if (dk == K_ && dv == V_)                                                                                         \
        return dt == KDA_BF16                                                                                         \
                   ? run<__nv_bfloat16, K_, V_>(q, k, v, qs, ks, vs, g, decay, scale, state, slots, pool, status, o, \
                                                N, H, s)                                                              \
                   : run<float, K_, V_>(q, k, v, qs, ks, vs, g, decay, scale, state, slots, pool, status, o, N, H, s);
    KDA_CASE(128, 128)
    KDA_CASE(64, 64)
    KDA_CASE(128, 64)
    KDA_CASE(64, 128)
#undef KDA_CASE
    return cudaErrorInvalidValue;
}

}  // namespace kda
