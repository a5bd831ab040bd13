// Pieces shared by the kernels that hold a row of channels in a few lanes: the
// norms with rotary positions, with a gate, and of the residual stream.
#pragma once

#include "kda_internal.cuh"
#include "kda_linear.cuh"

namespace kda {

template <typename T> struct Vec {  // 16 bytes of a row: N channels, as loaded and as pairs
    static constexpr int N = 16 / sizeof(T);
    uint32_t raw[4];
    __device__ __forceinline__ void zero() { raw[0] = raw[1] = raw[2] = raw[3] = 0u; }
    // a plain load: the same kernel may write there
    __device__ __forceinline__ void load(const T *p) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        raw[0] = x.x, raw[1] = x.y, raw[2] = x.z, raw[3] = x.w;
    }
    __device__ __forceinline__ void store(T *p) const {
        *reinterpret_cast<uint4 *>(p) = make_uint4(raw[0], raw[1], raw[2], raw[3]);
    }
    __device__ __forceinline__ F2 get(int i) const {  // channels 2 i, 2 i + 1
        if constexpr (sizeof(T) == 2) return f2(__uint_as_float(raw[i] << 16), __uint_as_float(raw[i] & 0xffff0000u));
        else return f2(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1]));
    }
    __device__ __forceinline__ void put(int i, F2 x) {
        float lo, hi;
        f2_get(x, lo, hi);
        if constexpr (sizeof(T) == 2) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(raw[i]) : "f"(hi), "f"(lo));
        } else {
            raw[2 * i] = __float_as_uint(lo);
            raw[2 * i + 1] = __float_as_uint(hi);
        }
    }
};

template <int LANES> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Two at once: the halves of the lanes carry one each, five shuffles of 16 lanes
// instead of eight. The same bits.
template <int LANES> __device__ __forceinline__ void row_sums(float &a, float &b) {
    const bool up = threadIdx.x & (LANES / 2);
    const float give = up ? a : b, keep = up ? b : a;
    const float v = row_sum<LANES / 2>(keep + __shfl_xor_sync(0xffffffffu, give, LANES / 2));
    const float other = __shfl_xor_sync(0xffffffffu, v, LANES / 2);
    a = up ? other : v;
    b = up ? v : other;
}

// From global or shared memory, 4 N-byte aligned.
template <int N> __device__ __forceinline__ void load_floats(const float *p, float *x) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + e);
            x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
        }
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x, x[1] = v.y;
    }
}
// rsqrtf is within 2 ulp
__device__ __forceinline__ float rnorm(float ss, int norm, float inv_d, float eps) {
    return norm == KDA_NORM_NONE ? 1.f : rsqrtf((norm == KDA_NORM_RMS ? ss * inv_d : ss) + eps);
}

// One 32-byte sector; a pointer that is 16-byte aligned alone (an output the
// caller cut out of a larger tensor) takes two stores.
__device__ __forceinline__ void st_v8(void *p, const uint32_t (&r)[8]) {
    if (reinterpret_cast<uintptr_t>(p) & 16) {
        uint4 *q = reinterpret_cast<uint4 *>(p);
        q[0] = make_uint4(r[0], r[1], r[2], r[3]);
        q[1] = make_uint4(r[4], r[5], r[6], r[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {  // zeros where not there
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// The blocks' shares of weights' gradients: dst[s][c] = sum over blocks of
// partial[block][s][c], in a fixed order. A lane has a column, a warp every 32nd
// block, so that loads are whole lines and most are on their way at once; then a
// warp adds up a column's 32 sums.
namespace {
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
kda_column_sum_kernel(const float *partial, int blocks, int D, float *d0, float *d1, float *d2) {
    static_assert(WARPS == 32, "a warp adds up a column's sums");
    __shared__ float red[WARPS][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, s = blockIdx.y;
    after_previous();
    float a = 0.f;
    if (c < D) {
#pragma unroll 10
        for (int b = warp; b < blocks; b += WARPS) a += partial[((int64_t)b * gridDim.y + s) * D + c];
    }
    red[warp][lane] = a;
    __syncthreads();
    a = row_sum<32>(red[lane][warp]);
    float *dst = s == 0 ? d0 : s == 1 ? d1 : d2;
    if (lane == 0 && dst && c + warp < D) dst[c + warp] = a;
}
inline cudaError_t column_sum(Launches &l, const float *partial, int blocks, int D, int sets, float *d0,
                              float *d1 = nullptr, float *d2 = nullptr) {
    return l.next(kda_column_sum_kernel<32>, dim3((D + 31) / 32, sets), 1024, 0, partial, blocks, D, d0, d1, d2);
}
}  // namespace

}  // namespace kda
