// What the kernels built of roles share (warps that meet at mbarriers, one CTA
// per SM): bounded waits with an abort flag, bf16 pairs, MMA descriptors of whole
// tiles, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_rows.cuh"
#include "kda_linear.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

__device__ int g_tc_error;  // of the including file's kernels

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
                atomicOr(&g_tc_error, 1);
                return false;
            }
        }
        return true;
    }
    // The same with the waiting itself out of line, for roles whose loops are to stay short for the instruction
    // cache; all lanes of a warp.
    __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity) const {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (*flag) return false;
            if (clock64() - t0 > kWaitCycles) {
                *flag = 1;
                atomicOr(&g_tc_error, 1);
                return false;
            }
        }
        return true;
    }
    __device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_on(bar, parity));
    }
};
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
// `bytes` in a row, a multiple of 16, both addresses 16-byte aligned.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
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
// D[tmem] (+)= A[tmem] * B[smem]: A holds two bf16 of K per 32-bit column.
template <bool ACC = true>
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "n"(ACC ? 1 : 0)
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
int sm_count() {
    static int n = [] {
        int dev = 0, v = 152;
        if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        return v;
    }();
    return n;
}

// Reads (and optionally clears) the error word of this file's waits.
cudaError_t read_tc_error(int *out, bool reset) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tc_error, sizeof(int));
    if (e != cudaSuccess) return e;
    *out = v;
    if (reset && v) {
        const int z = 0;
        e = cudaMemcpyToSymbol(g_tc_error, &z, sizeof(int));
    }
    return e;
}

}  // namespace
}  // namespace kda
