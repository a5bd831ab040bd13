// Host side of window attention (kda_window_* of include/kda.h): argument
// checks, then launches. Nothing here allocates, synchronises or reads device
// memory; every check comes before the first launch of a call.
#include "kda_checks.cuh"
#include "kda_window.cuh"

using namespace kda;

namespace {

kda_status_t common(kda_dtype_t dt, int N, int64_t T, int hq, int hk, int d, int sinks) {
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (hq <= 0 || hk <= 0 || hq % hk)
        return fail(KDA_ERR_INVALID_ARG, "H_q must be a positive multiple of H_k (got %d, %d)", hq, hk);
    if (d != 64 && d != 128)
        return fail(d > 0 ? KDA_ERR_UNSUPPORTED : KDA_ERR_INVALID_ARG, "the head size must be 64 or 128 (got %d)", d);
    if (N < 0 || T < 0) return fail(KDA_ERR_INVALID_ARG, "the sequence and token counts must be >= 0");
    if (sinks < 0 || sinks > kWinMaxSinks)
        return fail(sinks < 0 ? KDA_ERR_INVALID_ARG : KDA_ERR_UNSUPPORTED, "0 to %d sinks (got %d)", kWinMaxSinks, sinks);
    return KDA_OK;
}
// The tokens, and the largest grid: six blocks to a tile of 256 tokens and head.
kda_status_t sizes(int N, int64_t T, int hq, bool packed) {
    const int64_t tokens = packed ? T : N * T;
    if (tokens > 1 << 30) return fail(KDA_ERR_UNSUPPORTED, "2^30 tokens at most");
    const int64_t tiles = packed ? T / kWinTile + N : N * ((T + kWinTile - 1) / kWinTile);
    if (hq > 1024) return fail(KDA_ERR_UNSUPPORTED, "1024 query heads at most (got %d)", hq);
    if (!fits(tiles, 6, hq) || !fits(N, hq))
        return fail(KDA_ERR_UNSUPPORTED, "the 256-token tiles of all sequences times 6 H_q must fit in int32");
    return KDA_OK;
}
kda_status_t strides(int64_t &q, int64_t &k, int64_t &v, int hq, int hk, int d, kda_dtype_t dt) {
    KDA_CHECK(stride(q, hq, d, dt, "q_stride"));
    KDA_CHECK(stride(k, hk, d, dt, "k_stride"));
    return stride(v, hk, d, dt, "v_stride");
}

// A row's largest score is that of its largest product: the scale comes after.
kda_status_t scale_ok(float scale) {
    return scale > 0.f && std::isfinite(scale) ? KDA_OK
                                               : fail(KDA_ERR_INVALID_ARG, "scale must be positive and finite");
}

kda_status_t attention(WinArgs &a, bool packed, bool back, size_t workspace_bytes, cudaStream_t s) {
    KDA_CHECK(common(a.dt, a.N, a.T, a.hq, a.hk, a.d, a.sinks));
    KDA_CHECK(sizes(a.N, a.T, a.hq, packed));
    if (a.window < 1) return fail(KDA_ERR_INVALID_ARG, "window must be positive (got %d)", a.window);
    KDA_CHECK(scale_ok(a.scale));
    KDA_CHECK(strides(a.q_stride, a.k_stride, a.v_stride, a.hq, a.hk, a.d, a.dt));
    if (a.T > 0 && a.window > a.T) a.window = a.T;  // as good as any longer one
    const int64_t tokens = packed ? a.T : (int64_t)a.N * a.T;
    if (packed) {
        KDA_CHECK(maybe(a.status, "device_status", 4));
        if (a.N == 0)  // of no sequences with tokens all the same the offsets cannot be right
            return cuda_status(!a.status ? cudaSuccess
                               : a.T > 0 ? launch_linear_status(a.status, KDA_DEV_BAD_CU_SEQLENS, s)
                                         : cudaMemsetAsync(a.status, 0, sizeof(int32_t), s),
                               "status");
        KDA_CHECK(need(a.cu_seqlens, "cu_seqlens", 4));
    }
    if (tokens > 0) {
        KDA_CHECK(need(a.q, "q"));
        KDA_CHECK(need(a.k, "k"));
        KDA_CHECK(need(a.v, "v"));
        if (back) {
            KDA_CHECK(need(a.out, "o"));
            KDA_CHECK(need(a.lse, "lse", 4));
            KDA_CHECK(need(a.d_o, "d_o"));
            KDA_CHECK(need(a.dq, "dq"));
            KDA_CHECK(need(a.dk, "dk"));
            KDA_CHECK(need(a.dv, "dv"));
        } else {
            KDA_CHECK(need(a.o, "o"));
            KDA_CHECK(maybe(a.lse, "lse", 4));
        }
    } else if (!packed) {
        return ok();
    }
    KDA_CHECK(workspace_ok(a.workspace, workspace_bytes,
                           window_workspace_bytes(a.N, a.T, a.hq, a.hk, a.d, a.sinks, a.dt, packed, back)));
    return back ? cuda_status(launch_window_backward(a, s), "window attention backward launch")
                : cuda_status(launch_window(a, s), "window attention launch");
}

size_t workspace_bytes(int N, int64_t T, int hq, int hk, int d, int sinks, kda_dtype_t dt, bool packed, bool back) {
    if (common(dt, N, T, hq, hk, d, sinks) != KDA_OK || sizes(N, T, hq, packed) != KDA_OK) return 0;
    return window_workspace_bytes(N, T, hq, hk, d, sinks, dt, packed, back);
}

kda_status_t cache(WinCacheArgs &a) {
    KDA_CHECK(common(a.dt, a.N, a.T, a.hq, a.hk, a.d, a.sinks));
    if (a.entries <= a.sinks)
        return fail(KDA_ERR_INVALID_ARG, "a slot must have more entries than sinks (got %d, %d)", a.entries, a.sinks);
    if (a.pool <= 0) return fail(KDA_ERR_INVALID_ARG, "pool_size must be positive");
    if (a.hq > 1024) return fail(KDA_ERR_UNSUPPORTED, "1024 query heads at most (got %d)", a.hq);
    KDA_CHECK(maybe(a.status, "device_status", 4));
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_window_attention(const void *q, const void *k, const void *v, kda_dtype_t dtype, int64_t q_stride,
                                  int64_t k_stride, int64_t v_stride, float scale, int window, int sinks, void *o,
                                  float *lse, int B, int T, int H_q, int H_k, int d, kda_stream_t stream) {
    WinArgs a{};
    a.dt = dtype; a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.scale = scale; a.window = window; a.sinks = sinks; a.o = o; a.lse = lse;
    a.N = B; a.T = T; a.hq = H_q; a.hk = H_k; a.d = d;
    return attention(a, false, false, 0, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_window_varlen_attention_workspace_bytes(int N, int T_total, int H_q, int H_k, int d) {
    return workspace_bytes(N, T_total, H_q, H_k, d, 0, KDA_F32, true, false);
}

kda_status_t kda_window_varlen_attention(const void *q, const void *k, const void *v, kda_dtype_t dtype,
                                         int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale, int window,
                                         int sinks, void *o, float *lse, const int32_t *cu_seqlens, int N, int T_total,
                                         int H_q, int H_k, int d, void *workspace, size_t workspace_bytes,
                                         int32_t *device_status, kda_stream_t stream) {
    WinArgs a{};
    a.dt = dtype; a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.scale = scale; a.window = window; a.sinks = sinks; a.o = o; a.lse = lse;
    a.cu_seqlens = cu_seqlens; a.N = N; a.T = T_total; a.hq = H_q; a.hk = H_k; a.d = d;
    a.workspace = workspace; a.status = device_status;
    return attention(a, true, false, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_window_attention_backward_workspace_bytes(int B, int T, int H_q, int H_k, int d, int sinks, kda_dtype_t dtype) {
    return workspace_bytes(B, T, H_q, H_k, d, sinks, dtype, false, true);
}

kda_status_t kda_window_attention_backward(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                           const void *d_o, kda_dtype_t dtype, int64_t q_stride, int64_t k_stride,
                                           int64_t v_stride, float scale, int window, int sinks, void *dq, void *dk,
                                           void *dv, int B, int T, int H_q, int H_k, int d, void *workspace,
                                           size_t workspace_bytes, kda_stream_t stream) {
    WinArgs a{};
    a.dt = dtype; a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.scale = scale; a.window = window; a.sinks = sinks; a.out = o; a.lse = const_cast<float *>(lse); a.d_o = d_o;
    a.dq = dq; a.dk = dk; a.dv = dv; a.N = B; a.T = T; a.hq = H_q; a.hk = H_k; a.d = d; a.workspace = workspace;
    return attention(a, false, true, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_window_varlen_attention_backward_workspace_bytes(int N, int T_total, int H_q, int H_k, int d, int sinks,
                                                            kda_dtype_t dtype) {
    return workspace_bytes(N, T_total, H_q, H_k, d, sinks, dtype, true, true);
}

kda_status_t kda_window_varlen_attention_backward(const void *q, const void *k, const void *v, const void *o,
                                                  const float *lse, const void *d_o, kda_dtype_t dtype, int64_t q_stride,
                                                  int64_t k_stride, int64_t v_stride, float scale, int window, int sinks,
                                                  void *dq, void *dk, void *dv, const int32_t *cu_seqlens, int N,
                                                  int T_total, int H_q, int H_k, int d, void *workspace,
                                                  size_t workspace_bytes, int32_t *device_status, kda_stream_t stream) {
    WinArgs a{};
    a.dt = dtype; a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.scale = scale; a.window = window; a.sinks = sinks; a.out = o; a.lse = const_cast<float *>(lse); a.d_o = d_o;
    a.dq = dq; a.dk = dk; a.dv = dv; a.cu_seqlens = cu_seqlens; a.N = N; a.T = T_total; a.hq = H_q; a.hk = H_k; a.d = d;
    a.workspace = workspace; a.status = device_status;
    return attention(a, true, true, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_window_cache_write(const void *k, const void *v, kda_dtype_t dtype, int64_t k_stride, int64_t v_stride,
                                    const int32_t *cu_seqlens, const int32_t *slots, int sinks, void *k_cache,
                                    void *v_cache, int pool_size, int entries, int N, int T_total, int H_k, int d,
                                    int32_t *device_status, kda_stream_t stream) {
    WinCacheArgs a{};
    a.dt = dtype; a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride; a.cu_seqlens = cu_seqlens;
    a.slots = slots; a.sinks = sinks; a.k_cache = k_cache; a.v_cache = v_cache; a.pool = pool_size; a.entries = entries;
    a.N = N; a.T = T_total; a.hq = a.hk = H_k; a.d = d; a.status = device_status;
    KDA_CHECK(cache(a));
    int64_t none = 0;
    KDA_CHECK(strides(none, a.k_stride, a.v_stride, H_k, H_k, d, dtype));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0)
        return cuda_status(!device_status ? cudaSuccess
                           : T_total > 0 ? launch_linear_status(device_status, KDA_DEV_BAD_CU_SEQLENS, s)
                                         : cudaMemsetAsync(device_status, 0, sizeof(int32_t), s),
                           "status");
    if (N > 65535) return fail(KDA_ERR_UNSUPPORTED, "65535 sequences at most (got %d)", N);
    KDA_CHECK(need(cu_seqlens, "cu_seqlens", 4));
    KDA_CHECK(need(slots, "slots", 4));
    if (T_total > 0) {
        KDA_CHECK(need(k, "k"));
        KDA_CHECK(need(v, "v"));
    }
    KDA_CHECK(need(k_cache, "k_cache"));
    KDA_CHECK(need(v_cache, "v_cache"));
    if (device_status) {
        const cudaError_t e = cudaMemsetAsync(device_status, 0, sizeof(int32_t), s);
        if (e != cudaSuccess) return cuda_status(e, "status reset");
    }
    return cuda_status(launch_window_cache_write(a, s), "window cache write launch");
}

kda_status_t kda_window_decode_step(const void *q, const void *k, const void *v, kda_dtype_t dtype, int64_t q_stride,
                                    int64_t k_stride, int64_t v_stride, float scale, int sinks, void *k_cache,
                                    void *v_cache, int pool_size, int entries, const int32_t *slots,
                                    const int32_t *positions, void *o, int N, int H_q, int H_k, int d,
                                    int32_t *device_status, kda_stream_t stream) {
    WinCacheArgs a{};
    a.dt = dtype; a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.scale = scale; a.sinks = sinks; a.k_cache = k_cache; a.v_cache = v_cache; a.pool = pool_size; a.entries = entries;
    a.slots = slots; a.positions = positions; a.o = o; a.N = N; a.T = 1; a.hq = H_q; a.hk = H_k; a.d = d;
    a.status = device_status;
    KDA_CHECK(cache(a));
    KDA_CHECK(strides(a.q_stride, a.k_stride, a.v_stride, H_q, H_k, d, dtype));
    KDA_CHECK(scale_ok(scale));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N > 0) {
        if (!fits(N, H_k, 16) || !fits(N, H_q)) return fail(KDA_ERR_UNSUPPORTED, "N * H_k * 16 must fit in int32");
        KDA_CHECK(need(q, "q"));
        KDA_CHECK(need(k, "k"));
        KDA_CHECK(need(v, "v"));
        KDA_CHECK(need(o, "o"));
        KDA_CHECK(need(slots, "slots", 4));
        KDA_CHECK(need(positions, "positions", 4));
        KDA_CHECK(need(k_cache, "k_cache"));
        KDA_CHECK(need(v_cache, "v_cache"));
    }
    if (device_status) {  // KDA_DEV_OK unless a sequence finds a bad slot or position
        const cudaError_t e = cudaMemsetAsync(device_status, 0, sizeof(int32_t), s);
        if (e != cudaSuccess) return cuda_status(e, "status reset");
    }
    return N == 0 ? ok() : cuda_status(launch_window_decode(a, s), "window decode launch");
}

}  // extern "C"
