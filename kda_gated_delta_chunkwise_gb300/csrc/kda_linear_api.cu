// Host side of the linear-attention and query/key norm entry points of
// include/kda.h: argument checks, then launches. Nothing here allocates,
// synchronises or reads device memory; every check comes before the first
// launch of a call.
#include "kda_checks.cuh"
#include "kda_linear.cuh"

using namespace kda;

namespace {

kda_status_t common(kda_dtype_t dt, int decay, int N, int64_t T, int H, int dk, int dv, float scale) {
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown qkv dtype %d", (int)dt);
    if (decay != KDA_DECAY_TOKEN && decay != KDA_DECAY_HEAD && decay != KDA_DECAY_NONE)
        return fail(KDA_ERR_INVALID_ARG, "unknown decay kind %d", decay);
    if (H <= 0) return fail(KDA_ERR_INVALID_ARG, "H must be positive (got %d)", H);
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128))
        return fail(dk > 0 && dv > 0 ? KDA_ERR_UNSUPPORTED : KDA_ERR_INVALID_ARG,
                    "d_k, d_v must be 64 or 128 (got %d, %d)", dk, dv);
    if (N < 0 || T < 0) return fail(KDA_ERR_INVALID_ARG, "the sequence and token counts must be >= 0");
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    return KDA_OK;
}

// The token count, and the grids: one block per (chunk, head) at most, and
// dk * dv / 1024 per (sequence, head).
kda_status_t sizes(int N, int64_t T, int H, bool packed) {
    const int64_t tokens = packed ? T : N * T;
    if (tokens > INT32_MAX) return fail(KDA_ERR_UNSUPPORTED, "the token count must fit in int32");
    const int64_t chunks = packed ? T / kda::kLinChunk + 8ll * N + 8 : N * (T / kda::kLinChunk + 8);
    if (!fits(chunks, H) || !fits(N, H, 16))
        return fail(KDA_ERR_UNSUPPORTED, "the 64-token chunks of all sequences times H must fit in int32");
    return KDA_OK;
}

kda_status_t log_decay_ok(const float *g, int decay) {
    return decay == KDA_DECAY_NONE ? KDA_OK : need(g, "log_decay", 4);
}

// A call on no sequences: of a packed batch with tokens all the same, the
// offsets cannot be right; the sum of a head's gradients over no token is zero.
kda_status_t nothing(const kda::LinArgs &a, bool packed, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (packed) {
        KDA_CHECK(maybe(a.status, "device_status", 4));
        if (a.status)
            e = a.T > 0 ? kda::launch_linear_status(a.status, KDA_DEV_BAD_CU_SEQLENS, s)
                        : cudaMemsetAsync(a.status, 0, sizeof(int32_t), s);
        if (a.T > 0) return cuda_status(e, "status");
    }
    if (e == cudaSuccess && a.d_decay && a.decay == KDA_DECAY_HEAD) {
        KDA_CHECK(need(a.d_decay, "dlog_decay", 4));
        e = cudaMemsetAsync(a.d_decay, 0, sizeof(float) * a.H, s);
    }
    return cuda_status(e, "results of no sequences");
}

kda_status_t prefill(kda::LinArgs a, bool packed, size_t workspace_bytes, cudaStream_t s) {
    KDA_CHECK(common(a.dt, a.decay, a.N, a.T, a.H, a.dk, a.dv, a.scale));
    KDA_CHECK(sizes(a.N, a.T, a.H, packed));
    KDA_CHECK(stride(a.q_stride, a.H, a.dk, a.dt, "q_stride"));
    KDA_CHECK(stride(a.k_stride, a.H, a.dk, a.dt, "k_stride"));
    KDA_CHECK(stride(a.v_stride, a.H, a.dv, a.dt, "v_stride"));
    if (a.N == 0) return nothing(a, packed, s);
    const int64_t tokens = packed ? a.T : (int64_t)a.N * a.T;
    if (packed) {
        KDA_CHECK(need(a.cu_seqlens, "cu_seqlens", 4));
        KDA_CHECK(maybe(a.status, "device_status", 4));
    }
    if (tokens > 0) {
        KDA_CHECK(need(a.q, "q"));
        KDA_CHECK(need(a.k, "k"));
        KDA_CHECK(need(a.v, "v"));
        KDA_CHECK(need(a.o, "o"));
        KDA_CHECK(log_decay_ok(a.log_decay, a.decay));
    }
    KDA_CHECK(maybe(a.s0, "initial_state"));
    KDA_CHECK(maybe(a.sT, "final_state"));
    KDA_CHECK(workspace_ok(a.workspace, workspace_bytes,
                           kda::linear_workspace_bytes(a.N, a.T, a.H, a.dk, a.dv, a.dt, packed)));
    return cuda_status(kda::launch_linear(a, s), "linear prefill launch");
}

kda_status_t backward(kda::LinArgs a, bool packed, size_t workspace_bytes, cudaStream_t s) {
    KDA_CHECK(common(a.dt, a.decay, a.N, a.T, a.H, a.dk, a.dv, a.scale));
    KDA_CHECK(sizes(a.N, a.T, a.H, packed));
    KDA_CHECK(stride(a.q_stride, a.H, a.dk, a.dt, "q_stride"));
    KDA_CHECK(stride(a.k_stride, a.H, a.dk, a.dt, "k_stride"));
    KDA_CHECK(stride(a.v_stride, a.H, a.dv, a.dt, "v_stride"));
    if (a.decay == KDA_DECAY_NONE) a.d_decay = nullptr;
    if (a.N == 0) return nothing(a, packed, s);
    const int64_t tokens = packed ? a.T : (int64_t)a.N * a.T;
    if (packed) {
        KDA_CHECK(need(a.cu_seqlens, "cu_seqlens", 4));
        KDA_CHECK(maybe(a.status, "device_status", 4));
    }
    if (tokens > 0) {
        KDA_CHECK(need(a.q, "q"));
        KDA_CHECK(need(a.k, "k"));
        KDA_CHECK(need(a.v, "v"));
        KDA_CHECK(need(a.d_o, "d_o"));
        KDA_CHECK(need(a.dq, "dq"));
        KDA_CHECK(need(a.dk_out, "dk"));
        KDA_CHECK(need(a.dv_out, "dv"));
        KDA_CHECK(log_decay_ok(a.log_decay, a.decay));
    }
    KDA_CHECK(maybe(a.d_decay, "dlog_decay", 4));
    KDA_CHECK(maybe(a.s0, "initial_state"));
    KDA_CHECK(maybe(a.dsT, "d_final_state"));
    KDA_CHECK(maybe(a.ds0, "d_initial_state"));
    KDA_CHECK(workspace_ok(a.workspace, workspace_bytes,
                           kda::linear_backward_workspace_bytes(a.N, a.T, a.H, a.dk, a.dv, a.dt, packed)));
    return cuda_status(kda::launch_linear_backward(a, s), "linear backward launch");
}

kda_status_t decode(const void *q, const void *k, const void *v, kda_dtype_t dt, int64_t qs, int64_t ks, int64_t vs,
                    const float *g, int decay, float scale, float *state, const int32_t *slots, int pool,
                    int32_t *status, void *o, int N, int H, int dk, int dv, cudaStream_t s) {
    KDA_CHECK(common(dt, decay, N, 1, H, dk, dv, scale));
    KDA_CHECK(stride(qs, H, dk, dt, "q_stride"));
    KDA_CHECK(stride(ks, H, dk, dt, "k_stride"));
    KDA_CHECK(stride(vs, H, dv, dt, "v_stride"));
    if (N == 0) {
        KDA_CHECK(maybe(status, "device_status", 4));
        return cuda_status(status ? cudaMemsetAsync(status, 0, sizeof(int32_t), s) : cudaSuccess, "status reset");
    }
    if (!fits(N, H, 4)) return fail(KDA_ERR_UNSUPPORTED, "N * H * 4 must fit in int32");
    KDA_CHECK(need(q, "q"));
    KDA_CHECK(need(k, "k"));
    KDA_CHECK(need(v, "v"));
    KDA_CHECK(need(o, "o"));
    KDA_CHECK(need(state, slots ? "state_pool" : "state"));
    KDA_CHECK(log_decay_ok(g, decay));
    if (status) {  // KDA_DEV_OK unless a head finds a bad slot
        const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
        if (e != cudaSuccess) return cuda_status(e, "status reset");
    }
    return cuda_status(kda::launch_linear_decode(q, k, v, dt, qs, ks, vs, g, decay, scale, state, slots, pool, status, o,
                                                 N, H, dk, dv, s),
                       "linear decode launch");
}

bool bad_sizes(int N, int64_t T, int H, int dk, int dv, kda_dtype_t dt, bool packed) {
    return common(dt, KDA_DECAY_NONE, N, T, H, dk, dv, 1.f) != KDA_OK || sizes(N, T, H, packed) != KDA_OK;
}

// Several axes: each channel pair's axis, from the caller's array.
kda_status_t axes_of(kda::NormRopeArgs &p, const uint8_t *pair_axis, int axes) {
    if (axes < 1 || axes > kRopeAxes)
        return fail(axes < 1 ? KDA_ERR_INVALID_ARG : KDA_ERR_UNSUPPORTED, "1 to %d axes (got %d)", kRopeAxes, axes);
    if (p.rot <= 0 || p.rot > 128)
        return fail(KDA_ERR_INVALID_ARG, "positions of several axes need a rotary size up to the head size (got %d)", p.rot);
    if (!pair_axis) return fail(KDA_ERR_INVALID_ARG, "pair_axis must not be NULL");
    p.axes = axes;
    p.quads = true;
    for (int i = 0; i < p.rot / 2; ++i) {
        if (pair_axis[i] >= axes)
            return fail(KDA_ERR_INVALID_ARG, "pair_axis[%d] is %d, there are %d axes", i, pair_axis[i], axes);
        p.axis_bits[i >> 5] |= (uint64_t)pair_axis[i] << (2 * (i & 31));
        if (pair_axis[i] != pair_axis[i & ~3]) p.quads = false;
    }
    return KDA_OK;
}

kda_status_t norm_rope(kda::NormRopeArgs &p, int64_t tokens) {
    if (p.dt != KDA_F32 && p.dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)p.dt);
    if (p.norm != KDA_NORM_NONE && p.norm != KDA_NORM_L2 && p.norm != KDA_NORM_RMS)
        return fail(KDA_ERR_INVALID_ARG, "unknown norm kind %d", p.norm);
    if (p.layout != KDA_ROPE_HALF && p.layout != KDA_ROPE_INTERLEAVED)
        return fail(KDA_ERR_INVALID_ARG, "unknown rotary layout %d", p.layout);
    if (tokens < 0 || p.hq < 0 || p.hk < 0)
        return fail(KDA_ERR_INVALID_ARG, "the token and head counts must be >= 0");
    if (p.d != 64 && p.d != 128)
        return fail(p.d > 0 ? KDA_ERR_UNSUPPORTED : KDA_ERR_INVALID_ARG, "the head size must be 64 or 128 (got %d)", p.d);
    if (p.norm != KDA_NORM_NONE && !(p.eps > 0.f && std::isfinite(p.eps)))
        return fail(KDA_ERR_INVALID_ARG, "eps must be positive and finite");
    if (p.rot < 0 || p.rot > p.d || p.rot % 16)
        return fail(p.rot < 0 || p.rot > p.d ? KDA_ERR_INVALID_ARG : KDA_ERR_UNSUPPORTED,
                    "the rotary size must be a multiple of 16 up to the head size (got %d)", p.rot);
    if (p.rot > 0 && p.max_position <= 0) return fail(KDA_ERR_INVALID_ARG, "max_position must be positive");
    KDA_CHECK(stride(p.q_stride, p.hq, p.d, p.dt, "q_stride"));
    KDA_CHECK(stride(p.k_stride, p.hk, p.d, p.dt, "k_stride"));
    // a warp takes four rows of one token at a time at least
    const int64_t units = tokens * (((int64_t)p.hq + 3) / 4 + ((int64_t)p.hk + 3) / 4);
    if (tokens > INT32_MAX || units > INT32_MAX)
        return fail(KDA_ERR_UNSUPPORTED, "too many tokens and heads for one launch");
    p.tokens = tokens;
    if (tokens > 0) {
        if (p.hq > 0) KDA_CHECK(need(p.q, "q"));
        if (p.hk > 0) KDA_CHECK(need(p.k, "k"));
        if (p.rot > 0) {
            KDA_CHECK(need(p.positions, "positions", 4));
            KDA_CHECK(need(p.table, "rope_table"));
        }
    }
    KDA_CHECK(maybe(p.wq, "q_weight"));
    KDA_CHECK(maybe(p.wk, "k_weight"));
    return maybe(p.status, "device_status", 4);
}

kda_status_t norm_rope_forward(kda::NormRopeArgs &p, int64_t tokens, cudaStream_t s) {
    KDA_CHECK(norm_rope(p, tokens));
    if (tokens > 0 && p.hq > 0) KDA_CHECK(need(p.yq, "q_out"));
    if (tokens > 0 && p.hk > 0) KDA_CHECK(need(p.yk, "k_out"));
    if (p.status) {
        const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(int32_t), s);
        if (e != cudaSuccess) return cuda_status(e, "status reset");
    }
    if (tokens == 0 || p.hq + p.hk == 0) return ok();
    return cuda_status(kda::launch_norm_rope(p, false, s), "norm and rotation launch");
}

kda_status_t norm_rope_backward(kda::NormRopeArgs &p, int64_t tokens, void *workspace, size_t workspace_bytes,
                                cudaStream_t s) {
    KDA_CHECK(norm_rope(p, tokens));
    if (tokens > 0 && p.hq > 0) {
        KDA_CHECK(need(p.dyq, "dq_out"));
        KDA_CHECK(need(p.dxq, "dq"));
    }
    if (tokens > 0 && p.hk > 0) {
        KDA_CHECK(need(p.dyk, "dk_out"));
        KDA_CHECK(need(p.dxk, "dk"));
    }
    KDA_CHECK(maybe(p.dwq, "dq_weight", 4));
    KDA_CHECK(maybe(p.dwk, "dk_weight", 4));
    if (p.dwq || p.dwk) {
        KDA_CHECK(workspace_ok(workspace, workspace_bytes, kda_qk_norm_rope_backward_workspace_bytes(p.d)));
        p.partial = static_cast<float *>(workspace);
    }
    cudaError_t e = p.status ? cudaMemsetAsync(p.status, 0, sizeof(int32_t), s) : cudaSuccess;
    if (tokens == 0 || p.hq + p.hk == 0) {  // the sums over no rows
        if (e == cudaSuccess && p.dwq) e = cudaMemsetAsync(p.dwq, 0, sizeof(float) * p.d, s);
        if (e == cudaSuccess && p.dwk) e = cudaMemsetAsync(p.dwk, 0, sizeof(float) * p.d, s);
        return cuda_status(e, "weight gradient reset");
    }
    if (e != cudaSuccess) return cuda_status(e, "status reset");
    return cuda_status(kda::launch_norm_rope(p, true, s), "norm and rotation backward launch");
}

}  // namespace

extern "C" {

size_t kda_linear_prefill_workspace_bytes(int B, int T, int H, int d_k, int d_v, kda_dtype_t dt) {
    return bad_sizes(B, T, H, d_k, d_v, dt, false) ? 0 : kda::linear_workspace_bytes(B, T, H, d_k, d_v, dt, false);
}
size_t kda_linear_varlen_prefill_workspace_bytes(int N, int T_total, int H, int d_k, int d_v, kda_dtype_t dt) {
    return bad_sizes(N, T_total, H, d_k, d_v, dt, true) ? 0
                                                        : kda::linear_workspace_bytes(N, T_total, H, d_k, d_v, dt, true);
}
size_t kda_linear_prefill_backward_workspace_bytes(int B, int T, int H, int d_k, int d_v, kda_dtype_t dt) {
    return bad_sizes(B, T, H, d_k, d_v, dt, false)
               ? 0
               : kda::linear_backward_workspace_bytes(B, T, H, d_k, d_v, dt, false);
}
size_t kda_linear_varlen_prefill_backward_workspace_bytes(int N, int T_total, int H, int d_k, int d_v, kda_dtype_t dt) {
    return bad_sizes(N, T_total, H, d_k, d_v, dt, true)
               ? 0
               : kda::linear_backward_workspace_bytes(N, T_total, H, d_k, d_v, dt, true);
}

kda_status_t kda_linear_prefill(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype, int64_t q_stride,
                                int64_t k_stride, int64_t v_stride, const float *log_decay, kda_decay_t decay,
                                float scale, const float *initial_state, void *o, float *final_state, int B, int T,
                                int H, int d_k, int d_v, void *workspace, size_t workspace_bytes,
                                kda_stream_t stream) {
    kda::LinArgs a{};
    a.dt = qkv_dtype; a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.log_decay = log_decay; a.decay = decay; a.scale = scale;
    a.s0 = initial_state; a.o = o; a.sT = final_state;
    a.N = B; a.T = T; a.H = H; a.dk = d_k; a.dv = d_v;
    a.workspace = workspace;
    return prefill(a, false, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_linear_varlen_prefill(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                                       int64_t q_stride, int64_t k_stride, int64_t v_stride, const float *log_decay,
                                       kda_decay_t decay, float scale, const float *initial_state, void *o,
                                       float *final_state, const int32_t *cu_seqlens, int N, int T_total, int H,
                                       int d_k, int d_v, void *workspace, size_t workspace_bytes,
                                       int32_t *device_status, kda_stream_t stream) {
    kda::LinArgs a{};
    a.dt = qkv_dtype; a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.log_decay = log_decay; a.decay = decay; a.scale = scale;
    a.s0 = initial_state; a.o = o; a.sT = final_state;
    a.N = N; a.T = T_total; a.H = H; a.dk = d_k; a.dv = d_v;
    a.cu_seqlens = cu_seqlens; a.status = device_status; a.workspace = workspace;
    return prefill(a, true, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_linear_prefill_backward(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                                         int64_t q_stride, int64_t k_stride, int64_t v_stride, const float *log_decay,
                                         kda_decay_t decay, float scale, const float *initial_state, const void *d_o,
                                         const float *d_final_state, void *dq, void *dk, void *dv, float *dlog_decay,
                                         float *d_initial_state, int B, int T, int H, int d_k, int d_v,
                                         void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda::LinArgs a{};
    a.dt = qkv_dtype; a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.log_decay = log_decay; a.decay = decay; a.scale = scale;
    a.s0 = initial_state; a.d_o = d_o; a.dsT = d_final_state;
    a.dq = dq; a.dk_out = dk; a.dv_out = dv; a.d_decay = dlog_decay; a.ds0 = d_initial_state;
    a.N = B; a.T = T; a.H = H; a.dk = d_k; a.dv = d_v;
    a.workspace = workspace;
    return backward(a, false, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_linear_varlen_prefill_backward(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                                                int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                                const float *log_decay, kda_decay_t decay, float scale,
                                                const float *initial_state, const void *d_o,
                                                const float *d_final_state, void *dq, void *dk, void *dv,
                                                float *dlog_decay, float *d_initial_state, const int32_t *cu_seqlens,
                                                int N, int T_total, int H, int d_k, int d_v, void *workspace,
                                                size_t workspace_bytes, int32_t *device_status, kda_stream_t stream) {
    kda::LinArgs a{};
    a.dt = qkv_dtype; a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.log_decay = log_decay; a.decay = decay; a.scale = scale;
    a.s0 = initial_state; a.d_o = d_o; a.dsT = d_final_state;
    a.dq = dq; a.dk_out = dk; a.dv_out = dv; a.d_decay = dlog_decay; a.ds0 = d_initial_state;
    a.N = N; a.T = T_total; a.H = H; a.dk = d_k; a.dv = d_v;
    a.cu_seqlens = cu_seqlens; a.status = device_status; a.workspace = workspace;
    return backward(a, true, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_linear_decode_step(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                                    int64_t q_stride, int64_t k_stride, int64_t v_stride, const float *log_decay,
                                    kda_decay_t decay, float scale, float *state, void *o, int N, int H, int d_k,
                                    int d_v, kda_stream_t stream) {
    return decode(q, k, v, qkv_dtype, q_stride, k_stride, v_stride, log_decay, decay, scale, state, nullptr, 0, nullptr,
                  o, N, H, d_k, d_v, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_linear_decode_step_slots(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                                          int64_t q_stride, int64_t k_stride, int64_t v_stride, const float *log_decay,
                                          kda_decay_t decay, float scale, float *state_pool, const int32_t *slots,
                                          int pool_size, void *o, int N, int H, int d_k, int d_v,
                                          int32_t *device_status, kda_stream_t stream) {
    if (N > 0) {
        KDA_CHECK(need(slots, "slots", 4));
        if (pool_size <= 0) return fail(KDA_ERR_INVALID_ARG, "pool_size must be positive");
        if (H > 0 && (int64_t)pool_size * H > INT32_MAX)
            return fail(KDA_ERR_UNSUPPORTED, "pool_size * H must fit in int32");
        KDA_CHECK(maybe(device_status, "device_status", 4));
    }
    return decode(q, k, v, qkv_dtype, q_stride, k_stride, v_stride, log_decay, decay, scale, state_pool, slots,
                  pool_size, device_status, o, N, H, d_k, d_v, reinterpret_cast<cudaStream_t>(stream));
}

#define KDA_ROPE_ARGS                                                                                                 \
    p.dt = dtype; p.q = q; p.k = k; p.q_stride = q_stride; p.k_stride = k_stride;                                      \
    p.positions = positions; p.table = rope_table; p.max_position = max_position; p.rot = rotary; p.layout = layout;   \
    p.wq = q_weight; p.wk = k_weight; p.norm = norm; p.eps = eps; p.hq = H_q; p.hk = H_k; p.d = d;                     \
    p.status = device_status

kda_status_t kda_qk_norm_rope(const void *q, const void *k, kda_dtype_t dtype, int64_t q_stride, int64_t k_stride,
                              const int32_t *positions, const float *rope_table, int max_position, int rotary,
                              kda_rope_layout_t layout, const float *q_weight, const float *k_weight, kda_norm_t norm,
                              float eps, void *q_out, void *k_out, int64_t tokens, int H_q, int H_k, int d,
                              int32_t *device_status, kda_stream_t stream) {
    kda::NormRopeArgs p{};
    KDA_ROPE_ARGS;
    p.yq = q_out; p.yk = k_out;
    return norm_rope_forward(p, tokens, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_qk_norm_rope_axes(const void *q, const void *k, kda_dtype_t dtype, int64_t q_stride, int64_t k_stride,
                                   const int32_t *positions, int axes, const uint8_t *pair_axis, const float *rope_table,
                                   int max_position, int rotary, kda_rope_layout_t layout, const float *q_weight,
                                   const float *k_weight, kda_norm_t norm, float eps, void *q_out, void *k_out,
                                   int64_t tokens, int H_q, int H_k, int d, int32_t *device_status,
                                   kda_stream_t stream) {
    kda::NormRopeArgs p{};
    KDA_ROPE_ARGS;
    p.yq = q_out; p.yk = k_out;
    KDA_CHECK(axes_of(p, pair_axis, axes));
    return norm_rope_forward(p, tokens, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_qk_norm_rope_backward_workspace_bytes(int d) {
    return d > 0 ? (size_t)kda::kNormRopeBwdBlocks * 2 * d * sizeof(float) : 0;
}

kda_status_t kda_qk_norm_rope_backward(const void *q, const void *k, const void *dq_out, const void *dk_out,
                                       kda_dtype_t dtype, int64_t q_stride, int64_t k_stride,
                                       const int32_t *positions, const float *rope_table, int max_position, int rotary,
                                       kda_rope_layout_t layout, const float *q_weight, const float *k_weight,
                                       kda_norm_t norm, float eps, void *dq, void *dk, float *dq_weight,
                                       float *dk_weight, int64_t tokens, int H_q, int H_k, int d, void *workspace,
                                       size_t workspace_bytes, int32_t *device_status, kda_stream_t stream) {
    kda::NormRopeArgs p{};
    KDA_ROPE_ARGS;
    p.dyq = dq_out; p.dyk = dk_out; p.dxq = dq; p.dxk = dk; p.dwq = dq_weight; p.dwk = dk_weight;
    return norm_rope_backward(p, tokens, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

kda_status_t kda_qk_norm_rope_axes_backward(const void *q, const void *k, const void *dq_out, const void *dk_out,
                                            kda_dtype_t dtype, int64_t q_stride, int64_t k_stride,
                                            const int32_t *positions, int axes, const uint8_t *pair_axis,
                                            const float *rope_table, int max_position, int rotary,
                                            kda_rope_layout_t layout, const float *q_weight, const float *k_weight,
                                            kda_norm_t norm, float eps, void *dq, void *dk, float *dq_weight,
                                            float *dk_weight, int64_t tokens, int H_q, int H_k, int d, void *workspace,
                                            size_t workspace_bytes, int32_t *device_status, kda_stream_t stream) {
    kda::NormRopeArgs p{};
    KDA_ROPE_ARGS;
    p.dyq = dq_out; p.dyk = dk_out; p.dxq = dq; p.dxk = dk; p.dwq = dq_weight; p.dwk = dk_weight;
    KDA_CHECK(axes_of(p, pair_axis, axes));
    return norm_rope_backward(p, tokens, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
