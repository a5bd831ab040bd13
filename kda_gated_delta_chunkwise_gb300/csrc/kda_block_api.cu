// Host side of the entry points for the norms around a block (kda_gated_norm*,
// kda_residual_norm* of include/kda.h): argument checks, then launches.
#include "kda_block_norm.cuh"
#include "kda_checks.cuh"

using namespace kda;

namespace {

kda_status_t norm_kind(int norm, float eps, const char *name) {
    if (norm != KDA_NORM_NONE && norm != KDA_NORM_L2 && norm != KDA_NORM_RMS)
        return fail(KDA_ERR_INVALID_ARG, "unknown %s kind %d", name, norm);
    if (norm != KDA_NORM_NONE && !(eps > 0.f && std::isfinite(eps)))
        return fail(KDA_ERR_INVALID_ARG, "eps must be positive and finite");
    return KDA_OK;
}

kda_status_t gated(GatedArgs &p) {
    if (p.dt != KDA_F32 && p.dt != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)p.dt);
    KDA_CHECK(norm_kind(p.norm, p.eps, "norm"));
    if (p.act != KDA_ACT_SIGMOID && p.act != KDA_ACT_SILU)
        return fail(KDA_ERR_INVALID_ARG, "unknown activation %d", p.act);
    if (p.tokens < 0 || p.h < 0) return fail(KDA_ERR_INVALID_ARG, "the token and head counts must be >= 0");
    if (p.d != 64 && p.d != 128)
        return fail(p.d > 0 ? KDA_ERR_UNSUPPORTED : KDA_ERR_INVALID_ARG, "the head size must be 64 or 128 (got %d)", p.d);
    if (!fits(p.tokens, p.h)) return fail(KDA_ERR_UNSUPPORTED, "tokens * H must fit in int32");
    KDA_CHECK(stride(p.x_stride, p.h, p.d, p.dt, "x_stride"));
    KDA_CHECK(stride(p.g_stride, p.h, p.d, p.dt, "gate_stride"));
    KDA_CHECK(maybe(p.w, "weight"));
    if (p.tokens * p.h > 0) {
        KDA_CHECK(need(p.x, "x"));
        KDA_CHECK(need(p.gate, "gate"));
    }
    p.by_heads = FastDiv(p.h > 0 ? p.h : 1);
    return KDA_OK;
}

kda_status_t residual(const ResidualArgs &p) {
    for (const kda_dtype_t t : {p.stream_dt, p.dt})
        if (t != KDA_F32 && t != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)t);
    if (p.dt == KDA_F32 && p.stream_dt != KDA_F32)
        return fail(KDA_ERR_UNSUPPORTED, "a float32 branch needs a float32 residual stream");
    KDA_CHECK(norm_kind(p.branch_norm, p.eps, "branch norm"));
    if (!(p.eps > 0.f && std::isfinite(p.eps))) return fail(KDA_ERR_INVALID_ARG, "eps must be positive and finite");
    if (!std::isfinite(p.scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    if (p.tokens < 0 || p.tokens > INT32_MAX)
        return fail(p.tokens < 0 ? KDA_ERR_INVALID_ARG : KDA_ERR_UNSUPPORTED, "the token count must be >= 0 and fit in int32");
    if (p.D <= 0 || p.D % 8 || p.D > kResidualMaxWidth)
        return fail(p.D <= 0 ? KDA_ERR_INVALID_ARG : KDA_ERR_UNSUPPORTED,
                    "the width must be a multiple of 8 up to %d (got %d)", kResidualMaxWidth, p.D);
    KDA_CHECK(maybe(p.w, "weight"));
    KDA_CHECK(maybe(p.wb, "branch_weight"));
    return maybe(p.c, "channel_scale");
}

}  // namespace

extern "C" {

kda_status_t kda_gated_norm(const void *x, const void *gate, kda_dtype_t dtype, int64_t x_stride, int64_t gate_stride,
                            const float *weight, kda_norm_t norm, kda_activation_t activation, float eps, void *out,
                            int64_t tokens, int H, int d, kda_stream_t stream) {
    GatedArgs p{};
    p.dt = dtype; p.x = x; p.gate = gate; p.x_stride = x_stride; p.g_stride = gate_stride;
    p.w = weight; p.norm = norm; p.act = activation; p.eps = eps; p.y = out; p.tokens = tokens; p.h = H; p.d = d;
    KDA_CHECK(gated(p));
    if (tokens == 0 || H == 0) return ok();
    KDA_CHECK(need(out, "out"));
    return cuda_status(launch_gated_norm(p, false, reinterpret_cast<cudaStream_t>(stream)), "gated norm launch");
}

size_t kda_gated_norm_backward_workspace_bytes(int d) {
    return d > 0 ? (size_t)kGatedBwdBlocks * d * sizeof(float) : 0;
}

kda_status_t kda_gated_norm_backward(const void *x, const void *gate, const void *d_out, kda_dtype_t dtype,
                                     int64_t x_stride, int64_t gate_stride, const float *weight, kda_norm_t norm,
                                     kda_activation_t activation, float eps, void *dx, void *dgate, float *dweight,
                                     int64_t tokens, int H, int d, void *workspace, size_t workspace_bytes,
                                     kda_stream_t stream) {
    GatedArgs p{};
    p.dt = dtype; p.x = x; p.gate = gate; p.x_stride = x_stride; p.g_stride = gate_stride; p.dy = d_out;
    p.w = weight; p.norm = norm; p.act = activation; p.eps = eps; p.dx = dx; p.dgate = dgate; p.dw = dweight;
    p.tokens = tokens; p.h = H; p.d = d;
    KDA_CHECK(gated(p));
    KDA_CHECK(maybe(dweight, "dweight", 4));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0 || H == 0)  // the sum over no rows
        return cuda_status(dweight ? cudaMemsetAsync(dweight, 0, sizeof(float) * d, s) : cudaSuccess,
                           "weight gradient reset");
    KDA_CHECK(need(d_out, "d_out"));
    KDA_CHECK(need(dx, "dx"));
    KDA_CHECK(need(dgate, "dgate"));
    if (dweight) {
        KDA_CHECK(workspace_ok(workspace, workspace_bytes, kda_gated_norm_backward_workspace_bytes(d)));
        p.partial = static_cast<float *>(workspace);
    }
    return cuda_status(launch_gated_norm(p, true, s), "gated norm backward launch");
}

kda_status_t kda_residual_norm(const void *residual_in, const void *branch, kda_dtype_t stream_dtype, kda_dtype_t dtype,
                               const float *weight, kda_norm_t branch_norm, const float *branch_weight,
                               const float *channel_scale, float scale, float eps, void *hidden, void *out,
                               int64_t tokens, int D, kda_stream_t stream) {
    ResidualArgs p{};
    p.stream_dt = stream_dtype; p.dt = dtype; p.x = residual_in; p.b = branch;
    p.w = weight; p.branch_norm = branch_norm; p.wb = branch_weight; p.c = channel_scale;
    p.scale = scale; p.eps = eps; p.h = hidden; p.y = out; p.tokens = tokens; p.D = D;
    KDA_CHECK(residual(p));
    if (tokens == 0) return ok();
    KDA_CHECK(need(residual_in, "residual"));
    KDA_CHECK(need(branch, "branch"));
    KDA_CHECK(need(hidden, "hidden"));
    KDA_CHECK(need(out, "out"));
    return cuda_status(launch_residual_norm(p, false, reinterpret_cast<cudaStream_t>(stream)), "residual norm launch");
}

size_t kda_residual_norm_backward_workspace_bytes(int D) {
    return D > 0 && D <= kResidualMaxWidth ? (size_t)kResidualBwdBlocks * 3 * D * sizeof(float) : 0;
}

kda_status_t kda_residual_norm_backward(const void *hidden, const void *branch, const void *d_out, const void *d_hidden,
                                        kda_dtype_t stream_dtype, kda_dtype_t dtype, const float *weight,
                                        kda_norm_t branch_norm, const float *branch_weight, const float *channel_scale,
                                        float scale, float eps, void *d_residual, void *d_branch, float *dweight,
                                        float *dbranch_weight, float *dchannel_scale, int64_t tokens, int D,
                                        void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    ResidualArgs p{};
    p.stream_dt = stream_dtype; p.dt = dtype; p.x = hidden; p.b = branch; p.dy = d_out; p.dh = d_hidden;
    p.w = weight; p.branch_norm = branch_norm; p.wb = branch_weight; p.c = channel_scale;
    p.scale = scale; p.eps = eps; p.dx = d_residual; p.db = d_branch;
    p.dw = dweight; p.dwb = dbranch_weight; p.dc = dchannel_scale; p.tokens = tokens; p.D = D;
    KDA_CHECK(residual(p));
    float *const sums[3] = {dweight, dbranch_weight, dchannel_scale};
    const char *const names[3] = {"dweight", "dbranch_weight", "dchannel_scale"};
    for (int i = 0; i < 3; ++i) KDA_CHECK(maybe(sums[i], names[i], 4));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0) {  // the sums over no rows
        cudaError_t e = cudaSuccess;
        for (float *d : sums)
            if (d && e == cudaSuccess) e = cudaMemsetAsync(d, 0, sizeof(float) * D, s);
        return cuda_status(e, "weight gradient reset");
    }
    KDA_CHECK(need(hidden, "hidden"));
    KDA_CHECK(need(d_out, "d_out"));
    KDA_CHECK(maybe(d_hidden, "d_hidden"));
    KDA_CHECK(need(d_residual, "d_residual"));
    KDA_CHECK(need(d_branch, "d_branch"));
    if (branch_norm != KDA_NORM_NONE || branch_weight || channel_scale || dbranch_weight || dchannel_scale)
        KDA_CHECK(need(branch, "branch"));
    if (dweight || dbranch_weight || dchannel_scale) {
        KDA_CHECK(workspace_ok(workspace, workspace_bytes, kda_residual_norm_backward_workspace_bytes(D)));
        p.partial = static_cast<float *>(workspace);
    }
    return cuda_status(launch_residual_norm(p, true, s), "residual norm backward launch");
}

}  // extern "C"
