// updater_api.hip -- the ABI calls of the learned updater's operators: argument checks and launches.
#include <cmath>

#include "gsr_internal.hpp"

using namespace gsr;

namespace {

constexpr int64_t kMaxRows = (1ll << 31) - 512;
constexpr int64_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxStride = 1 << 21;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t elem(int dtype) { return dtype == GS_F32 ? 4 : 2; }

gs_status launched(hipError_t e, const char* where) {
    return e == hipSuccess ? GS_OK : fail(GS_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

// an array of rows x width elements with a row stride; may be null when it has no elements
gs_status check_array(const char* call, const char* name, const void* p, int64_t rows, int64_t width, int64_t ld,
                      size_t align) {
    if (rows == 0) return GS_OK;
    if (!p) return fail(GS_ERR_INVALID_ARGUMENT, "%s: %s is null", call, name);
    if (!aligned(p, align)) return fail(GS_ERR_INVALID_ARGUMENT, "%s: %s is not %zu-byte aligned", call, name, align);
    if (ld < width)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: row stride %lld of %s is below its width %lld", call, (long long)ld,
                    name, (long long)width);
    if (ld > kMaxStride)
        return fail(GS_ERR_UNSUPPORTED, "%s: row stride %lld of %s exceeds %lld", call, (long long)ld, name,
                    (long long)kMaxStride);
    return GS_OK;
}

gs_status check_workspace(const char* call, const void* ws, size_t have, size_t need) {
    if (need == 0) return GS_OK;
    if (!ws || !aligned(ws, 256))
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: workspace is null or not 256-byte aligned", call);
    if (have < need)
        return fail(GS_ERR_WORKSPACE_TOO_SMALL, "%s: needs %zu bytes of workspace, got %zu", call, need, have);
    return GS_OK;
}

#define GSR_CHECK(x)                   \
    do {                               \
        gs_status s_ = (x);            \
        if (s_ != GS_OK) return s_;    \
    } while (0)

gs_status check_dtype(const char* call, int dtype) {
    if (dtype != GS_F32 && dtype != GS_BF16 && dtype != GS_F16)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", call, dtype);
    return GS_OK;
}

gs_status check_ffn(const char* call, const gs_ffn_dims* d) {
    if (!d) return fail(GS_ERR_INVALID_ARGUMENT, "%s: dims is null", call);
    GSR_CHECK(check_dtype(call, d->dtype));
    if (d->activation != GS_ACT_SILU && d->activation != GS_ACT_GELU)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: unknown activation %d", call, d->activation);
    if (d->rows < 0 || d->d_in < 1 || d->d_hidden < 1 || d->d_out < 1)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: rows %lld, d_in %d, d_hidden %d, d_out %d", call,
                    (long long)d->rows, d->d_in, d->d_hidden, d->d_out);
    if (d->rows > kMaxRows || d->d_in > kMaxWidth || d->d_hidden > kMaxWidth || d->d_out > kMaxWidth)
        return fail(GS_ERR_UNSUPPORTED, "%s: rows %lld, d_in %d, d_hidden %d, d_out %d exceed the limits", call,
                    (long long)d->rows, d->d_in, d->d_hidden, d->d_out);
    return GS_OK;
}

gs_status check_ffn_weights(const char* call, const gs_ffn_dims* d, const gs_ffn_weights* w) {
    if (!w) return fail(GS_ERR_INVALID_ARGUMENT, "%s: weights is null", call);
    const size_t e = elem(d->dtype);
    GSR_CHECK(check_array(call, "weights.gate", w->gate, d->d_hidden, d->d_in, d->d_in, e));
    GSR_CHECK(check_array(call, "weights.up", w->up, d->d_hidden, d->d_in, d->d_in, e));
    return check_array(call, "weights.down", w->down, d->d_out, d->d_hidden, d->d_hidden, e);
}

gs_status check_scan(const char* call, const gs_scan_dims* d) {
    if (!d) return fail(GS_ERR_INVALID_ARGUMENT, "%s: dims is null", call);
    GSR_CHECK(check_dtype(call, d->dtype));
    if (d->rows < 0 || d->n_seq < 0 || d->channels < 1)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: rows %lld, n_seq %lld, channels %d", call, (long long)d->rows,
                    (long long)d->n_seq, d->channels);
    if (d->rows > kMaxRows || d->n_seq > kMaxRows || d->channels > kMaxWidth)
        return fail(GS_ERR_UNSUPPORTED, "%s: rows %lld, n_seq %lld, channels %d exceed the limits", call,
                    (long long)d->rows, (long long)d->n_seq, d->channels);
    return GS_OK;
}

gs_status check_scan_inputs(const char* call, const gs_scan_dims* d, const int64_t* offsets,
                            const gs_scan_inputs* in) {
    if (!in) return fail(GS_ERR_INVALID_ARGUMENT, "%s: inputs is null", call);
    if (!aligned(offsets, 8)) return fail(GS_ERR_INVALID_ARGUMENT, "%s: offsets is not 8-byte aligned", call);
    if (d->rows > 0 && d->n_seq == 0)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: %lld rows but no sequence", call, (long long)d->rows);
    if (!offsets && d->n_seq > 0 && d->rows % d->n_seq != 0)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: %lld rows are not %lld sequences of equal length", call,
                    (long long)d->rows, (long long)d->n_seq);
    const size_t e = elem(d->dtype);
    GSR_CHECK(check_array(call, "gate", in->gate, d->rows, d->channels, in->ld_gate, e));
    GSR_CHECK(check_array(call, "x", in->x, d->rows, d->channels, in->ld_x, e));
    if (!aligned(in->h0, 4)) return fail(GS_ERR_INVALID_ARGUMENT, "%s: h0 is not 4-byte aligned", call);
    return GS_OK;
}

// States that go in and out may be one array, but not parts of each other's: a sequence's result would replace what
// another one still reads.
gs_status check_in_place(const char* call, const gs_scan_dims* d, const char* in_name, const float* in,
                         const char* out_name, const float* out) {
    const uintptr_t a = (uintptr_t)in, b = (uintptr_t)out, n = (uintptr_t)d->n_seq * (uintptr_t)d->channels * 4;
    if (!in || !out || a == b || a + n <= b || b + n <= a) return GS_OK;
    return fail(GS_ERR_INVALID_ARGUMENT, "%s: %s overlaps %s without being it", call, out_name, in_name);
}

gs_status check_ortho(const char* call, const gs_ortho_dims* d) {
    if (!d) return fail(GS_ERR_INVALID_ARGUMENT, "%s: dims is null", call);
    for (int t : {d->dtype, d->out_dtype})
        if (t != GS_F32 && t != GS_BF16)
            return fail(GS_ERR_INVALID_ARGUMENT, "%s: dtype %d (GS_F32 or GS_BF16 here)", call, t);
    if (d->rows < 1 || d->cols < 1 || d->batch < 0 || d->steps < 1)
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: rows %lld, cols %lld, batch %d, steps %d", call,
                    (long long)d->rows, (long long)d->cols, d->batch, d->steps);
    const int64_t lo = d->rows < d->cols ? d->rows : d->cols, hi = d->rows < d->cols ? d->cols : d->rows;
    if (lo > (1 << 15) || hi > kMaxWidth || d->batch > 65535 || d->steps > 64)
        return fail(GS_ERR_UNSUPPORTED, "%s: rows %lld, cols %lld, batch %d, steps %d exceed the limits", call,
                    (long long)d->rows, (long long)d->cols, d->batch, d->steps);
    if (!(d->eps > 0.f)) return fail(GS_ERR_INVALID_ARGUMENT, "%s: eps must be positive", call);
    if (!std::isfinite(d->a) || !std::isfinite(d->b) || !std::isfinite(d->c))
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: a coefficient is not finite", call);
    float xs, ps;
    if (!ortho_scales(*d, &xs, &ps))
        return fail(GS_ERR_UNSUPPORTED, "%s: %d steps with coefficients %g, %g, %g leave float16's range", call,
                    d->steps, (double)d->a, (double)d->b, (double)d->c);
    return GS_OK;
}

}  // namespace

extern "C" {

gs_status gs_ffn_sizes(const gs_ffn_dims* dims, size_t* saved_bytes, size_t* forward_bytes, size_t* backward_bytes) {
    GSR_CHECK(check_ffn("gs_ffn_sizes", dims));
    size_t s, f, b;
    ffn_sizes(*dims, &s, &f, &b);
    if (saved_bytes) *saved_bytes = s;
    if (forward_bytes) *forward_bytes = f;
    if (backward_bytes) *backward_bytes = b;
    return GS_OK;
}

gs_status gs_ffn_forward(const gs_ffn_dims* dims, const void* x, int64_t ld_x, const gs_ffn_weights* weights, void* y,
                         int64_t ld_y, void* saved, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const char* call = "gs_ffn_forward";
    GSR_CHECK(check_ffn(call, dims));
    const size_t e = elem(dims->dtype);
    GSR_CHECK(check_ffn_weights(call, dims, weights));
    GSR_CHECK(check_array(call, "x", x, dims->rows, dims->d_in, ld_x, e));
    GSR_CHECK(check_array(call, "y", y, dims->rows, dims->d_out, ld_y, e));
    if (!aligned(saved, 256)) return fail(GS_ERR_INVALID_ARGUMENT, "%s: saved is not 256-byte aligned", call);
    if (dims->rows == 0) return GS_OK;
    size_t s, f, b;
    ffn_sizes(*dims, &s, &f, &b);
    GSR_CHECK(check_workspace(call, workspace, workspace_bytes, f));
    return launched(launch_ffn_forward(*dims, x, ld_x, *weights, y, ld_y, saved, workspace, stream), call);
}

gs_status gs_ffn_backward(const gs_ffn_dims* dims, const void* x, int64_t ld_x, const gs_ffn_weights* weights,
                          const void* saved, const void* dy, int64_t ld_dy, const gs_ffn_grads* grads,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const char* call = "gs_ffn_backward";
    GSR_CHECK(check_ffn(call, dims));
    if (!grads) return fail(GS_ERR_INVALID_ARGUMENT, "%s: grads is null", call);
    const size_t e = elem(dims->dtype);
    GSR_CHECK(check_ffn_weights(call, dims, weights));
    GSR_CHECK(check_array(call, "x", x, dims->rows, dims->d_in, ld_x, e));
    GSR_CHECK(check_array(call, "dy", dy, dims->rows, dims->d_out, ld_dy, e));
    GSR_CHECK(check_array(call, "saved", saved, dims->rows, 0, 0, 256));
    if (grads->x) GSR_CHECK(check_array(call, "grads.x", grads->x, dims->rows, dims->d_in, grads->ld_x, e));
    if (!aligned(grads->gate, e) || !aligned(grads->up, e) || !aligned(grads->down, e))
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: a gradient is not %zu-byte aligned", call, e);
    size_t s, f, b;
    ffn_sizes(*dims, &s, &f, &b);
    GSR_CHECK(check_workspace(call, workspace, workspace_bytes, b));
    return launched(launch_ffn_backward(*dims, x, ld_x, *weights, saved, dy, ld_dy, *grads, grads->ld_x, workspace,
                                        stream), call);
}

gs_status gs_scan_sizes(const gs_scan_dims* dims, size_t* saved_bytes, size_t* workspace_bytes) {
    GSR_CHECK(check_scan("gs_scan_sizes", dims));
    size_t s, w;
    scan_sizes(*dims, &s, &w);
    if (saved_bytes) *saved_bytes = s;
    if (workspace_bytes) *workspace_bytes = w;
    return GS_OK;
}

gs_status gs_scan_forward(const gs_scan_dims* dims, const int64_t* offsets, const gs_scan_inputs* in, void* y,
                          int64_t ld_y, float* h_last, void* saved, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
    const char* call = "gs_scan_forward";
    GSR_CHECK(check_scan(call, dims));
    GSR_CHECK(check_scan_inputs(call, dims, offsets, in));
    GSR_CHECK(check_array(call, "y", y, dims->rows, dims->channels, ld_y, elem(dims->dtype)));
    if (!aligned(h_last, 4) || !aligned(saved, 256))
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: h_last or saved is misaligned", call);
    GSR_CHECK(check_in_place(call, dims, "h0", in->h0, "h_last", h_last));
    size_t s, w;
    scan_sizes(*dims, &s, &w);
    GSR_CHECK(check_workspace(call, workspace, workspace_bytes, w));
    return launched(launch_scan_forward(*dims, offsets, *in, y, ld_y, h_last, (float*)saved, workspace, stream), call);
}

gs_status gs_scan_backward(const gs_scan_dims* dims, const int64_t* offsets, const gs_scan_inputs* in,
                           const void* saved, const void* dy, int64_t ld_dy, const float* dh_last,
                           const gs_scan_grads* grads, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const char* call = "gs_scan_backward";
    GSR_CHECK(check_scan(call, dims));
    GSR_CHECK(check_scan_inputs(call, dims, offsets, in));
    if (!grads) return fail(GS_ERR_INVALID_ARGUMENT, "%s: grads is null", call);
    const size_t e = elem(dims->dtype);
    GSR_CHECK(check_array(call, "dy", dy, dims->rows, dims->channels, ld_dy, e));
    GSR_CHECK(check_array(call, "saved", saved, dims->rows, 0, 0, 256));
    if (grads->gate) GSR_CHECK(check_array(call, "grads.gate", grads->gate, dims->rows, dims->channels, grads->ld_gate, e));
    if (grads->x) GSR_CHECK(check_array(call, "grads.x", grads->x, dims->rows, dims->channels, grads->ld_x, e));
    if (!aligned(dh_last, 4) || !aligned(grads->h0, 4))
        return fail(GS_ERR_INVALID_ARGUMENT, "%s: dh_last or grads.h0 is not 4-byte aligned", call);
    GSR_CHECK(check_in_place(call, dims, "dh_last", dh_last, "grads.h0", grads->h0));
    GSR_CHECK(check_in_place(call, dims, "h0", in->h0, "grads.h0", grads->h0));
    size_t s, w;
    scan_sizes(*dims, &s, &w);
    GSR_CHECK(check_workspace(call, workspace, workspace_bytes, w));
    return launched(launch_scan_backward(*dims, offsets, *in, (const float*)saved, dy, ld_dy, dh_last, *grads,
                                         workspace, stream), call);
}

gs_status gs_default_ortho_dims(gs_ortho_dims* out) {
    if (!out) return fail(GS_ERR_INVALID_ARGUMENT, "gs_default_ortho_dims: null argument");
    *out = gs_ortho_dims{};
    out->steps = 5;
    out->a = 3.4445f;
    out->b = -4.7750f;
    out->c = 2.0315f;
    out->eps = 1e-7f;
    return GS_OK;
}

gs_status gs_ortho_size(const gs_ortho_dims* dims, size_t* workspace_bytes) {
    GSR_CHECK(check_ortho("gs_ortho_size", dims));
    if (!workspace_bytes) return fail(GS_ERR_INVALID_ARGUMENT, "gs_ortho_size: null argument");
    *workspace_bytes = ortho_workspace(*dims);
    return GS_OK;
}

gs_status gs_orthogonalize(const gs_ortho_dims* dims, const void* g, void* out, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    const char* call = "gs_orthogonalize";
    GSR_CHECK(check_ortho(call, dims));
    if (dims->batch == 0) return GS_OK;
    GSR_CHECK(check_array(call, "g", g, 1, 0, 0, elem(dims->dtype)));
    GSR_CHECK(check_array(call, "out", out, 1, 0, 0, elem(dims->out_dtype)));
    GSR_CHECK(check_workspace(call, workspace, workspace_bytes, ortho_workspace(*dims)));
    return launched(launch_ortho(*dims, g, out, workspace, stream), call);
}

}  // extern "C"
