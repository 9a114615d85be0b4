// extern "C" entry points of the token-block operators: argument checks and
// workspace sizes. Every refusal comes before anything is launched.
#include "common.cuh"
#include "kernels.cuh"

using namespace dlrm;

namespace {

constexpr int64_t INT31 = (int64_t)1 << 31;
constexpr int MAX_D = 65536;          // lookups
constexpr int MAX_NORM_D = 32768;     // norm: 1,024 threads of 32 elements

cudaStream_t cs(dlrm_stream s) { return reinterpret_cast<cudaStream_t>(s); }
bool float_dt(int dt) { return dt == DLRM_F32 || dt == DLRM_F16 || dt == DLRM_BF16; }
size_t elem(int dt) { return dt == DLRM_F32 ? 4 : dt == DLRM_E4M3 ? 1 : 2; }
bool on(const void* p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
bool ws_ok(const void* ws, size_t have, size_t need) { return ws && on(ws, 16) && have >= need; }

// A matrix whose rows need no alignment beyond the element's.
bool loose(const void* p, int64_t ld, int64_t width, int dt) { return p && on(p, elem(dt)) && ld >= width; }
// A matrix whose rows start on 16-byte boundaries.
bool tight(const void* p, int64_t ld, int64_t width, int dt) {
    return p && on(p, 16) && ld >= width && ld < INT31 && (ld * (int64_t)elem(dt)) % 16 == 0;
}

// One expert's weights span less than a tensor map's largest stride.
bool spans(int N, int64_t ld, int dt) { return (int64_t)N * ld * (int64_t)elem(dt) < (int64_t)1 << 40; }

dlrm_status experts_sizes(int E, int M, int N, int K) {
    if (E < 1 || M < 0 || N < 1 || K < 1) return DLRM_ERR_INVALID_ARG;
    if (E > DLRM_MAX_EXPERTS) return DLRM_ERR_UNSUPPORTED;
    // a tile's rows past its expert's last are numbered too
    if (M > INT31 - 256) return DLRM_ERR_UNSUPPORTED;
    // tiles of one expert are counted in 31 bits
    const int64_t wide = N > K ? N : K;
    if (((int64_t)M / 128 + 1) * (wide / 64 + 1) >= INT31) return DLRM_ERR_UNSUPPORTED;
    if ((wide / 256 + 1) * (wide / 256 + 1) >= INT31) return DLRM_ERR_UNSUPPORTED;
    return DLRM_OK;
}

}  // namespace

extern "C" {

dlrm_status dlrm_embed_fwd(const dlrm_tables* T, int k, int64_t n, const int32_t* indices, float scale, void* out,
                           int64_t ld_out, dlrm_dtype out_dt, void* ws, size_t ws_bytes, dlrm_stream stream) {
    if (!T || !T->rows || !T->data || T->K < 1 || T->d < 1 || k < 0 || k >= T->K) return DLRM_ERR_INVALID_ARG;
    if (T->dt == DLRM_U8ROW) return DLRM_ERR_UNSUPPORTED;
    if (!float_dt(T->dt) || !float_dt(out_dt) || !on(T->data, 16) || n < 0 || n >= INT31) return DLRM_ERR_INVALID_ARG;
    if (T->K > DLRM_MAX_TABLES || T->d > MAX_D) return DLRM_ERR_UNSUPPORTED;
    int64_t base = 0;
    for (int i = 0; i <= k; ++i) {
        if (T->rows[i] < 1) return DLRM_ERR_INVALID_ARG;
        if (i < k) base += T->rows[i];
    }
    if (T->rows[k] >= INT31) return DLRM_ERR_UNSUPPORTED;
    if (!ws_ok(ws, ws_bytes, DLRM_ERR_RECORD_BYTES)) return DLRM_ERR_WORKSPACE;
    if (n == 0) return DLRM_OK;
    if (!indices || !on(indices, 4) || !loose(out, ld_out, T->d, out_dt)) return DLRM_ERR_INVALID_ARG;
    const char* table = static_cast<const char*>(T->data) + (size_t)base * T->d * elem(T->dt);
    return launch_lookup(table, T->dt, T->rows[k], T->d, n, indices, scale, out, ld_out, out_dt,
                         static_cast<ErrRecord*>(ws), cs(stream));
}

dlrm_status dlrm_set_sort_clusters(int allowed) {
    set_sort_clusters(allowed != 0);
    return DLRM_OK;
}

size_t dlrm_embed_bwd_workspace_size(int64_t rows, int d, int64_t n) {
    if (rows < 1 || rows >= INT31 || d < 1 || d > MAX_D || n < 0 || n >= INT31 || !lookup_grad_fits(d, n)) return 0;
    return lookup_grad_workspace(rows, d, n);
}

dlrm_status dlrm_embed_bwd(int64_t rows, int d, int64_t n, const int32_t* indices, float scale, const void* dout,
                           int64_t ld_dout, dlrm_dtype dout_dt, void* dtable, dlrm_dtype dtable_dt, void* ws,
                           size_t ws_bytes, dlrm_stream stream) {
    if (rows < 1 || d < 1 || n < 0 || n >= INT31 || !float_dt(dout_dt) || !float_dt(dtable_dt))
        return DLRM_ERR_INVALID_ARG;
    if (rows >= INT31 || d > MAX_D || !lookup_grad_fits(d, n)) return DLRM_ERR_UNSUPPORTED;
    if (!loose(dtable, d, d, dtable_dt)) return DLRM_ERR_INVALID_ARG;
    if (n > 0 && (!indices || !on(indices, 4) || !loose(dout, ld_dout, d, dout_dt))) return DLRM_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, lookup_grad_workspace(rows, d, n))) return DLRM_ERR_WORKSPACE;
    return launch_lookup_grad(rows, d, n, indices, scale, dout, ld_dout, dout_dt, dtable, dtable_dt,
                              static_cast<char*>(ws), cs(stream));
}

dlrm_status dlrm_dropout(int64_t n, const void* x, const void* residual, dlrm_dtype dt, double p, const int64_t* rng,
                         void* y, dlrm_stream stream) {
    if (n < 0 || !float_dt(dt) || !(p >= 0.0 && p <= 1.0)) return DLRM_ERR_INVALID_ARG;
    if (n == 0) return DLRM_OK;
    if (!rng || !on(rng, 8) || !loose(x, 1, 1, dt) || !loose(y, 1, 1, dt) || !on(residual, elem(dt)))
        return DLRM_ERR_INVALID_ARG;
    return launch_dropout(n, x, residual, dt, p, rng, y, cs(stream));
}

dlrm_status dlrm_rmsnorm_fwd(int rows, int d, const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                             dlrm_dtype dt, const float* w, float eps, void* h, int64_t ld_h, void* y, int64_t ld_y,
                             dlrm_dtype y_dt, float* y_scale, float* rstd, dlrm_stream stream) {
    if (rows < 0 || d < 1 || !float_dt(dt) || (y_dt != dt && y_dt != DLRM_E4M3) || !(eps >= 0.f))
        return DLRM_ERR_INVALID_ARG;
    if ((y_dt == DLRM_E4M3) != (y_scale != nullptr)) return DLRM_ERR_INVALID_ARG;
    if (d > MAX_NORM_D) return DLRM_ERR_UNSUPPORTED;
    if (rows == 0) return DLRM_OK;
    if (!loose(x, ld_x, d, dt) || (residual && !loose(residual, ld_res, d, dt)) || (h && !loose(h, ld_h, d, dt)) ||
        !loose(y, ld_y, d, y_dt) || !on(w, 4) || !on(y_scale, 4) || !on(rstd, 4))
        return DLRM_ERR_INVALID_ARG;
    return launch_rmsnorm_fwd(rows, d, x, ld_x, residual, ld_res, w, eps, dt, h, ld_h, y, ld_y, y_scale, rstd,
                              cs(stream));
}

size_t dlrm_rmsnorm_bwd_workspace_size(int rows, int d) {
    if (rows < 0 || d < 1 || d > MAX_NORM_D) return 0;
    return DLRM_ERR_RECORD_BYTES + sizeof(float) * rmsnorm_bwd_partial_floats(rows, d);
}

dlrm_status dlrm_rmsnorm_bwd(int rows, int d, const void* dy, int64_t ld_dy, const void* h, int64_t ld_h,
                             const float* rstd, const float* w, const void* dh, int64_t ld_dh, dlrm_dtype dt, void* dx,
                             int64_t ld_dx, float* dw, void* ws, size_t ws_bytes, dlrm_stream stream) {
    if (rows < 0 || d < 1 || !float_dt(dt) || !on(dw, 4)) return DLRM_ERR_INVALID_ARG;
    if (d > MAX_NORM_D) return DLRM_ERR_UNSUPPORTED;
    if (rows > 0 && (!loose(dy, ld_dy, d, dt) || !loose(h, ld_h, d, dt) || (dh && !loose(dh, ld_dh, d, dt)) ||
                     !loose(dx, ld_dx, d, dt) || !rstd || !on(rstd, 4) || !on(w, 4)))
        return DLRM_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, dlrm_rmsnorm_bwd_workspace_size(rows, d))) return DLRM_ERR_WORKSPACE;
    return launch_rmsnorm_bwd(rows, d, dy, ld_dy, h, ld_h, rstd, w, dh, ld_dh, dt, dx, ld_dx, dw,
                              reinterpret_cast<float*>(static_cast<char*>(ws) + DLRM_ERR_RECORD_BYTES), cs(stream));
}

dlrm_status dlrm_experts_fwd(int E, int M, int N, int K, const int32_t* offsets, const void* X, int64_t ldx,
                             const float* x_scale, dlrm_dtype dt, const void* W, int64_t ldw, const float* w_scale,
                             const float* bias, int act, void* Y, int64_t ldy, dlrm_dtype y_dt, void* ws,
                             size_t ws_bytes, dlrm_stream stream) {
    if (dt == DLRM_F32) return DLRM_ERR_UNSUPPORTED;
    if ((!float_dt(dt) && dt != DLRM_E4M3) || !float_dt(y_dt)) return DLRM_ERR_INVALID_ARG;
    if (dt != DLRM_E4M3 && y_dt != dt && y_dt != DLRM_F32) return DLRM_ERR_UNSUPPORTED;
    if (act != DLRM_ACT_NONE && act != DLRM_ACT_RELU) return DLRM_ERR_INVALID_ARG;
    const dlrm_status r = experts_sizes(E, M, N, K);
    if (r != DLRM_OK) return r;
    if (!ws_ok(ws, ws_bytes, DLRM_ERR_RECORD_BYTES)) return DLRM_ERR_WORKSPACE;
    if (M == 0) return DLRM_OK;
    if (!offsets || !on(offsets, 4) || !tight(X, ldx, K, dt) || !tight(W, ldw, K, dt) || !tight(Y, ldy, N, y_dt) ||
        !on(bias, 4))
        return DLRM_ERR_INVALID_ARG;
    if (!spans(N, ldw, dt)) return DLRM_ERR_UNSUPPORTED;
    const bool scaled = dt == DLRM_E4M3;
    if (scaled != (x_scale != nullptr) || scaled != (w_scale != nullptr) || !on(x_scale, 4) || !on(w_scale, 4))
        return DLRM_ERR_INVALID_ARG;
    if (!experts_supported()) return DLRM_ERR_UNSUPPORTED;
    return launch_experts_fwd(E, M, N, K, offsets, X, ldx, x_scale, dt, W, ldw, w_scale, bias, act == DLRM_ACT_RELU, Y,
                              ldy, y_dt, static_cast<ErrRecord*>(ws), cs(stream));
}

size_t dlrm_experts_bwd_workspace_size(int E, int M, int N, int K, int act) {
    if (experts_sizes(E, M, N, K) != DLRM_OK || (act != DLRM_ACT_NONE && act != DLRM_ACT_RELU)) return 0;
    return experts_layout(E, M, N, K, act == DLRM_ACT_RELU).total;
}

dlrm_status dlrm_experts_bwd(int E, int M, int N, int K, const int32_t* offsets, const void* dY, int64_t lddy,
                             const void* Y, int64_t ldy, int act, const void* X, int64_t ldx, const void* W,
                             int64_t ldw, dlrm_dtype dt, void* dX, int64_t lddx, dlrm_dtype dx_dt, void* dW,
                             int64_t lddw, dlrm_dtype dw_dt, float* db, void* ws, size_t ws_bytes, dlrm_stream stream) {
    if (dt == DLRM_F32 || dt == DLRM_E4M3) return DLRM_ERR_UNSUPPORTED;
    if (!float_dt(dt) || (act != DLRM_ACT_NONE && act != DLRM_ACT_RELU)) return DLRM_ERR_INVALID_ARG;
    if ((dX && !float_dt(dx_dt)) || (dW && !float_dt(dw_dt))) return DLRM_ERR_INVALID_ARG;
    if ((dX && dx_dt != dt && dx_dt != DLRM_F32) || (dW && dw_dt != dt && dw_dt != DLRM_F32)) return DLRM_ERR_UNSUPPORTED;
    const dlrm_status r = experts_sizes(E, M, N, K);
    if (r != DLRM_OK) return r;
    const bool relu = act == DLRM_ACT_RELU;
    if (!ws_ok(ws, ws_bytes, dlrm_experts_bwd_workspace_size(E, M, N, K, act))) return DLRM_ERR_WORKSPACE;
    if (!offsets || !on(offsets, 4) || !on(db, 4)) return DLRM_ERR_INVALID_ARG;
    if ((dX && !tight(dX, lddx, K, dx_dt)) || (dW && !tight(dW, lddw, K, dw_dt))) return DLRM_ERR_INVALID_ARG;
    if (M > 0 && (!tight(dY, lddy, N, dt) || (relu && !tight(Y, ldy, N, dt)) || (dW && !tight(X, ldx, K, dt)) ||
                  (dX && !tight(W, ldw, K, dt))))
        return DLRM_ERR_INVALID_ARG;
    if ((dX && M > 0 && !spans(N, ldw, dt)) || (dW && !spans(N, lddw, dw_dt))) return DLRM_ERR_UNSUPPORTED;
    if (!experts_supported()) return DLRM_ERR_UNSUPPORTED;
    return launch_experts_bwd(E, M, N, K, offsets, dY, lddy, relu ? Y : nullptr, ldy, X, ldx, W, ldw, dt, dX, lddx, dx_dt,
                              dW, lddw, dw_dt, db, static_cast<char*>(ws), cs(stream));
}

}  // extern "C"
