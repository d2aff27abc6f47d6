// cgtp_train_api.cpp -- the C ABI of the node-side operators (see
// include/cgtp_train.h): argument checks and dispatch.  No exception, no
// allocation; every check comes before the first launch.
#include "cgtp_train.h"

#include <stdint.h>

#include <cmath>

#include "cgtp_train_internal.h"

namespace {

constexpr int64_t kMaxRows = INT32_MAX;       // rows, table rows and segments are below this
constexpr int64_t kMaxEmbedChannels = 1 << 20;
constexpr int64_t kMaxNormChannels = 1 << 16;
constexpr int64_t kMaxElems = int64_t(1) << 45;  // elements of one array: byte offsets stay far inside 64 bits

cgtp_status_t hip_status(hipError_t e) { return e == hipSuccess ? CGTP_OK : CGTP_ERR_HIP; }

bool type_ok(int t) { return t == CGTP_F32 || t == CGTP_BF16; }

// a workspace of at least `need` bytes, none for none
cgtp_status_t check_workspace(const void* ws, size_t ws_bytes, size_t need)
{
    if (need == 0) return CGTP_OK;
    if (!ws || ws_bytes < need) return CGTP_ERR_WORKSPACE;
    return ((uintptr_t)ws & 255u) != 0 ? CGTP_ERR_INVALID_ARG : CGTP_OK;
}

// a missing or misaligned array
bool bad(const void* p, int64_t align) { return !p || ((uintptr_t)p % (uintptr_t)align) != 0; }

bool too_long(int64_t rows, int64_t ld) { return rows > 0 && ld > kMaxElems / rows; }

cgtp_status_t check_embed(cgtp_dtype_t dtype, int64_t n_rows, int64_t table_rows, int64_t channels)
{
    if (!type_ok(dtype) || n_rows < 0 || table_rows < 1 || channels < 1) return CGTP_ERR_INVALID_ARG;
    if (n_rows >= kMaxRows || table_rows >= kMaxRows) return CGTP_ERR_INVALID_ARG;
    if (channels > kMaxEmbedChannels) return CGTP_ERR_UNSUPPORTED;
    if (too_long(table_rows, channels) || too_long(n_rows, channels)) return CGTP_ERR_INVALID_ARG;
    return CGTP_OK;
}

cgtp_status_t check_norm(cgtp_dtype_t dtype, int64_t n_rows, int64_t n_segments, int64_t channels, int64_t groups)
{
    if (!type_ok(dtype) || n_rows < 0 || n_segments < 0 || channels < 1 || groups < 1) return CGTP_ERR_INVALID_ARG;
    if (n_rows >= kMaxRows || n_segments >= kMaxRows || channels % groups != 0) return CGTP_ERR_INVALID_ARG;
    if (n_segments == 0 && n_rows > 0) return CGTP_ERR_INVALID_ARG;
    if (channels > kMaxNormChannels) return CGTP_ERR_UNSUPPORTED;
    return CGTP_OK;
}

cgtp::NormShape norm_shape(cgtp_dtype_t dtype, int act, int64_t N, int64_t B, int64_t C, int64_t G)
{
    cgtp::NormShape n{};
    n.dtype = dtype;
    n.act = act;
    n.N = N;
    n.B = B;
    n.C = (int32_t)C;
    n.G = (int32_t)G;
    return n;
}

// shared by both directions: sizes, offsets, activation, workspace
cgtp_status_t check_norm_call(const cgtp::NormShape& n, cgtp_act_t act, const int32_t* seg_ptr, const void* ws,
                              size_t ws_bytes, bool backward)
{
    if (act != CGTP_ACT_NONE && act != CGTP_ACT_SILU && act != CGTP_ACT_TANH) return CGTP_ERR_INVALID_ARG;
    if (seg_ptr ? bad(seg_ptr, 4) : n.B > 0 && n.N % n.B != 0) return CGTP_ERR_INVALID_ARG;
    return check_workspace(ws, ws_bytes, cgtp::norm_workspace_bytes(n, seg_ptr != nullptr, backward));
}

bool bad_rows(const void* p, int64_t rows, int64_t ld, int64_t width, int64_t align)
{
    return bad(p, align) || ld < width || too_long(rows, ld);
}

constexpr int64_t kMaxSide = 1 << 16, kMaxMatrixElems = int64_t(1) << 31, kMaxStack = int64_t(1) << 33;

cgtp_status_t check_ortho(cgtp_dtype_t dtype, int64_t batch, int64_t rows, int64_t cols)
{
    if (!type_ok(dtype) || batch < 0 || rows < 1 || cols < 1) return CGTP_ERR_INVALID_ARG;
    if (rows > kMaxSide || cols > kMaxSide || rows * cols > kMaxMatrixElems) return CGTP_ERR_UNSUPPORTED;
    // padded sides are at least 64: the launches stay below 2^32 threads
    const int64_t padded = (rows + 127) / 128 * 128 * ((cols + 127) / 128 * 128);
    if (batch > kMaxStack / padded) return CGTP_ERR_UNSUPPORTED;
    return CGTP_OK;
}

// the generator's arguments; thr = 65536 p, rounded
cgtp_status_t check_drop(double p, uint64_t seed, uint64_t offset, const int64_t* step, cgtp::Drop* d)
{
    if (!(p >= 0.0 && p < 1.0) || (step && bad(step, 8))) return CGTP_ERR_INVALID_ARG;
    const double t = std::floor(65536.0 * p + 0.5);
    d->thr = t < 65535.0 ? (uint32_t)t : 65535u;
    d->scale = (float)(1.0 / (1.0 - d->thr / 65536.0));
    d->seed = seed;
    d->offset = offset;
    d->step = d->thr ? step : nullptr;
    return CGTP_OK;
}

constexpr int64_t kMaxLinearRows = int64_t(1) << 30, kMaxLinearWidth = 1 << 16;

cgtp_status_t check_linear(cgtp_dtype_t dtype, int64_t n_rows, int64_t in, int64_t out, cgtp::LinShape* n)
{
    if (!type_ok(dtype) || n_rows < 0 || in < 1 || out < 1) return CGTP_ERR_INVALID_ARG;
    if (n_rows >= kMaxLinearRows || in > kMaxLinearWidth || out > kMaxLinearWidth) return CGTP_ERR_UNSUPPORTED;
    *n = cgtp::LinShape{};
    n->dtype = dtype;
    n->N = n_rows;
    n->K = in;
    n->M = out;
    return cgtp::linear_fits(*n) ? CGTP_OK : CGTP_ERR_UNSUPPORTED;
}

bool act_ok(int act) { return act == CGTP_ACT_NONE || act == CGTP_ACT_SILU || act == CGTP_ACT_TANH; }

cgtp::OrthoShape ortho_shape(cgtp_dtype_t dtype, int64_t batch, int64_t rows, int64_t cols)
{
    cgtp::OrthoShape o{};
    o.dtype = dtype;
    o.batch = batch;
    o.m = rows;
    o.n = cols;
    return o;
}

}  // namespace

extern "C" {

// ---- embedding -------------------------------------------------------------------
cgtp_status_t cgtp_embed_fwd(cgtp_dtype_t dtype, int64_t n_rows, int64_t table_rows, int64_t channels,
                             const int32_t* ids, const void* table, float scale, void* out, int64_t ld_out,
                             hipStream_t stream)
{
    const cgtp_status_t st = check_embed(dtype, n_rows, table_rows, channels);
    if (st != CGTP_OK) return st;
    if (n_rows == 0) return CGTP_OK;
    const int64_t es = cgtp::dtype_size(dtype);
    if (bad(ids, 4) || bad(table, es) || bad_rows(out, n_rows, ld_out, channels, es)) return CGTP_ERR_INVALID_ARG;
    const cgtp::EmbedShape e{dtype, n_rows, table_rows, channels, ld_out, scale};
    return hip_status(cgtp::launch_embed_fwd(e, ids, table, out, stream));
}

cgtp_status_t cgtp_embed_bwd_workspace_size(cgtp_dtype_t dtype, int64_t n_rows, int64_t table_rows,
                                            int64_t channels, size_t* bytes)
{
    if (!bytes) return CGTP_ERR_INVALID_ARG;
    const cgtp_status_t st = check_embed(dtype, n_rows, table_rows, channels);
    if (st != CGTP_OK) return st;
    *bytes = cgtp::embed_bwd_workspace_bytes(cgtp::EmbedShape{dtype, n_rows, table_rows, channels, channels, 1.0f});
    return CGTP_OK;
}

cgtp_status_t cgtp_embed_bwd(cgtp_dtype_t dtype, int64_t n_rows, int64_t table_rows, int64_t channels,
                             const int32_t* ids, const void* grad_out, int64_t ld_grad, float scale,
                             void* grad_table, void* ws, size_t ws_bytes, hipStream_t stream)
{
    const cgtp_status_t st = check_embed(dtype, n_rows, table_rows, channels);
    if (st != CGTP_OK) return st;
    const int64_t es = cgtp::dtype_size(dtype);
    if (bad(grad_table, es)) return CGTP_ERR_INVALID_ARG;
    const cgtp::EmbedShape e{dtype, n_rows, table_rows, channels, ld_grad, scale};
    if (n_rows > 0) {
        if (bad(ids, 4) || bad_rows(grad_out, n_rows, ld_grad, channels, es)) return CGTP_ERR_INVALID_ARG;
        const cgtp_status_t sw = check_workspace(ws, ws_bytes, cgtp::embed_bwd_workspace_bytes(e));
        if (sw != CGTP_OK) return sw;
    }
    return hip_status(cgtp::launch_embed_bwd(e, ids, grad_out, grad_table, ws, stream));
}

// ---- group normalisation with an activation ------------------------------------------
cgtp_status_t cgtp_norm_act_workspace_size(cgtp_dtype_t dtype, int64_t n_rows, int64_t n_segments,
                                           int64_t channels, int64_t groups, int ragged, int backward, size_t* bytes)
{
    if (!bytes) return CGTP_ERR_INVALID_ARG;
    const cgtp_status_t st = check_norm(dtype, n_rows, n_segments, channels, groups);
    if (st != CGTP_OK) return st;
    *bytes = cgtp::norm_workspace_bytes(norm_shape(dtype, 0, n_rows, n_segments, channels, groups), ragged != 0,
                                        backward != 0);
    return CGTP_OK;
}

cgtp_status_t cgtp_norm_act_fwd(cgtp_dtype_t dtype, cgtp_act_t act, int64_t n_rows, int64_t n_segments,
                                int64_t channels, int64_t groups, const int32_t* seg_ptr, float eps, const void* x,
                                int64_t ld_x, const float* gamma, const float* beta, void* y, int64_t ld_y,
                                float* mean, float* rstd, void* ws, size_t ws_bytes, hipStream_t stream)
{
    cgtp_status_t st = check_norm(dtype, n_rows, n_segments, channels, groups);
    if (st != CGTP_OK) return st;
    if (n_segments == 0) return CGTP_OK;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return CGTP_ERR_INVALID_ARG;
    cgtp::NormShape n = norm_shape(dtype, act, n_rows, n_segments, channels, groups);
    st = check_norm_call(n, act, seg_ptr, ws, ws_bytes, false);
    if (st != CGTP_OK) return st;
    const int64_t es = cgtp::dtype_size(dtype);
    if (bad(mean, 4) || bad(rstd, 4) || (gamma && bad(gamma, 4)) || (beta && bad(beta, 4)))
        return CGTP_ERR_INVALID_ARG;
    if (n_rows > 0 && (bad_rows(x, n_rows, ld_x, channels, es) || bad_rows(y, n_rows, ld_y, channels, es)))
        return CGTP_ERR_INVALID_ARG;
    n.seg = seg_ptr;
    n.eps = eps;
    n.ldx = ld_x;
    n.ldy = ld_y;
    return hip_status(cgtp::launch_norm_fwd(n, x, gamma, beta, y, mean, rstd, ws, stream));
}

cgtp_status_t cgtp_norm_act_bwd(cgtp_dtype_t dtype, cgtp_act_t act, int64_t n_rows, int64_t n_segments,
                                int64_t channels, int64_t groups, const int32_t* seg_ptr, const void* x,
                                int64_t ld_x, const float* mean, const float* rstd, const float* gamma,
                                const float* beta, const void* grad_y, int64_t ld_dy, void* grad_x, int64_t ld_dx,
                                float* grad_gamma, float* grad_beta, void* ws, size_t ws_bytes,
                                hipStream_t stream)
{
    cgtp_status_t st = check_norm(dtype, n_rows, n_segments, channels, groups);
    if (st != CGTP_OK) return st;
    if (!grad_x && !grad_gamma && !grad_beta) return CGTP_OK;
    cgtp::NormShape n = norm_shape(dtype, act, n_rows, n_segments, channels, groups);
    st = check_norm_call(n, act, seg_ptr, ws, ws_bytes, true);
    if (st != CGTP_OK) return st;
    const int64_t es = cgtp::dtype_size(dtype);
    for (const float* p : {gamma, beta, (const float*)grad_gamma, (const float*)grad_beta})
        if (p && bad(p, 4)) return CGTP_ERR_INVALID_ARG;
    if (n_rows > 0) {
        if (bad(mean, 4) || bad(rstd, 4)) return CGTP_ERR_INVALID_ARG;
        if (bad_rows(x, n_rows, ld_x, channels, es) || bad_rows(grad_y, n_rows, ld_dy, channels, es))
            return CGTP_ERR_INVALID_ARG;
        if (grad_x && bad_rows(grad_x, n_rows, ld_dx, channels, es)) return CGTP_ERR_INVALID_ARG;
    }
    n.seg = seg_ptr;
    n.ldx = ld_x;
    n.ldy = ld_dy;
    n.ldd = ld_dx;
    return hip_status(cgtp::launch_norm_bwd(n, x, mean, rstd, gamma, beta, grad_y, grad_x, grad_gamma, grad_beta, ws,
                                            stream));
}

// ---- dropout ---------------------------------------------------------------------------
cgtp_status_t cgtp_dropout(cgtp_dtype_t dtype, int64_t n_rows, int64_t channels, double p, uint64_t seed,
                           uint64_t offset, const int64_t* step, const void* x, int64_t ld_x, const void* residual,
                           int64_t ld_r, void* out, int64_t ld_out, hipStream_t stream)
{
    if (!type_ok(dtype) || n_rows < 0 || channels < 1 || n_rows >= kMaxRows) return CGTP_ERR_INVALID_ARG;
    if (channels > kMaxEmbedChannels) return CGTP_ERR_UNSUPPORTED;
    cgtp::DropShape d{};
    const cgtp_status_t st = check_drop(p, seed, offset, step, &d.drop);
    if (st != CGTP_OK) return st;
    if (n_rows == 0) return CGTP_OK;
    const int64_t es = cgtp::dtype_size(dtype);
    if (bad_rows(x, n_rows, ld_x, channels, es) || bad_rows(out, n_rows, ld_out, channels, es))
        return CGTP_ERR_INVALID_ARG;
    if (residual && bad_rows(residual, n_rows, ld_r, channels, es)) return CGTP_ERR_INVALID_ARG;
    d.dtype = dtype;
    d.N = n_rows;
    d.C = channels;
    d.ldx = ld_x;
    d.ldr = ld_r;
    d.ldo = ld_out;
    return hip_status(cgtp::launch_dropout(d, x, residual, out, stream));
}

// ---- product with bias, activation, dropout and residual -------------------------------
cgtp_status_t cgtp_linear_act_workspace_size(cgtp_dtype_t dtype, int64_t n_rows, int64_t in_channels,
                                             int64_t out_channels, int backward, size_t* bytes)
{
    if (!bytes) return CGTP_ERR_INVALID_ARG;
    cgtp::LinShape n;
    const cgtp_status_t st = check_linear(dtype, n_rows, in_channels, out_channels, &n);
    if (st != CGTP_OK) return st;
    *bytes = cgtp::linear_workspace_bytes(n, backward != 0);
    return CGTP_OK;
}

cgtp_status_t cgtp_linear_act_fwd(cgtp_dtype_t dtype, cgtp_act_t act, int64_t n_rows, int64_t in_channels,
                                  int64_t out_channels, const void* x, int64_t ld_x, const void* W, const float* bias,
                                  const void* residual, int64_t ld_r, double p, uint64_t seed, uint64_t offset,
                                  const int64_t* step, void* z, void* y, int64_t ld_y, void* ws, size_t ws_bytes,
                                  hipStream_t stream)
{
    cgtp::LinShape n;
    cgtp_status_t st = check_linear(dtype, n_rows, in_channels, out_channels, &n);
    if (st != CGTP_OK) return st;
    if (!act_ok(act)) return CGTP_ERR_INVALID_ARG;
    st = check_drop(p, seed, offset, step, &n.drop);
    if (st != CGTP_OK) return st;
    if (n_rows == 0) return CGTP_OK;
    const int64_t es = cgtp::dtype_size(dtype);
    if (bad_rows(x, n_rows, ld_x, in_channels, es) || bad(W, es) || bad_rows(y, n_rows, ld_y, out_channels, es))
        return CGTP_ERR_INVALID_ARG;
    if ((bias && bad(bias, 4)) || (z && bad(z, es))) return CGTP_ERR_INVALID_ARG;
    if (residual && bad_rows(residual, n_rows, ld_r, out_channels, es)) return CGTP_ERR_INVALID_ARG;
    st = check_workspace(ws, ws_bytes, cgtp::linear_workspace_bytes(n, false));
    if (st != CGTP_OK) return st;
    n.act = act;
    n.ldx = ld_x;
    n.ldr = ld_r;
    n.ldy = ld_y;
    return hip_status(cgtp::launch_linear_fwd(n, x, W, bias, residual, z, y, ws, stream));
}

cgtp_status_t cgtp_linear_act_bwd(cgtp_dtype_t dtype, cgtp_act_t act, int64_t n_rows, int64_t in_channels,
                                  int64_t out_channels, const void* x, int64_t ld_x, const void* W, const void* z,
                                  const void* grad_y, int64_t ld_dy, double p, uint64_t seed, uint64_t offset,
                                  const int64_t* step, void* grad_x, int64_t ld_dx, void* grad_W, float* grad_bias,
                                  void* ws, size_t ws_bytes, hipStream_t stream)
{
    cgtp::LinShape n;
    cgtp_status_t st = check_linear(dtype, n_rows, in_channels, out_channels, &n);
    if (st != CGTP_OK) return st;
    if (!act_ok(act)) return CGTP_ERR_INVALID_ARG;
    st = check_drop(p, seed, offset, step, &n.drop);
    if (st != CGTP_OK) return st;
    if (!grad_x && !grad_W && !grad_bias) return CGTP_OK;
    const int64_t es = cgtp::dtype_size(dtype);
    if ((grad_W && bad(grad_W, es)) || (grad_bias && bad(grad_bias, 4))) return CGTP_ERR_INVALID_ARG;
    if (n_rows > 0) {
        if (bad_rows(grad_y, n_rows, ld_dy, out_channels, es)) return CGTP_ERR_INVALID_ARG;
        if (act != CGTP_ACT_NONE && bad(z, es)) return CGTP_ERR_INVALID_ARG;
        if (grad_x && (bad(W, es) || bad_rows(grad_x, n_rows, ld_dx, in_channels, es))) return CGTP_ERR_INVALID_ARG;
        if (grad_W && bad_rows(x, n_rows, ld_x, in_channels, es)) return CGTP_ERR_INVALID_ARG;
        st = check_workspace(ws, ws_bytes, cgtp::linear_workspace_bytes(n, true));
        if (st != CGTP_OK) return st;
    }
    n.act = act;
    n.ldx = ld_x;
    n.ldg = ld_dy;
    n.ldd = ld_dx;
    return hip_status(cgtp::launch_linear_bwd(n, x, W, z, grad_y, grad_x, grad_W, grad_bias, ws, stream));
}

// ---- orthogonalised update -------------------------------------------------------------
cgtp_status_t cgtp_orthogonalize_workspace_size(cgtp_dtype_t dtype, int64_t batch, int64_t rows, int64_t cols,
                                                size_t* bytes)
{
    if (!bytes) return CGTP_ERR_INVALID_ARG;
    const cgtp_status_t st = check_ortho(dtype, batch, rows, cols);
    if (st != CGTP_OK) return st;
    *bytes = cgtp::ortho_workspace_bytes(ortho_shape(dtype, batch, rows, cols));
    return CGTP_OK;
}

cgtp_status_t cgtp_orthogonalize(cgtp_dtype_t dtype, int64_t batch, int64_t rows, int64_t cols, int steps, double a,
                                 double b, double c, float eps, float scale, const void* G, void* out, void* ws,
                                 size_t ws_bytes, hipStream_t stream)
{
    const cgtp_status_t st = check_ortho(dtype, batch, rows, cols);
    if (st != CGTP_OK) return st;
    if (steps < 1 || steps > cgtp::kMaxOrthoSteps || !(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(scale))
        return CGTP_ERR_INVALID_ARG;
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !cgtp::ortho_bounded(a, b, c, steps))
        return CGTP_ERR_INVALID_ARG;
    if (batch == 0) return CGTP_OK;
    const int64_t es = cgtp::dtype_size(dtype);
    if (bad(G, es) || bad(out, es)) return CGTP_ERR_INVALID_ARG;
    cgtp::OrthoShape o = ortho_shape(dtype, batch, rows, cols);
    const cgtp_status_t sw = check_workspace(ws, ws_bytes, cgtp::ortho_workspace_bytes(o));
    if (sw != CGTP_OK) return sw;
    o.steps = steps;
    o.a = a;
    o.b = b;
    o.c = c;
    o.eps = eps;
    o.scale = scale;
    return hip_status(cgtp::launch_orthogonalize(o, G, out, ws, stream));
}

}  // extern "C"
