// cgtp_train_internal.h -- shapes, workspaces and launchers of the node-side operators
// (kernels in cgtp_embed.hip, cgtp_norm.hip, cgtp_ortho.hip, cgtp_dropout.hip and
// cgtp_linear.hip; entry points in cgtp_train_api.cpp).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace cgtp {

// element types of the large arrays (values of cgtp_dtype_t)
enum : int { kF32 = 0, kBF16 = 1 };
constexpr int64_t dtype_size(int t) { return t == kF32 ? 4 : 2; }

// ---- embedding -------------------------------------------------------------------
struct EmbedShape {
    int dtype;
    int64_t N, V;  // rows looked up, table rows (both below 2^31)
    int64_t C;
    int64_t ld;  // row stride of out / grad_out
    float scale;
};

size_t embed_bwd_workspace_bytes(const EmbedShape& e);

hipError_t launch_embed_fwd(const EmbedShape& e, const int32_t* ids, const void* table, void* out, hipStream_t s);
hipError_t launch_embed_bwd(const EmbedShape& e, const int32_t* ids, const void* grad, void* gtab, void* ws,
                            hipStream_t s);

// ---- group normalisation with an activation ------------------------------------------
struct NormShape {
    int dtype, act;
    int64_t N, B;  // rows, segments (both below 2^31)
    int32_t C, G;
    const int32_t* seg;  // offsets [B+1], or nullptr: equal segments of N / B rows
    int64_t ldx, ldy, ldd;  // row strides of x, of y or grad_y, of grad_x
    float eps;
};

// of one direction; ragged: with offsets
size_t norm_workspace_bytes(const NormShape& n, bool ragged, bool backward);

hipError_t launch_norm_fwd(const NormShape& n, const void* x, const float* gamma, const float* beta, void* y,
                           float* mean, float* rstd, void* ws, hipStream_t s);
hipError_t launch_norm_bwd(const NormShape& n, const void* x, const float* mean, const float* rstd,
                           const float* gamma, const float* beta, const void* dy, void* dx, float* dgamma,
                           float* dbeta, void* ws, hipStream_t s);

// ---- orthogonalised update -------------------------------------------------------------
struct OrthoShape {
    int dtype;
    int64_t batch, m, n;  // matrices [batch][m][n]
    int steps;
    double a, b, c;
    float eps, scale;
};

constexpr int kMaxOrthoSteps = 64;

struct OrthoPoly {
    int32_t steps;
    double a, b, c;
    float eps, scale;
};

// The orientation that is worked on: s <= t, sp and tp padded to whole tiles;
// tall: the stored matrices are [t][s].
struct OrthoDims {
    int64_t s, t, sp, tp;
    int32_t tall;
};

// whether the iterates of these coefficients stay within the fixed-point units
bool ortho_bounded(double a, double b, double c, int steps);

size_t ortho_workspace_bytes(const OrthoShape& o);

hipError_t launch_orthogonalize(const OrthoShape& o, const void* G, void* out, void* ws, hipStream_t s);

// ---- dropout ---------------------------------------------------------------------------
struct Drop {
    uint32_t thr;  // of 65536: fields below it are dropped; 0: none
    float scale;   // 1 / (1 - thr / 65536)
    uint64_t seed, offset;
    const int64_t* step;  // on the device, added to the offset; or nullptr
};

struct DropShape {
    int dtype;
    int64_t N;  // rows (below 2^31)
    int64_t C;
    int64_t ldx, ldr, ldo;
    Drop drop;
};

hipError_t launch_dropout(const DropShape& d, const void* x, const void* residual, void* out, hipStream_t s);

// ---- product with bias, activation, dropout and residual -------------------------------
struct LinShape {
    int dtype, act;
    int64_t N, K, M;  // rows (below 2^30), inputs, outputs
    int64_t ldx, ldr, ldy, ldg, ldd;  // row strides of x, residual, y, grad_y, grad_x
    Drop drop;
};

// whether the launches stay below 2^32 threads
bool linear_fits(const LinShape& n);
size_t linear_workspace_bytes(const LinShape& n, bool backward);

hipError_t launch_linear_fwd(const LinShape& n, const void* x, const void* W, const float* bias, const void* residual,
                             void* z, void* y, void* ws, hipStream_t s);
hipError_t launch_linear_bwd(const LinShape& n, const void* x, const void* W, const void* z, const void* grad_y,
                             void* grad_x, void* grad_W, float* grad_bias, void* ws, hipStream_t s);

}  // namespace cgtp
