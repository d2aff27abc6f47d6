// cgtp_norm.hip -- group normalisation with an activation over segments of
// channels-last rows, forward and backward.
//
//   mean, var over the M = rows x C/G values of a segment's group,
//   rstd = 1 / sqrt(var + eps), xhat = (x - mean) rstd, z = xhat gamma + beta,
//   y = act(z)
// and, with dz = dy act'(z), h = dz gamma,
//   dbeta = sum dz,  dgamma = sum dz xhat           over all rows
//   dx = rstd (h - sum h / M - xhat sum(h xhat) / M)   sums over the group
//
// Bound by memory: the forward has to read x and write y, the backward reads x
// and dy and writes dx.  A block takes a run of consecutive rows with the
// lanes along the channels, so every access is a contiguous row.  A run may
// hold the end of one segment and the beginning of others; each (run, segment)
// piece leaves its sums at the place run + segment of a list, which is unique
// because every new piece moves on by a run or a segment, and a second kernel
// adds the pieces of a segment in order.  Sums are fp64: var comes from the sum
// of squares, and the fp64 adds are hidden behind the loads.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "cgtp_internal.h"
#include "cgtp_train_internal.h"
#include "cgtp_vec.h"

namespace cgtp {
namespace {

constexpr int kThreads = 256;

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t kMaxBlocks = 1 << 22;  // the kernels stride over what is left
inline unsigned grid_of(int64_t n) { return (unsigned)(n < kMaxBlocks ? n : kMaxBlocks); }

// Channels are cut into slices of at most kThreads accesses; a slice holds
// whole groups, or one of the `parts` parts of a group wider than that.
struct Slices {
    int32_t n, parts;      // slices; parts per group
    int32_t width, groups; // channels and groups per slice (parts == 1), channels per part otherwise
};

struct NormArgs {
    int64_t N, B, R, runs, ldx, ldy, ldd;
    int32_t C, G, cpg;
    Slices sl;
    float eps;
    int act;
    const int32_t* seg;
    const float *gamma, *beta, *mean, *rstd;
    float *omean, *orstd;
    double* part;  // [runs + B][G][parts][2]
    double* chan;  // backward: [runs][2][C]
    double* coef;  // backward: [B][G][2], the group means of h and h xhat
};

struct Slice {
    int32_t c0, c1, g0, g1, part;
};

__device__ __forceinline__ Slice slice_of(const NormArgs& a, int32_t s)
{
    Slice r;
    if (a.sl.parts == 1) {
        r.g0 = s * a.sl.groups;
        r.g1 = r.g0 + a.sl.groups < a.G ? r.g0 + a.sl.groups : a.G;
        r.c0 = r.g0 * a.cpg;
        r.c1 = r.g1 * a.cpg;
        r.part = 0;
    } else {
        r.g0 = s / a.sl.parts;
        r.g1 = r.g0 + 1;
        r.part = s - r.g0 * a.sl.parts;
        r.c0 = r.g0 * a.cpg + r.part * a.sl.width;
        const int32_t end = r.c0 + a.sl.width, last = r.g1 * a.cpg;
        r.c1 = end < last ? end : last;
    }
    return r;
}

__device__ __forceinline__ int64_t seg_at(const NormArgs& a, int64_t b)
{
    if (!a.seg) return b * (a.N / a.B);
    const int64_t v = a.seg[b];
    return v < 0 ? 0 : v > a.N ? a.N : v;
}

// Last segment that begins at or before row r, found by the whole block: every
// round counts the probes at or below r among kThreads spread over what is left.
__device__ __forceinline__ int64_t find_segment(const NormArgs& a, int64_t r)
{
    if (!a.seg) return r / (a.N / a.B);
    int64_t lo = 0, n = a.B;
    while (n > 1) {
        const int64_t step = (n + kThreads - 1) / kThreads;
        const int64_t i = lo + (int64_t)threadIdx.x * step;
        const int c = __syncthreads_count((int64_t)threadIdx.x * step < n && seg_at(a, i) <= r);
        const int64_t k = c > 0 ? c - 1 : 0, left = n - k * step;
        lo += k * step;
        n = step < left ? step : left;
    }
    return lo;
}

// f(segment, first row, end row) for every piece of rows [r0, r1), the same for
// the whole block.  Stops where offsets break the precondition.
template <class F>
__device__ __forceinline__ void for_pieces(const NormArgs& a, int64_t r0, int64_t r1, F&& f)
{
    int64_t r = r0, b = find_segment(a, r0);
    while (r < r1) {
        int64_t e = seg_at(a, b + 1);
        if (e <= r) {  // empty segments: find the one that holds row r
            b = find_segment(a, r);
            e = seg_at(a, b + 1);
            if (e <= r) return;
        }
        if (e > r1) e = r1;
        f(b, r, e);
        r = e;
        if (++b >= a.B) return;
    }
}

// ---- activation ----------------------------------------------------------------------
// 1 ulp reciprocal and exp2: the error stays at that of the fp32 arguments
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// tanh from exp(2|z|): 1 - 2 / (e + 1), by its series where that would cancel
__device__ __forceinline__ float tanh_f(float z)
{
    const float t = fabsf(z);
    if (t < 0.3f) {
        const float u = z * z;
        // z (1 - u/3 + 2u^2/15 - 17u^3/315 + 62u^4/2835 - 1382u^5/155925)
        return z * (1.0f + u * (-0.33333334f + u * (0.13333334f + u * (-0.053968254f + u * (0.021869488f + u * -0.0088632355f)))));
    }
    const float e = __expf(2.0f * t);
    return copysignf(1.0f - 2.0f * __builtin_amdgcn_rcpf(e + 1.0f), z);
}

__device__ __forceinline__ float act_of(int act, float z)
{
    if (act == 0) return z;
    return act == 1 ? z * sigmoid(z) : tanh_f(z);
}

// act'(z)
__device__ __forceinline__ float act_slope(int act, float z)
{
    if (act == 0) return 1.0f;
    if (act == 1) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    const float t = tanh_f(z);
    return 1.0f - t * t;
}

// ---- lanes ---------------------------------------------------------------------------
// The block's place in its slice: L lanes along the channels, RL rows at a time.
template <int VEC>
struct Lanes {
    int32_t L, RL, rl, c;  // c: the lane's first channel
    bool on;
    __device__ __forceinline__ Lanes(const Slice& s)
    {
        L = (s.c1 - s.c0) / VEC;
        RL = kThreads / L;
        rl = (int32_t)threadIdx.x / L;
        c = s.c0 + ((int32_t)threadIdx.x - rl * L) * VEC;
        on = rl < RL;
    }
};

template <int VEC>
__device__ __forceinline__ void load_chan(float (&v)[VEC], const float* __restrict__ p, int32_t c, float none)
{
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = p ? p[c + j] : none;
}

// out[(group)] = sums over the block of two values per (lane, channel) for each group of the slice, written by the
// group's first thread to dst(g)[0..1].  s: kThreads * VEC * 2 doubles.
template <int VEC, class Dst>
__device__ __forceinline__ void group_sums(const NormArgs& a, const Slice& sl, const Lanes<VEC>& ln,
                                           const double (&u)[VEC], const double (&v)[VEC], double* s, Dst&& dst)
{
    // channels of one access in one group: one pair per lane, else one per channel
    const bool lane_sums = a.cpg % VEC == 0;
    const int32_t per = lane_sums ? 1 : VEC, w = ln.L * per;  // pairs per row lane
    __syncthreads();
    if (ln.on) {
        double* d = s + ((int64_t)ln.rl * w + (ln.c - sl.c0) / VEC * per) * 2;
        if (lane_sums) {
            double x = 0.0, y = 0.0;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                x += u[j];
                y += v[j];
            }
            d[0] = x;
            d[1] = y;
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                d[2 * j] = u[j];
                d[2 * j + 1] = v[j];
            }
        }
    }
    __syncthreads();
    // teams of up to 64 threads, one group each
    const int32_t groups = sl.g1 - sl.g0, each = w / groups;  // pairs of a group per row lane
    int32_t team = 64;
    while (team > 1 && team * groups > kThreads) team /= 2;
    const int32_t m = (int32_t)threadIdx.x & (team - 1);
    for (int32_t g = (int32_t)threadIdx.x / team; g - (int32_t)threadIdx.x / team < groups; g += kThreads / team) {
        double x = 0.0, y = 0.0;
        if (g < groups)
            for (int32_t k = m; k < each * ln.RL; k += team) {
                const int32_t row = k / each, at = (row * w + g * each + (k - row * each)) * 2;
                x += s[at];
                y += s[at + 1];
            }
        for (int32_t d = team / 2; d > 0; d /= 2) {
            x += __shfl_down(x, d, team);
            y += __shfl_down(y, d, team);
        }
        if (m == 0 && g < groups) {
            double* o = dst(sl.g0 + g);
            o[0] = x;
            o[1] = y;
        }
    }
}

__device__ __forceinline__ double* piece_sums(const NormArgs& a, int64_t run, int64_t b, int32_t g, int32_t part)
{
    return a.part + (((run + b) * a.G + g) * a.sl.parts + part) * 2;
}

// ---- forward -------------------------------------------------------------------------
// sums of x and x^2 of every piece
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_norm_sums(NormArgs a, const T* __restrict__ x)
{
    __shared__ double s[kThreads * VEC * 2];
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(sl);
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        const int64_t r0 = run * a.R, r1 = r0 + a.R < a.N ? r0 + a.R : a.N;
        for_pieces(a, r0, r1, [&](int64_t b, int64_t p, int64_t e) {
            double u[VEC], v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[j] = v[j] = 0.0;
            if (ln.on) {
#pragma unroll 4
                for (int64_t r = p + ln.rl; r < e; r += ln.RL) {
                    float f[VEC];
                    load_vec<T, VEC>(f, x + r * a.ldx + ln.c);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const double d = (double)f[j];
                        u[j] += d;
                        v[j] += d * d;
                    }
                }
            }
            group_sums<VEC>(a, sl, ln, u, v, s, [&](int32_t g) { return piece_sums(a, run, b, g, sl.part); });
        });
    }
}

// Sums of the pieces of one (segment, group), by one wave, in an order that
// depends on the shapes only.
__device__ __forceinline__ void sum_pieces(const NormArgs& a, int64_t b, int32_t g, double& x, double& y, double& M)
{
    const int lane = threadIdx.x & 63;
    const int64_t p = seg_at(a, b), e = seg_at(a, b + 1);
    x = y = 0.0;
    M = (double)(e > p ? e - p : 0) * a.cpg;
    if (e > p) {
        const int64_t k0 = p / a.R + b, n = ((e - 1) / a.R + b - k0 + 1) * a.sl.parts;
        for (int64_t k = lane; k < n; k += 64) {
            const int64_t at = ((k0 + k / a.sl.parts) * a.G + g) * a.sl.parts + k % a.sl.parts;
            x += a.part[2 * at];
            y += a.part[2 * at + 1];
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) {
        x += __shfl_xor(x, d, 64);
        y += __shfl_xor(y, d, 64);
    }
}

// mean and rstd of (segment, group): one wave each
__device__ __forceinline__ void finish_stats(const NormArgs& a, double x, double y, double M, float& mean, float& rstd)
{
    const double mu = M > 0.0 ? x / M : 0.0, sq = M > 0.0 ? y / M : 0.0;
    double var = sq - mu * mu;
    if (var < 0.0) var = 0.0;  // rounding; a NaN stays
    mean = (float)mu;
    rstd = (float)(1.0 / sqrt(var + (double)a.eps));
}

__global__ void __launch_bounds__(kThreads) k_norm_stats(NormArgs a)
{
    const int64_t n = a.B * a.G, step = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64; i < n; i += step) {
        double x, y, M;
        sum_pieces(a, i / a.G, (int32_t)(i % a.G), x, y, M);
        if ((threadIdx.x & 63) == 0) finish_stats(a, x, y, M, a.omean[i], a.orstd[i]);
    }
}

// per-channel values of a lane: its groups' values v[b][g] (stride 1 or 2)
template <int VEC, class S>
__device__ __forceinline__ void load_group(S (&o)[VEC], const S* __restrict__ v, const NormArgs& a, int64_t b,
                                           int32_t c, int32_t stride, int32_t off)
{
    const S* p = v + b * a.G * stride + off;
    if (a.cpg % VEC == 0) {
        const S w = p[c / a.cpg * stride];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = w;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = p[(c + j) / a.cpg * stride];
    }
}

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_norm_apply(NormArgs a, const T* __restrict__ x, T* __restrict__ y)
{
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(sl);
    float gm[VEC], bt[VEC];
    if (ln.on) {
        load_chan<VEC>(gm, a.gamma, ln.c, 1.0f);
        load_chan<VEC>(bt, a.beta, ln.c, 0.0f);
    }
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        const int64_t r0 = run * a.R, r1 = r0 + a.R < a.N ? r0 + a.R : a.N;
        for_pieces(a, r0, r1, [&](int64_t b, int64_t p, int64_t e) {
            if (!ln.on) return;
            float mu[VEC], rs[VEC];
            load_group(mu, a.omean, a, b, ln.c, 1, 0);
            load_group(rs, a.orstd, a, b, ln.c, 1, 0);
#pragma unroll 4
            for (int64_t r = p + ln.rl; r < e; r += ln.RL) {
                float f[VEC];
                load_vec<T, VEC>(f, x + r * a.ldx + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) f[j] = act_of(a.act, (f[j] - mu[j]) * rs[j] * gm[j] + bt[j]);
                store_vec<T, VEC>(y + r * a.ldy + ln.c, f);
            }
        });
    }
}

// ---- backward ------------------------------------------------------------------------
// sums of h and h xhat of every piece, and of dz xhat and dz of every run
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_sums(NormArgs a, const T* __restrict__ x,
                                                            const T* __restrict__ dy)
{
    __shared__ double s[kThreads * VEC * 2];
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(sl);
    float gm[VEC], bt[VEC];
    if (ln.on) {
        load_chan<VEC>(gm, a.gamma, ln.c, 1.0f);
        load_chan<VEC>(bt, a.beta, ln.c, 0.0f);
    }
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        const int64_t r0 = run * a.R, r1 = r0 + a.R < a.N ? r0 + a.R : a.N;
        double tu[VEC], tv[VEC];  // dz xhat and dz of the run
#pragma unroll
        for (int j = 0; j < VEC; ++j) tu[j] = tv[j] = 0.0;
        for_pieces(a, r0, r1, [&](int64_t b, int64_t p, int64_t e) {
            double u[VEC], v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[j] = v[j] = 0.0;
            if (ln.on) {
                float mu[VEC], rs[VEC];
                load_group(mu, a.mean, a, b, ln.c, 1, 0);
                load_group(rs, a.rstd, a, b, ln.c, 1, 0);
#pragma unroll 2
                for (int64_t r = p + ln.rl; r < e; r += ln.RL) {
                    float f[VEC], d[VEC];
                    load_vec<T, VEC>(f, x + r * a.ldx + ln.c);
                    load_vec<T, VEC>(d, dy + r * a.ldy + ln.c);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float xh = (f[j] - mu[j]) * rs[j];
                        const double dz = (double)(d[j] * act_slope(a.act, xh * gm[j] + bt[j]));
                        u[j] += dz * (double)xh;
                        v[j] += dz;
                    }
                }
            }
            double hu[VEC], hv[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                tu[j] += u[j];
                tv[j] += v[j];
                hu[j] = ln.on ? v[j] * (double)gm[j] : 0.0;
                hv[j] = ln.on ? u[j] * (double)gm[j] : 0.0;
            }
            if (a.coef)
                group_sums<VEC>(a, sl, ln, hu, hv, s, [&](int32_t g) { return piece_sums(a, run, b, g, sl.part); });
        });
        if (!a.chan) continue;
        // the run's sums per channel
        const int32_t w = ln.L * VEC;
        __syncthreads();
        if (ln.on) {
            double* d = s + ((int64_t)ln.rl * w + (ln.c - sl.c0)) * 2;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                d[2 * j] = tu[j];
                d[2 * j + 1] = tv[j];
            }
        }
        __syncthreads();
        for (int32_t k = threadIdx.x; k < 2 * w; k += kThreads) {
            double t = 0.0;
            for (int32_t r = 0; r < ln.RL; ++r) t += s[(int64_t)r * w * 2 + k];
            a.chan[(run * 2 + (k & 1)) * a.C + sl.c0 + k / 2] = t;
        }
        __syncthreads();
    }
}

// blocks [0, cblocks): dgamma and dbeta of kChan channels each, from the runs;
// the others: the two group means of dx, one wave per (segment, group)
constexpr int kChan = 8;
__global__ void __launch_bounds__(kThreads) k_norm_bwd_join(NormArgs a, int32_t cblocks, float* __restrict__ dgamma,
                                                            float* __restrict__ dbeta)
{
    if ((int32_t)blockIdx.x < cblocks) {
        __shared__ double s[kThreads];
        constexpr int kW = 2 * kChan, kR = kThreads / kW;  // 16 sums, 16 rows of runs at a time
        const int32_t col = (int32_t)threadIdx.x % kW, row = (int32_t)threadIdx.x / kW;
        const int32_t which = col / kChan, c = (int32_t)blockIdx.x * kChan + col % kChan;
        double t = 0.0;
        if (c < a.C)
#pragma unroll 4
            for (int64_t r = row; r < a.runs; r += kR) t += a.chan[(r * 2 + which) * a.C + c];
        s[threadIdx.x] = t;
        __syncthreads();
        if (row == 0 && c < a.C) {
            double v = 0.0;
            for (int k = 0; k < kR; ++k) v += s[k * kW + col];
            float* o = which == 0 ? dgamma : dbeta;
            if (o) o[c] = (float)v;
        }
        return;
    }
    const int64_t n = a.B * a.G, step = (int64_t)(gridDim.x - cblocks) * (kThreads / 64);
    for (int64_t i = (int64_t)((int32_t)blockIdx.x - cblocks) * (kThreads / 64) + threadIdx.x / 64; i < n; i += step) {
        double x, y, M;
        sum_pieces(a, i / a.G, (int32_t)(i % a.G), x, y, M);
        if ((threadIdx.x & 63) == 0) {
            a.coef[2 * i] = M > 0.0 ? x / M : 0.0;
            a.coef[2 * i + 1] = M > 0.0 ? y / M : 0.0;
        }
    }
}

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_apply(NormArgs a, const T* __restrict__ x,
                                                             const T* __restrict__ dy, T* __restrict__ dx)
{
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(sl);
    float gm[VEC], bt[VEC];
    if (ln.on) {
        load_chan<VEC>(gm, a.gamma, ln.c, 1.0f);
        load_chan<VEC>(bt, a.beta, ln.c, 0.0f);
    }
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        const int64_t r0 = run * a.R, r1 = r0 + a.R < a.N ? r0 + a.R : a.N;
        for_pieces(a, r0, r1, [&](int64_t b, int64_t p, int64_t e) {
            if (!ln.on) return;
            float mu[VEC], rs[VEC];
            double s1[VEC], s2[VEC];
            load_group(mu, a.mean, a, b, ln.c, 1, 0);
            load_group(rs, a.rstd, a, b, ln.c, 1, 0);
            load_group(s1, a.coef, a, b, ln.c, 2, 0);
            load_group(s2, a.coef, a, b, ln.c, 2, 1);
#pragma unroll 2
            for (int64_t r = p + ln.rl; r < e; r += ln.RL) {
                float f[VEC], d[VEC];
                load_vec<T, VEC>(f, x + r * a.ldx + ln.c);
                load_vec<T, VEC>(d, dy + r * a.ldy + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float xh = (f[j] - mu[j]) * rs[j];
                    const float dz = d[j] * act_slope(a.act, xh * gm[j] + bt[j]);
                    // fp64: the three terms cancel where a group holds few values
                    f[j] = rs[j] * (float)((double)dz * (double)gm[j] - s1[j] - (double)xh * s2[j]);
                }
                store_vec<T, VEC>(dx + r * a.ldd + ln.c, f);
            }
        });
    }
}

// ---- layout --------------------------------------------------------------------------
// Rows per run: about 2048 blocks over the rows, at least 16 rows, so that the
// sums of a run are a small share of its rows.
int64_t rows_per_run(int64_t N)
{
    const int64_t r = cdiv64(N, 2048);
    return r < 16 ? 16 : r;
}

struct NormLayout {
    int64_t R, runs, parts;
    size_t part, chan, coef, bytes;
};

NormLayout norm_layout(const NormShape& n)
{
    NormLayout w{};
    w.R = rows_per_run(n.N);
    w.runs = cdiv64(n.N, w.R);
    const int64_t cpg = n.C / n.G;
    w.parts = cdiv64(cpg, kThreads);  // at least as many as any form needs
    size_t o = 0;
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o += align256((size_t)bytes);
        return at;
    };
    w.part = take((w.runs + n.B) * n.G * w.parts * 2 * (int64_t)sizeof(double));
    w.chan = take(w.runs * 2 * n.C * (int64_t)sizeof(double));
    w.coef = take(n.B * n.G * 2 * (int64_t)sizeof(double));
    w.bytes = o > 0 ? o : 256;  // never none, so that a workspace always has an address
    return w;
}

Slices slices_of(const NormShape& n, int vec)
{
    Slices s{};
    const int32_t cpg = n.C / n.G, most = kThreads * vec;
    if (cpg <= most) {
        s.parts = 1;
        s.groups = most / cpg < n.G ? most / cpg : n.G;
        s.width = s.groups * cpg;
        s.n = (n.G + s.groups - 1) / s.groups;
    } else {
        s.groups = 1;
        s.parts = (cpg + most - 1) / most;
        s.width = ((cpg + s.parts - 1) / s.parts + vec - 1) / vec * vec;
        s.n = n.G * s.parts;
    }
    return s;
}

// 16-byte accesses need every slice to begin and end on them
bool wide_ok(const NormShape& n, int vec)
{
    if (n.C % vec != 0) return false;
    return n.C <= kThreads * vec || (n.C / n.G) % vec == 0;
}

NormArgs norm_args(const NormShape& n, int vec, void* ws)
{
    const NormLayout w = norm_layout(n);
    NormArgs a{};
    a.N = n.N;
    a.B = n.B;
    a.R = w.R;
    a.runs = w.runs;
    a.ldx = n.ldx;
    a.ldy = n.ldy;
    a.ldd = n.ldd;
    a.C = n.C;
    a.G = n.G;
    a.cpg = n.C / n.G;
    a.sl = slices_of(n, vec);
    a.eps = n.eps;
    a.act = n.act;
    a.seg = n.seg;
    a.part = (double*)((char*)ws + w.part);
    a.chan = (double*)((char*)ws + w.chan);
    a.coef = (double*)((char*)ws + w.coef);
    return a;
}

inline unsigned stat_blocks(const NormArgs& a) { return grid_of(cdiv64(a.B * a.G, kThreads / 64)); }

template <class T, int VEC>
hipError_t norm_fwd(const NormArgs& a, const void* x, void* y, hipStream_t s)
{
    const dim3 grid(grid_of(a.runs), (unsigned)a.sl.n);
    if (a.N > 0) hipLaunchKernelGGL((k_norm_sums<T, VEC>), grid, dim3(kThreads), 0, s, a, (const T*)x);
    hipLaunchKernelGGL(k_norm_stats, dim3(stat_blocks(a)), dim3(kThreads), 0, s, a);
    if (a.N > 0) hipLaunchKernelGGL((k_norm_apply<T, VEC>), grid, dim3(kThreads), 0, s, a, (const T*)x, (T*)y);
    return hipGetLastError();
}

template <class T, int VEC>
hipError_t norm_bwd(const NormArgs& a, const void* x, const void* dy, void* dx, float* dgamma, float* dbeta,
                    hipStream_t s)
{
    const dim3 grid(grid_of(a.runs), (unsigned)a.sl.n);
    if (a.N > 0)
        hipLaunchKernelGGL((k_norm_bwd_sums<T, VEC>), grid, dim3(kThreads), 0, s, a, (const T*)x, (const T*)dy);
    const unsigned cb = a.chan ? (unsigned)cdiv64(a.C, kChan) : 0, sb = a.coef ? stat_blocks(a) : 0;
    if (cb + sb > 0)
        hipLaunchKernelGGL(k_norm_bwd_join, dim3(cb + sb), dim3(kThreads), 0, s, a, (int32_t)cb, dgamma, dbeta);
    if (a.N > 0 && dx)
        hipLaunchKernelGGL((k_norm_bwd_apply<T, VEC>), grid, dim3(kThreads), 0, s, a, (const T*)x, (const T*)dy,
                           (T*)dx);
    return hipGetLastError();
}

}  // namespace

size_t norm_workspace_bytes(const NormShape& n) { return norm_layout(n).bytes; }

hipError_t launch_norm_fwd(const NormShape& n, const void* x, const float* gamma, const float* beta, void* y,
                           float* mean, float* rstd, void* ws, hipStream_t s)
{
    if (n.B == 0) return hipSuccess;
    const int64_t es = dtype_size(n.dtype);
    const int vec = (int)(16 / es);
    const bool wide = wide_ok(n, vec) && aligned_rows(x, n.ldx, es) && aligned_rows(y, n.ldy, es);
    NormArgs a = norm_args(n, wide ? vec : 1, ws);
    a.gamma = gamma;
    a.beta = beta;
    a.omean = mean;
    a.orstd = rstd;
    if (n.dtype == kF32)
        return wide ? norm_fwd<float, kWide<float>>(a, x, y, s) : norm_fwd<float, 1>(a, x, y, s);
    return wide ? norm_fwd<bf16_t, kWide<bf16_t>>(a, x, y, s) : norm_fwd<bf16_t, 1>(a, x, y, s);
}

hipError_t launch_norm_bwd(const NormShape& n, const void* x, const float* mean, const float* rstd,
                           const float* gamma, const float* beta, const void* dy, void* dx, float* dgamma,
                           float* dbeta, void* ws, hipStream_t s)
{
    const int64_t es = dtype_size(n.dtype);
    const int vec = (int)(16 / es);
    const bool wide = wide_ok(n, vec) && aligned_rows(x, n.ldx, es) && aligned_rows(dy, n.ldy, es) &&
                      (!dx || aligned_rows(dx, n.ldd, es));
    NormArgs a = norm_args(n, wide ? vec : 1, ws);
    a.mean = mean;
    a.rstd = rstd;
    a.gamma = gamma;
    a.beta = beta;
    if (!dx) a.coef = nullptr;
    if (!dgamma && !dbeta) a.chan = nullptr;
    if (n.dtype == kF32)
        return wide ? norm_bwd<float, kWide<float>>(a, x, dy, dx, dgamma, dbeta, s)
                    : norm_bwd<float, 1>(a, x, dy, dx, dgamma, dbeta, s);
    return wide ? norm_bwd<bf16_t, kWide<bf16_t>>(a, x, dy, dx, dgamma, dbeta, s)
                : norm_bwd<bf16_t, 1>(a, x, dy, dx, dgamma, dbeta, s);
}

}  // namespace cgtp
