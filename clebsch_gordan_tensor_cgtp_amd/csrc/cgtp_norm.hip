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
// and dy and writes dx.  The lanes of a block run along the channels, so every
// access is a contiguous row.  Two forms:
//   - a block per segment (and slice of whole groups), its rows kept in registers
//     between the statistics and the result: one pass over memory, one launch;
//   - for segments too long for that, blocks take runs of consecutive rows of
//     equal length.  A run may hold the end of one segment and the beginning of
//     others; each (run, segment) piece leaves its sums at the place run + segment
//     of a list, which is unique because every new piece moves on by a run or a
//     segment, a second kernel adds the pieces of a segment in order, and a third
//     reads the rows again.
// The lengths of ragged segments are known on the device only: where their mean
// is short but the total is large enough that one long segment would hold up the
// chip, both forms are launched and each takes the segments on its side of a
// length.  Sums over the rows are fp64.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

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
    int64_t longest;  // rows of a segment that a block takes whole; the runs take the longer ones
    int32_t C, G, cpg;
    Slices sl;
    float eps;
    const int32_t* seg;
    const float *gamma, *beta, *mean, *rstd;
    float *omean, *orstd;
    double* part;  // [runs + B][G][parts][2]
    double* chan;  // backward: [runs, then the whole segments' blocks][2][C]
    int64_t nchan;
    float* coef;   // backward: [B][G][2], the group means of h and h xhat
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

// f(segment, first row, end row) for every piece of rows [r0, r1) of a segment of
// more than `longest` rows, the same for the whole block.  Stops where offsets
// break the precondition.
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
        const bool take = e - seg_at(a, b) > a.longest;
        if (e > r1) e = r1;
        if (take) f(b, r, e);
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
    const float t = fabsf(z), u = z * z;
    // z (1 - u/3 + 2u^2/15 - 17u^3/315 + 62u^4/2835 - 1382u^5/155925)
    const float near = z * (1.0f + u * (-0.33333334f + u * (0.13333334f + u * (-0.053968254f + u * (0.021869488f + u * -0.0088632355f)))));
    const float far = copysignf(1.0f - 2.0f * __builtin_amdgcn_rcpf(__expf(2.0f * t) + 1.0f), z);
    return t < 0.3f ? near : far;
}

enum : int { kNone = 0, kSilu = 1, kTanh = 2 };  // values of cgtp_act_t

template <int ACT>
__device__ __forceinline__ float act_of(float z)
{
    if constexpr (ACT == kNone) return z;
    if constexpr (ACT == kSilu) return z * sigmoid(z);
    return tanh_f(z);
}

// act'(z)
template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == kNone) return 1.0f;
    if constexpr (ACT == kSilu) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    const float t = tanh_f(z);
    return 1.0f - t * t;
}

// ---- lanes ---------------------------------------------------------------------------
// The block's place in its slice: L lanes along the channels, RL rows at a time.
template <int VEC, int THR = kThreads>
struct Lanes {
    int32_t L, RL, rl, c;  // c: the lane's first channel
    int32_t g[VEC];        // its channels' groups
    bool on;
    __device__ __forceinline__ Lanes(const NormArgs& a, const Slice& s)
    {
        L = (s.c1 - s.c0) / VEC;
        RL = THR / L;
        rl = (int32_t)threadIdx.x / L;
        c = s.c0 + ((int32_t)threadIdx.x - rl * L) * VEC;
        on = rl < RL;
        // the divisions are done here, once
        const bool one = a.cpg % VEC == 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[j] = one && j > 0 ? g[0] : (c + j) / a.cpg;
    }
};

template <int VEC>
__device__ __forceinline__ void load_chan(float (&v)[VEC], const float* __restrict__ p, int32_t c, float none)
{
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = p ? p[c + j] : none;
}

// LDS of a block: doubles for the group sums (a pair per lane, or per channel
// where a group's channels are no whole accesses), for the backward those of dz
// xhat and dz of every lane and channel, then the groups' two results.
extern __shared__ __attribute__((aligned(16))) char norm_lds[];

__host__ __device__ inline int sum_doubles(int32_t cpg, int vec, int threads, bool channels)
{
    return 2 * (cpg % vec == 0 ? threads : threads * vec) + (channels ? 2 * threads * vec : 0);
}

// out[(group)] = sums over the block of two values per (lane, channel) for each group of the slice, written by the
// group's first thread by dst(g, sum, sum).  s: THR * VEC * 2 doubles (THR * 2
// where a group's channels are whole accesses).
template <int VEC, int THR, class Dst>
__device__ __forceinline__ void group_sums(const NormArgs& a, const Slice& sl, const Lanes<VEC, THR>& ln,
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
    while (team > 1 && team * groups > THR) team /= 2;
    const int32_t m = (int32_t)threadIdx.x & (team - 1);
    for (int32_t g = (int32_t)threadIdx.x / team; g - (int32_t)threadIdx.x / team < groups; g += THR / team) {
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
        if (m == 0 && g < groups) dst(sl.g0 + g, x, y);
    }
}

__device__ __forceinline__ void put_piece(const NormArgs& a, int64_t run, int64_t b, int32_t g, int32_t part, double x,
                                          double y)
{
    double* o = a.part + (((run + b) * a.G + g) * a.sl.parts + part) * 2;
    o[0] = x;
    o[1] = y;
}

// Rows first, first + RL, .. below e of a lane, kAt at a time and two such batches in
// turn: load(row, batch) brings a batch (rows beyond e as the first), work(row, batch,
// masked) takes it; the next loads are out before the work on these.
template <int kAt, class Batch, class Load, class Work>
__device__ __forceinline__ void row_batches(int64_t first, int64_t e, int32_t RL, Load&& load, Work&& work)
{
    if (first >= e) return;
    const int64_t step = (int64_t)kAt * RL;
    int64_t r = first;
    Batch b0, b1;
    load(r, b0);
    for (; r + 2 * step - RL < e; r += 2 * step) {
        load(r + step, b1);
        work(r, b0, std::false_type{});
        load(r + 2 * step, b0);
        work(r + step, b1, std::false_type{});
    }
    if (r < e) {
        load(r + step, b1);
        work(r, b0, std::true_type{});
        work(r + step, b1, std::true_type{});
    }
}

// u += x, v += x^2 over the lane's rows below e, in fp64 (fp32 holds no squares beyond
// 1.8e19).  Taken from the lane's first value of each channel, so that little cancels:
// sum x = n ref + D, sum x^2 = n ref^2 + 2 ref D + Q with D = sum (x - ref) and
// Q = sum (x - ref)^2.
template <int kAt, class T, int VEC, class Ln>
__device__ __forceinline__ void fwd_rows(const NormArgs& a, const Ln& ln, const T* __restrict__ x, int64_t p,
                                         int64_t e, double (&u)[VEC], double (&v)[VEC])
{
    struct Batch {
        Raw<T, VEC> f[kAt];
    };
    const int64_t first = p + ln.rl;
    if (first >= e) return;
    const T* xp = x + first * a.ldx + ln.c;
    double ref[VEC], D[VEC], Q[VEC];
    {
        Raw<T, VEC> f;
        f.load(xp);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            ref[j] = (double)f[j];
            D[j] = Q[j] = 0.0;
        }
    }
    auto load = [&](int64_t r, Batch& b) {
#pragma unroll
        for (int k = 0; k < kAt; ++k) b.f[k].load(r + k * ln.RL < e ? xp + (r - first + k * ln.RL) * a.ldx : xp);
    };
    auto work = [&](int64_t r, const Batch& b, auto masked) {
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
            // a row beyond e was loaded as the first: its difference is zero
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const double d = (double)b.f[k][j] - ref[j];
                D[j] += d;
                Q[j] += d * d;
            }
        }
    };
    row_batches<kAt, Batch>(first, e, ln.RL, load, work);
    const double n = (double)((e - first + ln.RL - 1) / ln.RL);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        u[j] += n * ref[j] + D[j];
        v[j] += ref[j] * (n * ref[j] + 2.0 * D[j]) + Q[j];
    }
}

// ---- forward -------------------------------------------------------------------------
// Figures of the runs are for eight segments of 50001 x 256 rows (bf16 205 MB, fp32 410 MB).
// sums of x and x^2 of every piece: bound by reading x, bf16 46 us, fp32 92 us (4.5 TB/s).
// The fp64 arithmetic hides behind it (four rows in fp32 first: the same within 1 %).
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_norm_sums(NormArgs a, const T* __restrict__ x)
{
    double* s = reinterpret_cast<double*>(norm_lds);
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(a, sl);
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        const int64_t r0 = run * a.R, r1 = r0 + a.R < a.N ? r0 + a.R : a.N;
        for_pieces(a, r0, r1, [&](int64_t b, int64_t p, int64_t e) {
            double u[VEC], v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[j] = v[j] = 0.0;
            if (ln.on) fwd_rows<4, T, VEC>(a, ln, x, p, e, u, v);
            group_sums(a, sl, ln, u, v, s,
                       [&](int32_t g, double x, double y) { put_piece(a, run, b, g, sl.part, x, y); });
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

// a wave per (segment, group): 6 us, a launch and the pieces' latency
__global__ void __launch_bounds__(kThreads) k_norm_stats(NormArgs a)
{
    const int64_t n = a.B * a.G, step = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64; i < n; i += step) {
        double x, y, M;
        if (a.longest > 0 && seg_at(a, i / a.G + 1) - seg_at(a, i / a.G) <= a.longest) continue;
        sum_pieces(a, i / a.G, (int32_t)(i % a.G), x, y, M);
        if ((threadIdx.x & 63) == 0) finish_stats(a, x, y, M, a.omean[i], a.orstd[i]);
    }
}

// per-channel values of a lane: its groups' values v[b][g] (stride 1 or 2)
template <int VEC, class Ln>
__device__ __forceinline__ void load_group(float (&o)[VEC], const float* __restrict__ v, const NormArgs& a, int64_t b,
                                           const Ln& ln, int32_t stride, int32_t off)
{
    const float* p = v + b * a.G * stride + off;
    if (a.cpg % VEC == 0) {
        const float w = p[ln.g[0] * stride];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = w;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = p[ln.g[j] * stride];
    }
}

// Bound by memory: bf16 79 us (5.2 TB/s read and written), fp32 146 us (5.6 TB/s).
template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads) k_norm_apply(NormArgs a, const T* __restrict__ x, T* __restrict__ y)
{
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(a, sl);
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
            load_group(mu, a.omean, a, b, ln, 1, 0);
            load_group(rs, a.orstd, a, b, ln, 1, 0);
#pragma unroll 4
            for (int64_t r = p + ln.rl; r < e; r += ln.RL) {
                Raw<T, VEC> f;
                float g[VEC];
                f.load(x + r * a.ldx + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = act_of<ACT>((f[j] - mu[j]) * rs[j] * gm[j] + bt[j]);
                store_vec<T, VEC>(y + r * a.ldy + ln.c, g);
            }
        });
    }
}

// ---- backward ------------------------------------------------------------------------
// sums of h and h xhat of every piece, and of dz xhat and dz of every run
// u += dz xhat, v += dz over rows p + rl, p + rl + RL, .. below e, kAt rows' loads at
// a time: fp32 terms, fp64 sums
template <int kAt, class T, int VEC, int ACT, class Ln>
__device__ __forceinline__ void bwd_rows(const NormArgs& a, const Ln& ln, const T* __restrict__ x,
                                         const T* __restrict__ dy, int64_t p, int64_t e, const float (&mu)[VEC],
                                         const float (&rs)[VEC], const float (&gm)[VEC], const float (&bt)[VEC],
                                         double (&u)[VEC], double (&v)[VEC])
{
    struct Batch {
        Raw<T, VEC> f[kAt], d[kAt];
    };
    const int64_t first = p + ln.rl;
    const T *xp = x + first * a.ldx + ln.c, *dp = dy + first * a.ldy + ln.c;
    auto load = [&](int64_t r, Batch& b) {
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
            const bool in = r + k * ln.RL < e;
            b.f[k].load(in ? xp + (r - first + k * ln.RL) * a.ldx : xp);
            b.d[k].load(in ? dp + (r - first + k * ln.RL) * a.ldy : dp);
        }
    };
    auto work = [&](int64_t r, const Batch& b, auto masked) {
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
            const bool in = !decltype(masked)::value || r + k * ln.RL < e;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float xh = (b.f[k][j] - mu[j]) * rs[j];
                const float dz = in ? b.d[k][j] * act_slope<ACT>(xh * gm[j] + bt[j]) : 0.0f;
                u[j] += (double)(dz * xh);
                v[j] += (double)dz;
            }
        }
    };
    row_batches<kAt, Batch>(first, e, ln.RL, load, work);
}

// dx of one element.  h is rounded as the group sums' terms are, so that a group
// of one value gives exactly zero.
__device__ __forceinline__ float dx_of(float xh, float dz, float rs, float gm, float s1, float s2)
{
    return rs * (__fmul_rn(dz, gm) - s1 - xh * s2);
}

template <int ACT>
__device__ __forceinline__ float dx_of(float x, float dy, float mu, float rs, float gm, float bt, float s1, float s2)
{
    const float xh = (x - mu) * rs;
    return dx_of(xh, dy * act_slope<ACT>(xh * gm + bt), rs, gm, s1, s2);
}

// Sums over a block's pieces of dz xhat and of dz, kept in LDS (they change once a
// piece): place j of lane t of the first at j THR + t, the second VEC THR further on.
template <int VEC, int THR>
struct Totals {
    double* t;
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < 2 * VEC; ++j) t[j * THR + threadIdx.x] = 0.0;
    }
    __device__ __forceinline__ void add(const double (&u)[VEC], const double (&v)[VEC])
    {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            t[j * THR + threadIdx.x] += u[j];
            t[(VEC + j) * THR + threadIdx.x] += v[j];
        }
    }
    // their sums over the rows' lanes to row `row` of a.chan
    __device__ __forceinline__ void store(const NormArgs& a, const Slice& sl, const Lanes<VEC, THR>& ln, int64_t row)
    {
        const int32_t w = ln.L * VEC;
        __syncthreads();
        for (int32_t k = threadIdx.x; k < 2 * w; k += THR) {
            const int32_t which = k / w, c = k - which * w;
            double v = 0.0;
            for (int32_t r = 0; r < ln.RL; ++r) v += t[(which * VEC + c % VEC) * THR + r * ln.L + c / VEC];
            a.chan[(row * 2 + which) * a.C + sl.c0 + c] = v;
        }
        __syncthreads();
    }
};

// Bound by reading x and dy: bf16 96 us, fp32 192 us (4.3 TB/s).
template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, 4) k_norm_bwd_sums(NormArgs a, const T* __restrict__ x,
                                                            const T* __restrict__ dy)
{
    double* s = reinterpret_cast<double*>(norm_lds);
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(a, sl);
    Totals<VEC, kThreads> total{s + sum_doubles(a.cpg, VEC, kThreads, false)};
    float gm[VEC], bt[VEC];
    if (ln.on) {
        load_chan<VEC>(gm, a.gamma, ln.c, 1.0f);
        load_chan<VEC>(bt, a.beta, ln.c, 0.0f);
    }
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        const int64_t r0 = run * a.R, r1 = r0 + a.R < a.N ? r0 + a.R : a.N;
        total.clear();
        for_pieces(a, r0, r1, [&](int64_t b, int64_t p, int64_t e) {
            double u[VEC], v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[j] = v[j] = 0.0;
            if (ln.on) {
                float mu[VEC], rs[VEC];
                load_group(mu, a.mean, a, b, ln, 1, 0);
                load_group(rs, a.rstd, a, b, ln, 1, 0);
                bwd_rows<2, T, VEC, ACT>(a, ln, x, dy, p, e, mu, rs, gm, bt, u, v);
            }
            total.add(u, v);
            double hu[VEC], hv[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                hu[j] = ln.on ? v[j] * (double)gm[j] : 0.0;
                hv[j] = ln.on ? u[j] * (double)gm[j] : 0.0;
            }
            if (a.coef)
                group_sums(a, sl, ln, hu, hv, s,
                           [&](int32_t g, double x, double y) { put_piece(a, run, b, g, sl.part, x, y); });
        });
        if (a.chan) total.store(a, sl, ln, run);
    }
}

// blocks [0, cblocks): dgamma and dbeta of kChan channels each, from the runs;
// the others: the two group means of dx, one wave per (segment, group).  8 us, and 6 us
// behind 1024 segments taken whole: a launch, and sums of a few hundred rows in turn.
constexpr int kChan = 4, kJoin = 1024;
__global__ void __launch_bounds__(kJoin) k_norm_bwd_join(NormArgs a, int32_t cblocks, float* __restrict__ dgamma,
                                                         float* __restrict__ dbeta)
{
    if ((int32_t)blockIdx.x < cblocks) {
        __shared__ double s[kJoin];
        constexpr int kW = 2 * kChan, kR = kJoin / kW;  // 8 sums, 128 rows of runs at a time
        const int32_t col = (int32_t)threadIdx.x % kW, row = (int32_t)threadIdx.x / kW;
        const int32_t which = col / kChan, c = (int32_t)blockIdx.x * kChan + col % kChan;
        double t = 0.0;
        if (c < a.C)
#pragma unroll 8
            for (int64_t r = row; r < a.nchan; r += kR) t += a.chan[(r * 2 + which) * a.C + c];
        s[threadIdx.x] = t;
        __syncthreads();
        for (int d = kR / 2; d > 0; d /= 2) {
            if (row < d) s[threadIdx.x] += s[threadIdx.x + d * kW];
            __syncthreads();
        }
        if (row == 0 && c < a.C) {
            float* o = which == 0 ? dgamma : dbeta;
            if (o) o[c] = (float)s[col];
        }
        return;
    }
    const int64_t n = a.B * a.G, step = (int64_t)(gridDim.x - cblocks) * (kJoin / 64);
    for (int64_t i = (int64_t)((int32_t)blockIdx.x - cblocks) * (kJoin / 64) + threadIdx.x / 64; i < n; i += step) {
        double x, y, M;
        if (a.longest > 0 && seg_at(a, i / a.G + 1) - seg_at(a, i / a.G) <= a.longest) continue;
        sum_pieces(a, i / a.G, (int32_t)(i % a.G), x, y, M);
        if ((threadIdx.x & 63) == 0) {
            a.coef[2 * i] = M > 0.0 ? (float)(x / M) : 0.0f;
            a.coef[2 * i + 1] = M > 0.0 ? (float)(y / M) : 0.0f;
        }
    }
}

// Bound by memory: bf16 115 us (5.3 TB/s), fp32 222 us (5.5 TB/s).  (Going through the
// segments in parts small enough to stay in the last-level cache between the two passes
// gained nothing: a part's launches cost what its cached reads save.)
template <class T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_apply(NormArgs a, const T* __restrict__ x,
                                                             const T* __restrict__ dy, T* __restrict__ dx)
{
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    const Lanes<VEC> ln(a, sl);
    float gm[VEC], bt[VEC];
    if (ln.on) {
        load_chan<VEC>(gm, a.gamma, ln.c, 1.0f);
        load_chan<VEC>(bt, a.beta, ln.c, 0.0f);
    }
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        // the rows that were read last first: the cache may still hold them
        const int64_t r0 = (a.runs - 1 - run) * a.R, r1 = r0 + a.R < a.N ? r0 + a.R : a.N;
        for_pieces(a, r0, r1, [&](int64_t b, int64_t p, int64_t e) {
            if (!ln.on) return;
            float mu[VEC], rs[VEC], s1[VEC], s2[VEC];
            load_group(mu, a.mean, a, b, ln, 1, 0);
            load_group(rs, a.rstd, a, b, ln, 1, 0);
            load_group(s1, a.coef, a, b, ln, 2, 0);
            load_group(s2, a.coef, a, b, ln, 2, 1);
#pragma unroll 4
            for (int64_t r = p + ln.rl; r < e; r += ln.RL) {
                Raw<T, VEC> f, d;
                float g[VEC];
                f.load(x + r * a.ldx + ln.c);
                d.load(dy + r * a.ldy + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = dx_of<ACT>(f[j], d[j], mu[j], rs[j], gm[j], bt[j], s1[j], s2[j]);
                store_vec<T, VEC>(dx + r * a.ldd + ln.c, g);
            }
        });
    }
}

// ---- a block per segment -----------------------------------------------------------------
// Bound by a block's chain of a load, two sums over its lanes and a store: 1024 segments of
// 25000 x 128 bf16 rows in all 11.1 us (1.2 TB/s), one segment of 2000 x 128 fp32 rows
// 10.4 us; backward, 1024 segments, fp32, 20.1 us (1.9 TB/s; its fp64 sums are 2.3 us of that:
// four rows in fp32 first lost small terms beside large ones).  A wave for each segment instead
// of a block took longer: few rows were in flight.
// Rows of a lane that stay in registers between the two passes; the rows of a
// longer segment are read again.
template <int THR>
constexpr int kKeep = THR == kThreads ? 4 : 8;
constexpr int kKeepBwd = 4;

// values of the lane's channels from v[group of the slice]
template <int VEC, class Ln>
__device__ __forceinline__ void slice_group(float (&o)[VEC], const float* v, const Slice& sl, const Ln& ln)
{
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = v[ln.g[j] - sl.g0];
}

template <class T, int VEC, int THR, int ACT>
__global__ void __launch_bounds__(THR) k_norm_seg(NormArgs a, const T* __restrict__ x, T* __restrict__ y)
{
    constexpr int KEEP = kKeep<THR>;
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    double* s = reinterpret_cast<double*>(norm_lds);
    float* st[2];
    st[0] = reinterpret_cast<float*>(s + sum_doubles(a.cpg, VEC, THR, false));
    st[1] = st[0] + a.sl.groups;
    const Lanes<VEC, THR> ln(a, sl);
    float gm[VEC], bt[VEC];
    if (ln.on) {
        load_chan<VEC>(gm, a.gamma, ln.c, 1.0f);
        load_chan<VEC>(bt, a.beta, ln.c, 0.0f);
    }
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int64_t p = seg_at(a, b), e = seg_at(a, b + 1);
        if (e - p > a.longest) continue;
        const double M = (double)(e > p ? e - p : 0) * a.cpg;
        Raw<T, VEC> f[KEEP];
        double u[VEC], v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[j] = v[j] = 0.0;
        const bool on = ln.on && p + ln.rl < e;
        const T* xp = x + (p + ln.rl) * a.ldx + ln.c;  // the lane's first row
        T* yp = y + (p + ln.rl) * a.ldy + ln.c;
        if (on) {
#pragma unroll
            for (int k = 0; k < KEEP; ++k) {
                const int64_t r = p + ln.rl + (int64_t)k * ln.RL;
                f[k].load(xp + (r < e ? (int64_t)k * ln.RL * a.ldx : 0));
            }
#pragma unroll
            for (int k = 0; k < KEEP; ++k)
                if (p + ln.rl + (int64_t)k * ln.RL < e)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const double d = (double)f[k][j];
                        u[j] += d;
                        v[j] += d * d;
                    }
#pragma unroll 4
            for (int64_t r = p + ln.rl + (int64_t)KEEP * ln.RL; r < e; r += ln.RL) {
                float g[VEC];
                load_vec<T, VEC>(g, x + r * a.ldx + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const double d = (double)g[j];
                    u[j] += d;
                    v[j] += d * d;
                }
            }
        }
        group_sums(a, sl, ln, u, v, s, [&](int32_t g, double x, double y) {
            float m, r;
            finish_stats(a, x, y, M, m, r);
            st[0][g - sl.g0] = m;
            st[1][g - sl.g0] = r;
            a.omean[b * a.G + g] = m;
            a.orstd[b * a.G + g] = r;
        });
        __syncthreads();
        if (on) {
            float mu[VEC], rs[VEC];
            slice_group(mu, st[0], sl, ln);
            slice_group(rs, st[1], sl, ln);
#pragma unroll
            for (int k = 0; k < KEEP; ++k) {
                const int64_t r = p + ln.rl + (int64_t)k * ln.RL;
                if (r < e) {
                    float g[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) g[j] = act_of<ACT>((f[k][j] - mu[j]) * rs[j] * gm[j] + bt[j]);
                    store_vec<T, VEC>(yp + (int64_t)k * ln.RL * a.ldy, g);
                }
            }
#pragma unroll 4
            for (int64_t r = p + ln.rl + (int64_t)KEEP * ln.RL; r < e; r += ln.RL) {
                float g[VEC];
                load_vec<T, VEC>(g, x + r * a.ldx + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = act_of<ACT>((g[j] - mu[j]) * rs[j] * gm[j] + bt[j]);
                store_vec<T, VEC>(y + r * a.ldy + ln.c, g);
            }
        }
        __syncthreads();  // st
    }
}

template <class T, int VEC, int THR, int ACT>
__global__ void __launch_bounds__(THR, THR == 256 ? 4 : 1) k_norm_bwd_seg(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                      T* __restrict__ dx)
{
    constexpr int KEEP = kKeepBwd;
    const Slice sl = slice_of(a, (int32_t)blockIdx.y);
    double* s = reinterpret_cast<double*>(norm_lds);
    float* st[2];
    st[0] = reinterpret_cast<float*>(s + sum_doubles(a.cpg, VEC, THR, true));
    st[1] = st[0] + a.sl.groups;
    const Lanes<VEC, THR> ln(a, sl);
    float gm[VEC], bt[VEC];
    if (ln.on) {
        load_chan<VEC>(gm, a.gamma, ln.c, 1.0f);
        load_chan<VEC>(bt, a.beta, ln.c, 0.0f);
    }
    Totals<VEC, THR> total{s + sum_doubles(a.cpg, VEC, THR, false)};
    total.clear();
    // consecutive segments to a block
    const int64_t each = (a.B + gridDim.x - 1) / gridDim.x, b0 = blockIdx.x * each;
    const int64_t b1 = b0 + each < a.B ? b0 + each : a.B;
    for (int64_t b = b0; b < b1; ++b) {
        const int64_t p = seg_at(a, b), e = seg_at(a, b + 1);
        if (e <= p || e - p > a.longest) continue;
        const double M = (double)(e - p) * a.cpg;
        float xh[KEEP][VEC], dz[KEEP][VEC];  // of the rows that are kept
        float mu[VEC], rs[VEC];
        double u[VEC], v[VEC], hu[VEC], hv[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[j] = v[j] = 0.0;
        const bool on = ln.on && p + ln.rl < e;
        const T *xp = x + (p + ln.rl) * a.ldx + ln.c, *dp = dy + (p + ln.rl) * a.ldy + ln.c;  // the lane's first row
        if (on) {
            load_group(mu, a.mean, a, b, ln, 1, 0);
            load_group(rs, a.rstd, a, b, ln, 1, 0);
            Raw<T, VEC> f[KEEP], d[KEEP];
#pragma unroll
            for (int k = 0; k < KEEP; ++k) {
                const bool in = p + ln.rl + (int64_t)k * ln.RL < e;
                f[k].load(xp + (in ? (int64_t)k * ln.RL * a.ldx : 0));
                d[k].load(dp + (in ? (int64_t)k * ln.RL * a.ldy : 0));
            }
#pragma unroll
            for (int k = 0; k < KEEP; ++k)
                if (p + ln.rl + (int64_t)k * ln.RL < e)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        xh[k][j] = (f[k][j] - mu[j]) * rs[j];
                        dz[k][j] = d[k][j] * act_slope<ACT>(xh[k][j] * gm[j] + bt[j]);
                        u[j] += (double)(dz[k][j] * xh[k][j]);
                        v[j] += (double)dz[k][j];
                    }
#pragma unroll 2
            for (int64_t r = p + ln.rl + (int64_t)KEEP * ln.RL; r < e; r += ln.RL) {
                Raw<T, VEC> g, h;
                g.load(x + r * a.ldx + ln.c);
                h.load(dy + r * a.ldy + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float xh = (g[j] - mu[j]) * rs[j];
                    const float dz = h[j] * act_slope<ACT>(xh * gm[j] + bt[j]);
                    u[j] += (double)(dz * xh);
                    v[j] += (double)dz;
                }
            }
        }
        total.add(u, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            hu[j] = on ? v[j] * (double)gm[j] : 0.0;
            hv[j] = on ? u[j] * (double)gm[j] : 0.0;
        }
        if (!dx) continue;
        group_sums(a, sl, ln, hu, hv, s, [&](int32_t g, double x, double y) {
            st[0][g - sl.g0] = (float)(x / M);
            st[1][g - sl.g0] = (float)(y / M);
        });
        __syncthreads();
        if (on) {
            float s1[VEC], s2[VEC];
            slice_group(s1, st[0], sl, ln);
            slice_group(s2, st[1], sl, ln);
#pragma unroll
            for (int k = 0; k < KEEP; ++k) {
                const int64_t r = p + ln.rl + (int64_t)k * ln.RL;
                if (r < e) {
                    float g[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) g[j] = dx_of(xh[k][j], dz[k][j], rs[j], gm[j], s1[j], s2[j]);
                    store_vec<T, VEC>(dx + (p + ln.rl) * a.ldd + ln.c + (int64_t)k * ln.RL * a.ldd, g);
                }
            }
#pragma unroll 2
            for (int64_t r = p + ln.rl + (int64_t)KEEP * ln.RL; r < e; r += ln.RL) {
                float g[VEC], h[VEC];
                load_vec<T, VEC>(g, x + r * a.ldx + ln.c);
                load_vec<T, VEC>(h, dy + r * a.ldy + ln.c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = dx_of<ACT>(g[j], h[j], mu[j], rs[j], gm[j], bt[j], s1[j], s2[j]);
                store_vec<T, VEC>(dx + r * a.ldd + ln.c, g);
            }
        }
        __syncthreads();  // st
    }
    if (a.chan) total.store(a, sl, ln, a.nchan - gridDim.x + blockIdx.x);
}

// ---- layout and form -----------------------------------------------------------------------
// Rows per run: about 1024 blocks over the rows (four to a compute unit, which
// is what their registers allow), at least 16 rows, so that the sums of a run are
// a small share of its rows.
int64_t rows_per_run(int64_t N)
{
    const int64_t r = cdiv64(N, 1024);
    return r < 16 ? 16 : r;
}

constexpr int64_t kSegBlocks = 1024;   // blocks of the whole segments' backward, each with one row of channel sums
constexpr int64_t kLong = 256 << 10;  // bytes of a segment's slice that one block takes
constexpr int64_t kFill = 256;        // blocks that fill the chip
// Bytes up to which ragged segments go out as whole ones alone, although one segment may hold
// all rows.  The runs beside them cost launches that mostly find nothing; without them a long
// segment is one block's work, bound by the few rows that it has in flight.  25000 x 128 in 1024
// segments, fp32, whole alone and with runs beside: of equal lengths forward 13 and 23 us,
// backward 21 and 40; one of 500 rows 30 and 43, 65 and 83; one of 2000 rows 120 and 133 (a
// block takes that one whole in either), 200 and 44; one of 8000 rows 660 and 26, 820 and 44; one of
// 24000 rows 1960 and 43, 2420 and 53.  Batches of structures of like sizes, the usual ones, are
// served; a batch with one that is a hundred times longer is quicker with that one in a call of
// its own.
constexpr int64_t kTotal = 32 << 20;

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
    w.chan = take((w.runs + kSegBlocks) * 2 * n.C * (int64_t)sizeof(double));
    w.coef = take(n.B * n.G * 2 * (int64_t)sizeof(float));
    w.bytes = o > 0 ? o : 256;  // never none, so that a workspace always has an address
    return w;
}

// at least `want` slices, if groups and whole 64-byte pieces allow
Slices slices_of(const NormShape& n, int vec, int threads, int64_t want)
{
    Slices s{};
    const int32_t cpg = n.C / n.G, most = threads * vec;
    if (cpg <= most) {
        s.parts = 1;
        int64_t groups = n.G / (want < n.G ? want : n.G);
        const int64_t least = cdiv64(64, cpg * dtype_size(n.dtype));
        if (groups < least) groups = least;
        while (groups * cpg % vec != 0 && groups < n.G) ++groups;
        if (groups > n.G) groups = n.G;
        s.groups = (int32_t)(groups * cpg <= most ? groups : most / cpg);
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

// Elements of a wide access, for either type: with eight of bf16 the sums of a
// lane's channels take so many registers that half the waves fit (backward's sums of
// 400008 x 256: 119 us where four took 100 us, before the batches that make it 96 us).
constexpr int kVec = 4;

// wide accesses need every slice to begin and end on them
bool wide_ok(const NormShape& n, int vec)
{
    if (n.C % vec != 0) return false;
    return n.C <= kThreads * vec || (n.C / n.G) % vec == 0;
}

struct NormPlan {
    NormArgs a;      // slices of the runs
    Slices seg;      // slices of the whole segments
    bool whole, runs;
    int threads;     // of the whole segments' blocks
    NormShape n;
    bool wide16;     // rows begin on 16 bytes
};

// Which forms run (the header comment says why): whole segments where their mean
// length leaves a block at most kLong bytes; beside the runs where the segments
// are ragged and all rows together exceed kTotal.  `arrays`: rows read per row.
NormPlan norm_plan(const NormShape& n, int vec, int arrays, void* ws)
{
    const NormLayout w = norm_layout(n);
    NormPlan p{};
    NormArgs& a = p.a;
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
    a.eps = n.eps;
    a.seg = n.seg;
    a.part = (double*)((char*)ws + w.part);
    a.chan = (double*)((char*)ws + w.chan);
    a.coef = (float*)((char*)ws + w.coef);
    a.sl = slices_of(n, vec, kThreads, 1);
    const int64_t mean = n.B > 0 ? cdiv64(n.N, n.B) : 0, es = dtype_size(n.dtype);
    // 1024 threads where the registers of 256 could not keep the rows and the group
    // sums fit in LDS
    p.threads = kThreads;
    p.seg = slices_of(n, vec, p.threads, n.B > 0 ? cdiv64(kFill, n.B) : 1);
    const int64_t lanes = p.seg.width / vec, keep = arrays == 1 ? kKeep<kThreads> : kKeepBwd;
    if (p.seg.parts == 1 && mean > keep * (kThreads / lanes) && a.cpg % vec == 0) p.threads = 1024;
    p.whole = p.seg.parts == 1 && mean * p.seg.width * es * arrays <= kLong;
    const bool safe = !n.seg || n.N * p.seg.width * es * arrays <= kTotal;
    p.runs = n.N > 0 && (!p.whole || !safe);
    if (!p.whole) a.longest = 0;
    else if (!p.runs) a.longest = n.N;
    else a.longest = kLong * 4 / (p.seg.width * es * arrays);
    a.nchan = (p.runs ? w.runs : 0);
    return p;
}

inline unsigned lds_bytes(const NormArgs& a, int vec, int threads, bool channels, bool groups)
{
    return (unsigned)(sum_doubles(a.cpg, vec, threads, channels) * (int)sizeof(double) + (groups ? 8 * a.sl.groups : 0));
}

inline unsigned stat_blocks(const NormArgs& a, int threads) { return grid_of(cdiv64(a.B * a.G, threads / 64)); }

template <class T, int VEC, int ACT>
hipError_t norm_fwd(const NormPlan& p, const void* x, void* y, hipStream_t s)
{
    if (p.whole) {
        NormArgs a = p.a;
        a.sl = p.seg;
        const dim3 grid(grid_of(a.B), (unsigned)a.sl.n);
        const unsigned lds = lds_bytes(a, VEC, p.threads, false, true);
        if (p.threads == 1024)
            hipLaunchKernelGGL((k_norm_seg<T, VEC, 1024, ACT>), grid, dim3(1024), lds, s, a, (const T*)x, (T*)y);
        else
            hipLaunchKernelGGL((k_norm_seg<T, VEC, kThreads, ACT>), grid, dim3(kThreads), lds, s, a, (const T*)x,
                               (T*)y);
    }
    if (p.runs || !p.whole) {
        const NormArgs& a = p.a;
        const dim3 grid(grid_of(a.runs), (unsigned)a.sl.n);
        if (a.N > 0) 
            hipLaunchKernelGGL((k_norm_sums<T, VEC>), grid, dim3(kThreads), lds_bytes(a, VEC, kThreads, false, false), s,
                               a, (const T*)x);
        hipLaunchKernelGGL(k_norm_stats, dim3(stat_blocks(a, kThreads)), dim3(kThreads), 0, s, a);
        if (a.N > 0 && p.wide16) {  // no sums to keep: the widest accesses where they fit
            NormArgs w = a;
            w.sl = slices_of(p.n, kWide<T>, kThreads, 1);
            hipLaunchKernelGGL((k_norm_apply<T, kWide<T>, ACT>), dim3(grid_of(w.runs), (unsigned)w.sl.n), dim3(kThreads), 0,
                               s, w, (const T*)x, (T*)y);
        } else if (a.N > 0) {
            hipLaunchKernelGGL((k_norm_apply<T, VEC, ACT>), grid, dim3(kThreads), 0, s, a, (const T*)x, (T*)y);
        }
    }
    return hipGetLastError();
}

template <class T, int VEC, int ACT>
hipError_t norm_bwd(NormPlan& p, const void* x, const void* dy, void* dx, float* dgamma, float* dbeta, hipStream_t s)
{
    const bool chan = dgamma || dbeta;
    NormArgs a = p.a;
    if (!dx) a.coef = nullptr;
    if (!chan) a.chan = nullptr;
    if (p.whole && a.N > 0) {
        const int64_t blocks = a.B < kSegBlocks ? a.B : kSegBlocks;
        a.nchan += blocks;
        NormArgs w = a;
        w.sl = p.seg;
        const dim3 grid((unsigned)blocks, (unsigned)w.sl.n);
        const unsigned lds = lds_bytes(w, VEC, p.threads, true, true);
        if (p.threads == 1024)
            hipLaunchKernelGGL((k_norm_bwd_seg<T, VEC, 1024, ACT>), grid, dim3(1024), lds, s, w, (const T*)x,
                               (const T*)dy, (T*)dx);
        else
            hipLaunchKernelGGL((k_norm_bwd_seg<T, VEC, kThreads, ACT>), grid, dim3(kThreads), lds, s, w, (const T*)x,
                               (const T*)dy, (T*)dx);
    }
    const dim3 grid(grid_of(a.runs), (unsigned)a.sl.n);
    if (p.runs)
        hipLaunchKernelGGL((k_norm_bwd_sums<T, VEC, ACT>), grid, dim3(kThreads), lds_bytes(a, VEC, kThreads, true, false),
                           s, a, (const T*)x, (const T*)dy);
    const unsigned cb = chan ? (unsigned)cdiv64(a.C, kChan) : 0, sb = dx && p.runs ? stat_blocks(a, kJoin) : 0;
    if (cb + sb > 0) hipLaunchKernelGGL(k_norm_bwd_join, dim3(cb + sb), dim3(kJoin), 0, s, a, (int32_t)cb, dgamma, dbeta);
    if (p.runs && dx) {
        // no sums to keep: shorter runs, and the widest accesses where they fit
        NormArgs w = a;
        w.R = cdiv64(a.R, 2);
        w.runs = cdiv64(a.N, w.R);
        if (p.wide16) w.sl = slices_of(p.n, kWide<T>, kThreads, 1);
        const dim3 g(grid_of(w.runs), (unsigned)w.sl.n);
        if (p.wide16)
            hipLaunchKernelGGL((k_norm_bwd_apply<T, kWide<T>, ACT>), g, dim3(kThreads), 0, s, w, (const T*)x,
                               (const T*)dy, (T*)dx);
        else
            hipLaunchKernelGGL((k_norm_bwd_apply<T, VEC, ACT>), g, dim3(kThreads), 0, s, w, (const T*)x,
                               (const T*)dy, (T*)dx);
    }
    return hipGetLastError();
}

// f(element type, elements of an access, activation) as constants
template <class F>
hipError_t with_form(const NormShape& n, bool wide, F&& f)
{
    auto act = [&](auto t, auto vec) {
        switch (n.act) {
            case kNone: return f(t, vec, std::integral_constant<int, kNone>{});
            case kSilu: return f(t, vec, std::integral_constant<int, kSilu>{});
            default: return f(t, vec, std::integral_constant<int, kTanh>{});
        }
    };
    if (n.dtype == kF32)
        return wide ? act(float{}, std::integral_constant<int, kVec>{}) : act(float{}, std::integral_constant<int, 1>{});
    return wide ? act(bf16_t{}, std::integral_constant<int, kVec>{})
                : act(bf16_t{}, std::integral_constant<int, 1>{});
}

}  // namespace

size_t norm_workspace_bytes(const NormShape& n, bool ragged, bool backward)
{
    if (!backward) {
        // none where whole segments take all rows, whichever accesses the arrays allow
        NormShape m = n;
        int32_t some = 0;
        m.seg = ragged ? &some : nullptr;  // only whether there are offsets matters to the plan
        if (!norm_plan(m, 1, 1, nullptr).runs && (!wide_ok(m, kVec) || !norm_plan(m, kVec, 1, nullptr).runs)) return 0;
    }
    return norm_layout(n).bytes;
}

hipError_t launch_norm_fwd(const NormShape& n, const void* x, const float* gamma, const float* beta, void* y,
                           float* mean, float* rstd, void* ws, hipStream_t s)
{
    if (n.B == 0) return hipSuccess;
    const int64_t es = dtype_size(n.dtype);
    const bool wide = wide_ok(n, kVec) && aligned_rows(x, n.ldx, es, kVec * es) && aligned_rows(y, n.ldy, es, kVec * es);
    NormPlan p = norm_plan(n, wide ? kVec : 1, 1, ws);
    p.a.gamma = gamma;
    p.a.beta = beta;
    p.n = n;
    p.wide16 = wide_ok(n, (int)(16 / es)) && aligned_rows(x, n.ldx, es) && aligned_rows(y, n.ldy, es);
    p.a.omean = mean;
    p.a.orstd = rstd;
    return with_form(n, wide, [&](auto t, auto v, auto act) {
        return norm_fwd<decltype(t), decltype(v)::value, decltype(act)::value>(p, x, y, s);
    });
}

hipError_t launch_norm_bwd(const NormShape& n, const void* x, const float* mean, const float* rstd,
                           const float* gamma, const float* beta, const void* dy, void* dx, float* dgamma,
                           float* dbeta, void* ws, hipStream_t s)
{
    const int64_t es = dtype_size(n.dtype);
    const bool wide = wide_ok(n, kVec) && aligned_rows(x, n.ldx, es, kVec * es) &&
                      aligned_rows(dy, n.ldy, es, kVec * es) && (!dx || aligned_rows(dx, n.ldd, es, kVec * es));
    NormPlan p = norm_plan(n, wide ? kVec : 1, 2, ws);
    p.a.mean = mean;
    p.a.rstd = rstd;
    p.a.gamma = gamma;
    p.a.beta = beta;
    p.n = n;
    p.wide16 = wide_ok(n, (int)(16 / es)) && aligned_rows(x, n.ldx, es) && aligned_rows(dy, n.ldy, es) &&
               (!dx || aligned_rows(dx, n.ldd, es));
    return with_form(n, wide, [&](auto t, auto v, auto act) {
        return norm_bwd<decltype(t), decltype(v)::value, decltype(act)::value>(p, x, dy, dx, dgamma, dbeta, s);
    });
}

}  // namespace cgtp
