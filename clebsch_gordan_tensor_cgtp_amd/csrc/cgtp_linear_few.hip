// cgtp_linear_few.hip -- y for few rows: one pass over W on the vector units.
//
// A block of 1024 threads takes 32 columns and the whole contraction: four lanes lie along
// a row of W (eight columns each), the others and the 16 waves along k; each thread's sums
// of its k go through the wave and then through LDS in a fixed order, all in fp32.  What bounds it
// is one pass over W, and at these sizes the latency of its loads and of the launch: 1 x 1024 x 4096
// bf16 4.3 us in a graph with SiLU (8.4 MB of W, 1.2 us of memory), 4 rows 5.9.  The contraction is not cut: a
// deep one over few columns leaves compute units idle (4 x 4096 x 1024 fp32 10.1, on 32 of them).  Sums that halve
// the columns from step to step (eight exchanges for eight columns) instead of whole ones (32): 5.9 us
// before.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "cgtp_linear.h"
#include "cgtp_linear_wide.h"

namespace cgtp {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kL = 4;                        // lanes along a row of W
constexpr int kRun = kThreads / kL;          // k of one load of all threads
constexpr int kAhead = 4;                    // loads of a thread under way
constexpr int kChunk = kRun * kAhead;

template <class T, int R, bool VEC>
__global__ void __launch_bounds__(kThreads) k_linear_few(GemmArgs a)
{
    constexpr int kCols = kL * 8;
    __shared__ float sums[kWaves][R][kCols];
    __shared__ __attribute__((aligned(16))) float total[R][kCols];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = tid % kL;
    const int64_t r0 = (int64_t)blockIdx.y * R, c = ((int64_t)blockIdx.x * kL + l) * 8;
    const int w = c >= a.cols ? 0 : a.cols - c < 8 ? (int)(a.cols - c) : 8;
    float acc[R][8] = {};
    for (int64_t k0 = 0; k0 < a.depth; k0 += kChunk) {
        Raw8<T> raw[kAhead];
        T x[kAhead][R];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t k = k0 + i * kRun + tid / kL;
            const bool in = k < a.depth && w > 0;
            const T* p = (const T*)a.B + (in ? k * a.ldb + c : 0);
            if constexpr (VEC) {
                raw[i].load(p);
                if (!in) raw[i].clear();
            } else {
                raw[i].load_some(p, in ? w : 0);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                // (outside: any value, its products are not kept or have a zero of W)
                const int64_t n = r0 + r < a.rows ? r0 + r : a.rows - 1;
                x[i][r] = ((const T*)a.A)[n * a.lda + (k < a.depth ? k : 0)];
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const bool in = k0 + i * kRun + tid / kL < a.depth;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float v = in ? to_f32(x[i][r]) : 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[r][j] = fmaf(v, raw[i][j], acc[r][j]);
            }
        }
    }
    // The wave's sixteen threads of each eight columns: at every step a thread gives half of its
    // columns away and adds the other half of its partner's, until one column is left, then that.
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int h = 4, d = kL; h > 0; h /= 2, d *= 2) {
            const bool up = lane & d;
#pragma unroll
            for (int j = 0; j < h; ++j) {
                const float give = up ? acc[r][j] : acc[r][j + h], keep = up ? acc[r][j + h] : acc[r][j];
                acc[r][j] = keep + __shfl_xor(give, d, 64);
            }
        }
        acc[r][0] += __shfl_xor(acc[r][0], 32, 64);
        if (lane < 32) {
            // the halves taken: column 4 (lane / 4 % 2) + 2 (lane / 8 % 2) + lane / 16 % 2
            const int j = 4 * (lane >> 2 & 1) + 2 * (lane >> 3 & 1) + (lane >> 4 & 1);
            sums[wave][r][l * 8 + j] = acc[r][0];
        }
    }
    __syncthreads();
    if (tid < R * kCols) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) t += sums[i][tid / kCols][tid % kCols];
        total[tid / kCols][tid % kCols] = t;
    }
    __syncthreads();
    const int r = tid / kL;
    if (r >= R || r0 + r >= a.rows || w == 0) return;
    float v[1][8], bias[8];
    bias8<VEC>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[0][j] = total[r][l * 8 + j];
    finish8<T, kFwd, VEC, 1>(a, drop_offset(a.drop), v, bias, {r0 + r}, {true}, c, w);
}

template <class T, bool VEC>
void launch(const GemmArgs& a, hipStream_t s)
{
    const int64_t slabs = cdiv64(a.cols, kL * 8);
    auto go = [&](auto kernel, int rows) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)slabs, (unsigned)cdiv64(a.rows, rows)), dim3(kThreads), 0, s, a);
    };
    if (a.rows == 1) go(k_linear_few<T, 1, VEC>, 1);
    else if (a.rows == 2) go(k_linear_few<T, 2, VEC>, 2);
    else go(k_linear_few<T, 4, VEC>, 4);
}

}  // namespace

hipError_t launch_linear_few(int dtype, bool vec, const GemmArgs& a, hipStream_t s)
{
    if (dtype == kF32) vec ? launch<float, true>(a, s) : launch<float, false>(a, s);
    else vec ? launch<bf16_t, true>(a, s) : launch<bf16_t, false>(a, s);
    return hipGetLastError();
}

}  // namespace cgtp
