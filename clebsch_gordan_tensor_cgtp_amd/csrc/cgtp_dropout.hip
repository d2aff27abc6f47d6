// cgtp_dropout.hip -- dropout of rows by a counter-based generator, with an
// optional residual: out = r + (keep ? x / (1 - p) : 0), on gradients as on values.
//
// One pass over x (and r), eight channels per thread and step: one block of the
// generator (cgtp_drop.h) decides them.  Bound by memory: 400008 x 256 fp32 with a residual
// 203 us (6.0 TB/s, where a plain copy of that size reaches 5.2); 16385 x 1024 bf16 12.0 us
// (5.6 TB/s), where the generator's products take some 9 us of the vector units; 2000 x 128
// 2.6 us, a launch.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "cgtp_drop.h"
#include "cgtp_internal.h"
#include "cgtp_train_internal.h"
#include "cgtp_vec.h"

namespace cgtp {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 16;  // the kernels stride over what is left

struct DropArgs {
    int64_t N, ldx, ldr, ldo;
    int32_t C, per;     // channels, blocks of eight to a row
    int64_t rows, step; // rows and blocks that a stride of the grid goes on by
    Drop d;
    const void *x, *r;
    void* out;
};

// Threads go through the blocks of eight channels row by row.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_dropout(DropArgs a)
{
    const uint64_t offset = drop_offset(a.d);
    const T* x = (const T*)a.x;
    const T* r = (const T*)a.r;
    T* out = (T*)a.out;
    const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    int64_t n = first / a.per;
    int32_t q = (int32_t)(first - n * a.per);
    while (n < a.N) {
        const int32_t c = q * 8;
        const int w = VEC || a.C - c >= 8 ? 8 : a.C - c;
        Raw8<T> v, s;
        v.load_some(x + n * a.ldx + c, w);
        s.load_some(r + n * a.ldr + c, r ? w : 0);
        const Drawn f = philox((uint32_t)q, (uint32_t)n, offset, a.d.seed);
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float k = f[j] >= a.d.thr ? v[j] * a.d.scale : 0.0f;
            t[j] = r ? s[j] + k : k;
        }
        store8<T>(out + n * a.ldo + c, t, w);
        q += (int32_t)a.step;
        n += a.rows;
        if (q >= a.per) {
            q -= a.per;
            ++n;
        }
    }
}

template <class T>
hipError_t launch(const DropShape& d, const void* x, const void* r, void* out, hipStream_t s)
{
    DropArgs a{};
    a.N = d.N;
    a.C = (int32_t)d.C;
    a.ldx = d.ldx;
    a.ldr = d.ldr;
    a.ldo = d.ldo;
    a.per = (int32_t)((d.C + 7) / 8);
    a.d = d.drop;
    a.x = x;
    a.r = r;
    a.out = out;
    int64_t blocks = (d.N * a.per + kThreads - 1) / kThreads;
    blocks = blocks < kMaxBlocks ? blocks : kMaxBlocks;
    a.rows = blocks * kThreads / a.per;
    a.step = blocks * kThreads % a.per;
    const bool vec = d.C % 8 == 0 && aligned_rows(x, d.ldx, sizeof(T)) && aligned_rows(out, d.ldo, sizeof(T)) &&
                     (!r || aligned_rows(r, d.ldr, sizeof(T)));
    if (vec) hipLaunchKernelGGL((k_dropout<T, true>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_dropout<T, false>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropShape& d, const void* x, const void* residual, void* out, hipStream_t s)
{
    if (d.N == 0) return hipSuccess;
    return d.dtype == kF32 ? launch<float>(d, x, residual, out, s) : launch<bf16_t>(d, x, residual, out, s);
}

}  // namespace cgtp
