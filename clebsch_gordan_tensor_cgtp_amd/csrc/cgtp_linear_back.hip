// cgtp_linear_back.hip -- the gradients of narrow products in one pass: dz = mask g act'(z) is
// formed once for
//   dx = dz W^T  (up to 128 outputs),  dW = x^T dz,  db = sum of dz's rows.
//
// Memory bounds these: g, z and x are read and dx is written once.  A block owns a KT x MT slab of
// W and goes through chunks of 64 (or 32) rows, one of every `splits`: dz and x go through registers
// (fetched while the chunk before is multiplied) into LDS as they lie in memory, as bf16 planes (three of
// dz with a slope, whatever the type).  dz is
// read along its rows for dx, whose other operand, the slab of W, each wave has cut once and keeps in
// registers; dz and x are read across their rows (by the transposing LDS read) for dW, whose sums stay
// in registers to the end and leave as one partial sum to a block, added in order by a launch of its own.
// 400000 x 128 x 128 with tanh: fp32 271 us (3.0 TB/s: the twelve products of dx and dW take 126 us at the rate
// of a large library product, cutting and slopes as much of the vector units again), bf16 151; without a slope 207
// and 67 (4.6 TB/s).  25000 x 128 x 128 bf16 with tanh 22.9 + 5.7, of which the parts (256 of 64 KB, written
// and read) are 33 MB against the arrays' 25; 2000 x 128 x 128 fp32 with SiLU 12.2 + 4.2.  By tiles, three
// launches each, these two take 37 and 28 us in all.  Slabs of 128 x 128 fp32 in chunks of 64 rows have 24
// registers more than there are: those go through scratch memory in every chunk.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "cgtp_linear.h"
#include "cgtp_linear_wide.h"

namespace cgtp {
namespace {

template <int KT, int MT>
constexpr int kBackThreads = KT + MT > 128 ? 512 : 256;

// kRows: of a chunk.  VEC: rows of whole blocks of eight on 16 bytes.
template <class T, int KT, int MT, int kRows, bool VEC, bool HZ>
__global__ void __launch_bounds__((kBackThreads<KT, MT>))
k_linear_back(GemmArgs a, const T* __restrict__ W, T* __restrict__ dx, int64_t ldd)
{
    constexpr int kThr = kBackThreads<KT, MT>, NW = kThr / 64, NP = kPlanes<T>, NZ = kSlopePlanes<T, HZ>;
    constexpr int kLdX = KT + 16, kLdZ = MT + 16, kPlaneX = kRows * kLdX, kPlaneZ = kRows * kLdZ;  // halves
    constexpr int kPerX = KT / 8, kPerZ = MT / 8, kAllX = kRows * kPerX, kAllZ = kRows * kPerZ;
    constexpr int kEachX = (kAllX + kThr - 1) / kThr, kEachZ = (kAllZ + kThr - 1) / kThr;
    // dW: waves along the outputs WQ, each FP x 1 tiles of 32
    constexpr int WQ = MT / 32, WP = NW / WQ, FP = KT / 32 / WP;
    static_assert(WP * FP * 32 == KT, "waves cover the slab");
    // dx: tiles of 32 rows by 32 inputs, a wave each
    constexpr int kMsteps = MT / 16;
    constexpr int kLdS = 36;
    constexpr int kTiles = (kPlaneX * NP + kPlaneZ * NZ) * 2, kSums = kThr * 64, kPatch = NW * 32 * kLdS * 4;
    __shared__ __attribute__((aligned(16))) char mem[kTiles + kPatch > kSums ? kTiles + kPatch : kSums];
    uint16_t* sx = reinterpret_cast<uint16_t*>(mem);
    uint16_t* sz = sx + kPlaneX * NP;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // a.tr slabs along the inputs, a.splits blocks to a slab
    const int64_t at = xcd_order(blockIdx.x, gridDim.x);
    const int64_t part = at / a.tr, i0 = at % a.tr * KT;
    const uint64_t offset = drop_offset(a.drop);

    // chunk's rows, zero outside
    Raw8<T> rx[kEachX], rg[kEachZ], rz[HZ ? kEachZ : 1];
    auto fetch = [&](int64_t n0) {
        auto load = [&](Raw8<T>& r, const void* base, int64_t ld, int64_t n, int64_t e, int64_t lim) {
            const bool in = n < a.depth && e < lim;
            const T* p = (const T*)base + (in ? n * ld + e : 0);
            if constexpr (VEC) {
                r.load(p);
                if (!in) r.clear();
            } else {
                r.load_some(p, !in ? 0 : lim - e < 8 ? (int)(lim - e) : 8);
            }
        };
#pragma unroll
        for (int i = 0; i < kEachZ; ++i) {
            const int b = tid + i * kThr;
            if (kAllZ < kThr && b >= kAllZ) break;
            load(rg[i], a.B, a.ldb, n0 + b / kPerZ, b % kPerZ * 8, a.cols);
            if (HZ && a.Z) load(rz[HZ ? i : 0], a.Z, a.ldz, n0 + b / kPerZ, b % kPerZ * 8, a.cols);
        }
        if (a.want) {
#pragma unroll
            for (int i = 0; i < kEachX; ++i) {
                const int b = tid + i * kThr;
                if (kAllX < kThr && b >= kAllX) break;
                load(rx[i], a.A, a.lda, n0 + b / kPerX, i0 + b % kPerX * 8, a.rows);
            }
        }
    };
    fetch(part * kRows);

    // this wave's 32 inputs of the slab of W, all outputs
    const int wr = wave % (kRows / 32) * 32, wi = wave / (kRows / 32) * 32;
    const bool to_dx = wi < KT && dx;
    b8 w[kMsteps][NP];
    {
        if (to_dx) {
            const int64_t ci = i0 + wi + (lane & 31);
#pragma unroll
            for (int s = 0; s < kMsteps; ++s) {
                const int64_t e = 16 * s + 8 * (lane >> 5);
                const bool in = ci < a.rows && e < a.cols;
                const T* p = W + (in ? ci * a.cols + e : 0);
                Raw8<T> r;
                if constexpr (VEC) {
                    r.load(p);
                    if (!in) r.clear();
                } else {
                    r.load_some(p, !in ? 0 : a.cols - e < 8 ? (int)(a.cols - e) : 8);
                }
                f8 v;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r[j];
                cut_along(v, w[s]);
            }
        }
    }

    f16v acc[FP];
#pragma unroll
    for (int x = 0; x < FP; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[x][e] = 0.0f;
    double sum[8] = {};
    const bool sums = a.db && i0 == 0;
    const int wp = wave / WQ * (32 * FP), wq = wave % WQ * 32, l = lane & 15;
    const uint16_t* px = sx + (8 * (lane >> 5) + l / 4) * kLdX + wp + (lane & 16) + 4 * (l % 4);
    const uint16_t* pz = sz + (8 * (lane >> 5) + l / 4) * kLdZ + wq + (lane & 16) + 4 * (l % 4);
    float* s = reinterpret_cast<float*>(mem + kTiles) + wave * (32 * kLdS);

    for (int64_t n0 = part * kRows; n0 < a.depth; n0 += a.splits * kRows) {
        if (n0 != part * kRows) __syncthreads();
        auto put = [&](uint16_t* to, int plane, const f8& v, auto planes) {
            constexpr int N = decltype(planes)::value;
            b8 p[N];
            cut(v, p);
#pragma unroll
            for (int i = 0; i < N; ++i) *reinterpret_cast<b8*>(to + i * plane) = p[i];
        };
#pragma unroll
        for (int i = 0; i < kEachZ; ++i) {
            const int b = tid + i * kThr, row = b / kPerZ, col = b % kPerZ * 8;
            if (kAllZ < kThr && b >= kAllZ) break;
            f8 v;
            float z[8] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = rg[i][j];
            if (HZ && a.Z) {
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = rz[HZ ? i : 0][j];
            }
            slope8<HZ>(a, offset, v, z, n0 + row, col / 8);
            if (sums) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += (double)v[j];
            }
            put(sz + row * kLdZ + col, kPlaneZ, v, std::integral_constant<int, NZ>{});
        }
        if (a.want) {
#pragma unroll
            for (int i = 0; i < kEachX; ++i) {
                const int b = tid + i * kThr;
                if (kAllX < kThr && b >= kAllX) break;
                f8 v;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = rx[i][j];
                put(sx + b / kPerX * kLdX + b % kPerX * 8, kPlaneX, v, std::integral_constant<int, NP>{});
            }
        }
        __syncthreads();
        if (n0 + a.splits * kRows < a.depth) fetch(n0 + a.splits * kRows);
        if (a.want) {
#pragma unroll
            for (int k = 0; k < kRows; k += 16) {
                b8 q[NZ], p[FP][NP];
#pragma unroll
                for (int o = NZ - 1; o >= 0; --o) q[o] = read_across(pz + o * kPlaneZ + k * kLdZ, kLdZ);
#pragma unroll
                for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                    for (int x = 0; x < FP; ++x) p[x][o] = read_across(px + o * kPlaneX + k * kLdX + 32 * x, kLdX);
                each_product<NP, NZ>([&](int i, int j) {
#pragma unroll
                    for (int x = 0; x < FP; ++x)
                        acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[j], p[x][i], acc[x], 0, 0, 0);
                });
            }
        }
        {
            if (to_dx) {
                f16v d;
#pragma unroll
                for (int e = 0; e < 16; ++e) d[e] = 0.0f;
                const uint16_t* pa = sz + (wr + (lane & 31)) * kLdZ + 8 * (lane >> 5);
#pragma unroll
                for (int k = 0; k < kMsteps; ++k) {
                    b8 p[NZ];
#pragma unroll
                    for (int o = NZ - 1; o >= 0; --o) p[o] = *reinterpret_cast<const b8*>(pa + o * kPlaneZ + 16 * k);
                    each_product<NZ, NP>(
                        [&](int i, int j) { d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[k][j], p[i], d, 0, 0, 0); });
                }
                // a lane holds row lane % 32, inputs 8 g + 4 (lane / 32) + 0 .. 3
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 v{d[4 * g], d[4 * g + 1], d[4 * g + 2], d[4 * g + 3]};
                    *reinterpret_cast<float4*>(&s[(lane & 31) * kLdS + 8 * g + 4 * (lane >> 5)]) = v;
                }
                __builtin_amdgcn_wave_barrier();
                const int64_t c = i0 + wi + lane % 4 * 8;
                const int width = c >= a.rows ? 0 : a.rows - c < 8 ? (int)(a.rows - c) : 8;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int row = 16 * g + lane / 4;
                    const int64_t n = n0 + wr + row;
                    if (n >= a.depth || width == 0) continue;
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = s[row * kLdS + lane % 4 * 8 + j] * a.drop.scale;
                    store8<T>(dx + n * ldd + c, v, VEC ? 8 : width);
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
    }

    if (a.want) {
        // rows lane % 32 of the tile, outputs 8 g + 4 (lane / 32) + 0 .. 3
#pragma unroll
        for (int x = 0; x < FP; ++x) {
            const int64_t i = i0 + wp + 32 * x + (lane & 31);
            if (i >= a.rows) continue;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int64_t c = wq + 8 * g + 4 * (lane >> 5);
                float* p = a.part + (part * a.rows + i) * a.cols + c;
                if (c + 4 <= a.cols) {
                    const float4 v{acc[x][4 * g], acc[x][4 * g + 1], acc[x][4 * g + 2], acc[x][4 * g + 3]};
                    store16(p, __builtin_bit_cast(uint4, v));
                } else {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (c + e < a.cols) p[e] = acc[x][4 * g + e];
                }
            }
        }
    }
    if (sums) {
        double* sd = reinterpret_cast<double*>(mem);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) sd[j * kThr + tid] = sum[j];
        __syncthreads();
        if (tid < MT && tid < a.cols) {
            double t = 0.0;
            for (int i = 0; i < kThr / kPerZ; ++i) t += sd[tid % 8 * kThr + i * kPerZ + tid / 8];
            a.db_part[part * a.cols + tid] = t;
        }
    }
}

template <class T, int KT, int MT, int R>
void launch(bool vec, const GemmArgs& a, const void* W, void* dx, int64_t ldd, hipStream_t s)
{
    const dim3 grid((unsigned)(a.tr * a.splits)), block(kBackThreads<KT, MT>);
    auto go = [&](auto z) {
        constexpr bool HZ = decltype(z)::value;
        if (vec) hipLaunchKernelGGL((k_linear_back<T, KT, MT, R, true, HZ>), grid, block, 0, s, a, (const T*)W, (T*)dx, ldd);
        else hipLaunchKernelGGL((k_linear_back<T, KT, MT, R, false, HZ>), grid, block, 0, s, a, (const T*)W, (T*)dx, ldd);
    };
    // (fp32 rows have three planes either way)
    if (kPlanes<T> == 3 || a.Z) go(std::true_type{});
    else if constexpr (kPlanes<T> == 1) go(std::false_type{});
}

template <class T, int R>
void launch(bool vec, const GemmArgs& a, const BackPlan& p, const void* W, void* dx, int64_t ldd, hipStream_t s)
{
    if (p.kt == 128 && p.mt == 128) launch<T, 128, 128, R>(vec, a, W, dx, ldd, s);
    else if (p.kt == 128) launch<T, 128, 64, R>(vec, a, W, dx, ldd, s);
    else if (p.mt == 128) launch<T, 64, 128, R>(vec, a, W, dx, ldd, s);
    else launch<T, 64, 64, R>(vec, a, W, dx, ldd, s);
}

template <class T>
void launch(bool vec, const GemmArgs& a, const BackPlan& p, const void* W, void* dx, int64_t ldd, hipStream_t s)
{
    if (p.rows == 32) launch<T, 32>(vec, a, p, W, dx, ldd, s);
    else launch<T, 64>(vec, a, p, W, dx, ldd, s);
}

}  // namespace

BackPlan back_plan(int64_t n, int64_t k, int64_t m)
{
    BackPlan p{};
    p.kt = k <= 64 ? 64 : 128;
    p.mt = m <= 64 ? 64 : 128;
    p.tr = cdiv64(k, p.kt);
    // Half chunks where whole ones would leave compute units idle: what a block forms and multiplies
    // one after the other is then half as long.
    p.rows = p.tr * cdiv64(n, 64) <= 64 ? 32 : 64;
    // a block to a compute unit (two of the smallest), every one with a chunk at least
    const int64_t chunks = cdiv64(n, p.rows), fill = cdiv64(p.kt + p.mt > 128 ? 256 : 512, p.tr);
    p.splits = chunks < fill ? chunks : fill;
    p.splits = p.splits < 1 ? 1 : p.splits;
    return p;
}

hipError_t launch_linear_back(int dtype, bool vec, const GemmArgs& a, const BackPlan& p, const void* W, void* dx,
                              int64_t ldd, hipStream_t s)
{
    if (dtype == kF32) launch<float>(vec, a, p, W, dx, ldd, s);
    else launch<bf16_t>(vec, a, p, W, dx, ldd, s);
    return hipGetLastError();
}

}  // namespace cgtp
