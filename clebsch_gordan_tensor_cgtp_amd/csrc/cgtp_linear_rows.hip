// cgtp_linear_rows.hip -- y of rows that registers hold whole (up to 128 inputs).
//
// Memory bounds these products: x is read and y written once.  Each wave loads its 32 rows
// of x straight into matrix operands, cuts them once and keeps them, and goes through the columns of
// W, which the block's four waves share: a tile of kCols columns goes through registers (fetched while the
// tile before is multiplied) into LDS as it lies in memory and is read by the transposing LDS read.
// A wave's results leave through a patch of LDS of its own, 32 rows of 32 columns at a time.
// 105730 x 64 x 1920 fp32 217 to 232 us, median 224, with the clock settled (3.7 TB/s; up to 305 in the first
// ten milliseconds of load, while the clock swings; with SiLU and z kept 333, 5.0 TB/s: the six products, 125 us at
// the rate of a large library product, hide behind the stores only in part), bf16 95; 105730 x 8 x 64 fp32
// 14.8; 2000 x 128 x 128 fp32 8.2, mostly one block's chain.  By tiles (cgtp_linear.hip), which cut x again for
// every tile of columns, the first takes 264 to 279 under the same conditions, the second 20, the third 7.2
// (7.7 here, both from a graph).  The form for 128 fp32 inputs whose rows or columns end inside has 8
// registers more than there are.
// WR waves lie along the rows, 4 / WR along the columns.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "cgtp_linear.h"
#include "cgtp_linear_wide.h"

namespace cgtp {
namespace {

constexpr int kThreads = 256, kCols = 64;

// every wave of the block is here and its LDS accesses are done (global ones may be under way)
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// NK: steps of 16 inputs
template <class T, int NK, int WR, bool VEC>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(NK * kPlanes<T> >= 8 ? 2 : 3)))
k_linear_rows(GemmArgs a)
{
    constexpr int NP = kPlanes<T>, WC = 4 / WR, FN = kCols / 32 / WC, kK = NK * 16;
    constexpr int kLd = kCols + 16, kPlane = kK * kLd;  // halves
    constexpr int kPer = kCols / 8, kBlocks = kK * kPer, kEach = (kBlocks + kThreads - 1) / kThreads;
    constexpr int kLdS = 36;
    __shared__ __attribute__((aligned(16))) uint16_t sw[NP * kPlane];
    __shared__ __attribute__((aligned(16))) float patch[4][32 * kLdS];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t at = xcd_order(blockIdx.x, gridDim.x);
    const int64_t r0 = at / a.tc * (32 * WR) + wave / WC * 32;  // a.tc: stretches of columns, a.run: their length
    const int64_t c0 = at % a.tc * a.run, c1 = c0 + a.run < a.cols ? c0 + a.run : a.cols;
    const uint64_t offset = drop_offset(a.drop);

    // W's tile from column c on.  The loads stand outside any condition (outside W at its first
    // element): what is outside becomes zero where it goes to LDS.
    Raw8<T> raw[kEach];
    auto inside = [&](int i, int64_t c, int64_t& k, int64_t& e) {
        const int b = tid + i * kThreads;
        k = b / kPer;
        e = c + b % kPer * 8;
        return k < a.depth && e < c1;
    };
    auto fetch = [&](int64_t c) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            int64_t k, e;
            const bool in = inside(i, c, k, e);
            const T* p = (const T*)a.B + (in ? k * a.ldb + e : 0);
            if constexpr (VEC) raw[i].load(p);
            else raw[i].load_some(p, !in ? 0 : c1 - e < 8 ? (int)(c1 - e) : 8);
        }
    };
    fetch(c0);
    // x: row lane % 32, inputs 16 s + 8 (lane / 32) + 0 .. 7
    b8 x[NK][NP];
    {
        const int64_t n = r0 + (lane & 31) < a.rows ? r0 + (lane & 31) : a.rows - 1;
        const T* p = (const T*)a.A + n * a.lda;
        Raw8<T> r[NK];
#pragma unroll
        for (int s = 0; s < NK; ++s) {
            const int k = 16 * s + 8 * (lane >> 5);
            if constexpr (VEC) {
                r[s].load(p + (k < a.depth ? k : 0));
                if (k >= a.depth) r[s].clear();
            } else {
                r[s].load_some(p + k, a.depth - k < 8 ? (int)(a.depth - k) : 8);
            }
        }
#pragma unroll
        for (int s = 0; s < NK; ++s) {
            if constexpr (NP > 1) {
                f8 v;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r[s][j];
                cut_along(v, x[s]);
            } else {
                x[s][0] = __builtin_bit_cast(b8, r[s].v[0]);
            }
        }
    }

    const int l = lane & 15;
    const uint16_t* sr = sw + (8 * (lane >> 5) + l / 4) * kLd + wave % WC * (32 * FN) + (lane & 16) + 4 * (l % 4);
    float* s = patch[wave];
    // FULL: no row, column or input is outside, so that no wait has to reckon with stores that
    // are skipped (it would wait for all of them)
    auto columns = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        for (int64_t c = c0; c < c1; c += kCols) {
            if (c != c0) lds_barrier();  // the tile before has been read
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int b = tid + i * kThreads;
                if (kBlocks % kThreads != 0 && b >= kBlocks) break;
                int64_t k, e;
                const bool in = FULL || inside(i, c, k, e);
                b8 planes[NP];
                if constexpr (NP > 1) {
                    f8 v;
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = in ? raw[i][j] : 0.0f;
                    cut(v, planes);
                } else {
                    uint4 v = raw[i].v[0];
                    if (!in) v = uint4{0, 0, 0, 0};
                    planes[0] = __builtin_bit_cast(b8, v);
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) *reinterpret_cast<b8*>(sw + p * kPlane + b / kPer * kLd + b % kPer * 8) = planes[p];
            }
            lds_barrier();
            // this lane's eight columns of each 32 that leave
            const int64_t ce = c + wave % WC * (32 * FN) + lane % 4 * 8;
            auto width = [&](int y) {
                const int64_t e = ce + 32 * y;
                return FULL ? 8 : e >= c1 ? 0 : c1 - e < 8 ? (int)(c1 - e) : 8;
            };
            float bias[FN][8];
#pragma unroll
            for (int y = 0; y < FN; ++y) bias8<FULL>(a, ce + 32 * y, width(y), bias[y]);
            if (c + kCols < c1) fetch(c + kCols);
            f16v acc[FN];
#pragma unroll
            for (int y = 0; y < FN; ++y)
#pragma unroll
                for (int q = 0; q < 16; ++q) acc[y][q] = 0.0f;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                b8 w[FN][NP];
#pragma unroll
                for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                    for (int y = 0; y < FN; ++y) w[y][p] = read_across(sr + p * kPlane + k * 16 * kLd + 32 * y, kLd);
#pragma unroll
                for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                    for (int p = 0; p <= o; ++p)
#pragma unroll
                        for (int y = 0; y < FN; ++y)
                            acc[y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[y][o - p], x[k][p], acc[y], 0, 0, 0);
            }
            // a lane holds row lane % 32, columns 8 g + 4 (lane / 32) + 0 .. 3
#pragma unroll
            for (int y = 0; y < FN; ++y) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 v{acc[y][4 * g], acc[y][4 * g + 1], acc[y][4 * g + 2], acc[y][4 * g + 3]};
                    *reinterpret_cast<float4*>(&s[(lane & 31) * kLdS + 8 * g + 4 * (lane >> 5)]) = v;
                }
                __builtin_amdgcn_wave_barrier();
                float v[2][8];
                int64_t n[2];
                bool on[2];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int row = 16 * g + lane / 4;
                    n[g] = r0 + row;
                    on[g] = FULL || (n[g] < a.rows && width(y) > 0);
#pragma unroll
                    for (int j = 0; j < 8; j += 4)
                        *reinterpret_cast<float4*>(&v[g][j]) = *reinterpret_cast<const float4*>(&s[row * kLdS + lane % 4 * 8 + j]);
                }
                finish8<T, kFwd, VEC, 2>(a, offset, v, bias[y], n, on, ce + 32 * y, width(y));
                __builtin_amdgcn_wave_barrier();
            }
        }
    };
    // (the same for all waves: they share barriers)
    if (VEC && a.depth == kK && at / a.tc * (32 * WR) + 32 * WR <= a.rows && (c1 - c0) % kCols == 0) columns(std::true_type{});
    else columns(std::false_type{});
}

template <class T, int NK, bool VEC>
void launch(GemmArgs& a, hipStream_t s)
{
    // All four waves along the rows where their blocks fill the chip (50000 x 128 x 128 bf16 13.0 us, two along
    // the columns 16.9; 20000 x 128 x 1024 23 and 30), with very few inputs, whose blocks are short,
    // where they do so twice (105730 x 8 x 64 fp32 15.8 and 14.5, x 16 x 128 23 and 25), and with 128 fp32 inputs
    // never: their registers would spill (50000 x 128 x 128 35.7 and 31.5).  Stretches of columns for some
    // 2048 blocks: what a block has cut of x serves a whole stretch.
    const int64_t tiles = cdiv64(a.cols, kCols);
    constexpr bool kTall = NK * kPlanes<T> <= 12;
    const bool tall = kTall && cdiv64(a.rows, 128) * tiles >= (NK == 1 ? 1536 : 768);
    a.tr = cdiv64(a.rows, tall ? 128 : 64);
    int64_t n = cdiv64(2048, a.tr);
    n = n < tiles ? n : tiles;
    a.run = cdiv64(tiles, n) * kCols;
    a.tc = cdiv64(a.cols, a.run);
    const dim3 grid((unsigned)(a.tr * a.tc));
    if (tall) hipLaunchKernelGGL((k_linear_rows<T, NK, kTall ? 4 : 2, VEC>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_linear_rows<T, NK, 2, VEC>), grid, dim3(kThreads), 0, s, a);
}

template <class T, bool VEC>
void launch(GemmArgs& a, hipStream_t s)
{
    if (a.depth <= 16) launch<T, 1, VEC>(a, s);
    else if (a.depth <= 32) launch<T, 2, VEC>(a, s);
    else if (a.depth <= 64) launch<T, 4, VEC>(a, s);
    else launch<T, 8, VEC>(a, s);
}

}  // namespace

hipError_t launch_linear_rows(int dtype, bool vec, GemmArgs a, hipStream_t s)
{
    if (dtype == kF32) vec ? launch<float, true>(a, s) : launch<float, false>(a, s);
    else vec ? launch<bf16_t, true>(a, s) : launch<bf16_t, false>(a, s);
    return hipGetLastError();
}

}  // namespace cgtp
