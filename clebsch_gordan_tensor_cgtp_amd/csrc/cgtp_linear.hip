// cgtp_linear.hip -- the product of rows with a weight matrix, with bias, activation,
// dropout and residual in its epilogue, and its gradients, on the bf16 matrix cores:
//
//   z = x W + b,  y = r + drop(act(z))                  [N][K] times [K][M]
//   dz = drop(g) act'(z),  dx = dz W^T,  dW = x^T dz,  db = sum of dz's rows
//
// Precision.  An fp32 operand v is cut into three bf16 numbers, h = bf16(v),
// m = bf16(v - h), l = bf16(v - h - m), which together hold all 24 bits of every
// value of 2^-102 or more (bf16 has fp32's range, so no units are needed; the matrix
// instructions take remainders below 2^-126 as zero), and
//   u v = hu hv + (hu mv + mu hv) + (hu lv + mu mv + lu hv)
// leaves out terms of at most 2^-25 of the product.  Six bf16 products with fp32
// accumulation run at a sixth of the bf16 rate where fp32 matrix instructions reach a
// sixteenth.  An infinity leaves a NaN in its remainders, so that the results it reaches
// are not finite (NaN, where an fp32 product might give an infinity).
// bf16 operands are multiplied as they are.  dz of a bf16 gradient is an fp32 number and cut into three
// like one, so that a gradient is rounded once, as a result (one bf16 number would add an error as
// large as that rounding, 2.3e-3 against 1.7e-3 in the 2-norm; two, 16 bits, would send more
// results the other way).  The scale of the dropout multiplies the fp32 results, so that without an
// activation dz is a masked g, and one number.
//
// Layout.  Tiles go through registers into LDS, as they lie in memory: a row of a tile is a
// run of k (x, g, W in dx) or, where the contraction runs across the rows (W in y; x and g
// in dW), a row of one k.  Operands of the first kind are read by 16 bytes along k, of the
// second by the transposing LDS read (ds_read_b64_tr_b16: sixteen lanes read 4 rows of 16
// elements, lane i gets column i).  The matrix instruction takes the weights' side first:
// a lane then holds four outputs in a row of one of the N rows.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "cgtp_linear.h"
#include "cgtp_linear_wide.h"

namespace cgtp {
namespace {

constexpr int kThreads = 256;
constexpr int kBK = 32;  // contraction per step

// A tile of RUNS rows of WIDTH elements in LDS, NP planes of it.  ALONG: the contraction
// runs along the rows.  The pads put the rows that are read together on different banks.
template <int kNP, int RUNS, int WIDTH, bool ALONG>
struct Side {
    static constexpr int NP = kNP;
    static constexpr bool kAlong = ALONG;
    static constexpr int kLd = WIDTH + (ALONG ? 8 : 16);
    static constexpr int kHalves = RUNS * kLd;  // of one plane
    static constexpr int kPer = WIDTH / 8;                     // blocks of eight in a row
    static constexpr int kEach = RUNS * WIDTH / 8 / kThreads;  // and per thread
    static_assert(RUNS * WIDTH % (8 * kThreads) == 0 && kThreads % (WIDTH / 8) == 0, "whole blocks per thread");

    // fragment of the 32 x 16 operand whose first row (of the matrix instruction's) is r0
    // and whose first k is k0
    __device__ static __forceinline__ b8 read(const uint16_t* s, int plane, int r0, int k0, int lane)
    {
        const uint16_t* p = s + plane * kHalves;
        if constexpr (ALONG) {
            return *reinterpret_cast<const b8*>(p + (r0 + (lane & 31)) * kLd + k0 + 8 * (lane >> 5));
        } else {
            const int l = lane & 15;
            p += (k0 + 8 * (lane >> 5) + l / 4) * kLd + r0 + (lane & 16) + 4 * (l % 4);
            return read_across(p, kLd);
        }
    }
};

// One BM x BN tile of the result (one part of its contraction): what no other form takes.  Each step of
// 32 k is fetched while the one before is multiplied, with one LDS buffer and two barriers; the blocks
// that share a compute unit fill each other's waits.  Bound by those at the sizes that come here, us with the
// join of the parts: 345 x 794 x 2198 fp32 33, 20 x 256 x 1024 bf16 7.2, 600 x 1024 x 1024 fp32 26 (its six
// products, 7.5 GFLOP, take 6 at the rate of a large library product).  VEC: every row of every array begins
// on 16 bytes and is a multiple of eight elements long.  HZ: there may be a z (kFwd: none).
template <class T, int KIND, int BM, int BN, bool VEC, bool HZ>
__global__ void __launch_bounds__(kThreads) k_linear(GemmArgs a)
{
    // rows' side P and columns' side Q
    constexpr bool kAlongP = KIND != kDw, kAlongQ = KIND == kDx;
    using P = Side<KIND == kDx ? kSlopePlanes<T, HZ> : kPlanes<T>, kAlongP ? BM : kBK, kAlongP ? kBK : BM, kAlongP>;
    using Q = Side<KIND == kDw ? kSlopePlanes<T, HZ> : kPlanes<T>, kAlongQ ? BN : kBK, kAlongQ ? kBK : BN, kAlongQ>;
    constexpr int WM = BM / 2, WN = BN / 2, FM = WM / 32, FN = WN / 32;
    constexpr bool kSlopeP = KIND == kDx, kSlopeQ = KIND == kDw;
    constexpr int kLdS = BN + 4, kHalf = BM / 2;  // the result leaves in two halves
    constexpr int kTiles = (P::kHalves * P::NP + Q::kHalves * Q::NP) * 2, kOut = kHalf * kLdS * 4, kSums = kThreads * 64;
    constexpr int kMem = kTiles > kOut ? kTiles : kOut;
    __shared__ __attribute__((aligned(16))) char mem[KIND == kDw && kSums > kMem ? kSums : kMem];
    uint16_t* sp = reinterpret_cast<uint16_t*>(mem);
    uint16_t* sq = sp + P::kHalves * P::NP;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t at = xcd_order(blockIdx.x, gridDim.x);
    const int64_t tile = at / a.splits, part = at % a.splits;
    const int64_t r0 = tile / a.tc * BM, c0 = tile % a.tc * BN;
    const int64_t k0 = part * a.run, k1 = k0 + a.run < a.depth ? k0 + a.run : a.depth;
    const uint64_t offset = drop_offset(a.drop);

    // The thread's blocks of eight: row `run` of the tile, element 8 * c.
    // Rows outside are taken as zero, elements outside too.
    Raw8<T> rp[P::kEach], rq[Q::kEach], rz[!HZ ? 1 : kSlopeP ? P::kEach : kSlopeQ ? Q::kEach : 1];
    auto fetch = [&](auto side, Raw8<T>* raw, const T* base, int64_t ld, int64_t n0, int64_t lim_n, int64_t e0,
                     int64_t lim_e) {
        using S = decltype(side);
        constexpr int kPer = S::kPer;
#pragma unroll
        for (int i = 0; i < S::kEach; ++i) {
            const int b = tid + i * kThreads;
            const int64_t n = n0 + b / kPer, e = e0 + b % kPer * 8;
            const bool in = n < lim_n && e < lim_e;
            const T* p = base + (in ? n * ld + e : 0);
            if constexpr (VEC) {
                raw[i].load(p);
                if (!in) raw[i].clear();
            } else {
                raw[i].load_some(p, !in ? 0 : lim_e - e < 8 ? (int)(lim_e - e) : 8);
            }
        }
    };
    const bool product = KIND != kDw || a.want;
    auto load = [&](int64_t k) {
        if constexpr (kAlongP) {
            fetch(P{}, rp, (const T*)a.A, a.lda, r0, a.rows, k, k1);
            if (kSlopeP && HZ && a.Z) fetch(P{}, rz, (const T*)a.Z, a.ldz, r0, a.rows, k, k1);
        } else {
            if (product) fetch(P{}, rp, (const T*)a.A, a.lda, k, k1, r0, a.rows);
        }
        if constexpr (kAlongQ) {
            fetch(Q{}, rq, (const T*)a.B, a.ldb, c0, a.cols, k, k1);
        } else {
            fetch(Q{}, rq, (const T*)a.B, a.ldb, k, k1, c0, a.cols);
            if (kSlopeQ && HZ && a.Z) fetch(Q{}, rz, (const T*)a.Z, a.ldz, k, k1, c0, a.cols);
        }
    };
    double sum[8] = {};  // of dz's columns 8 (tid % kPer) .. + 7
    const bool sums = KIND == kDw && a.db && r0 == 0;
    auto put = [&](auto side, uint16_t* s, const Raw8<T>* raw, auto slope, int64_t n0, int64_t e0) {
        using S = decltype(side);
        constexpr int kPer = S::kPer, NP = S::NP;
#pragma unroll
        for (int i = 0; i < S::kEach; ++i) {
            const int b = tid + i * kThreads;
            b8 planes[NP];
            if constexpr (decltype(slope)::value || NP > 1) {
                f8 v;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = raw[i][j];
                if constexpr (decltype(slope)::value) {
                    float z[8] = {};
                    if constexpr (HZ) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = rz[i][j];
                    }
                    slope8<HZ>(a, offset, v, z, n0 + b / kPer, (int32_t)((e0 + b % kPer * 8) / 8));
                    if (sums) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum[j] += (double)v[j];
                    }
                }
                if constexpr (S::kAlong) cut_along(v, planes);
                else cut(v, planes);
            } else {
                planes[0] = __builtin_bit_cast(b8, raw[i].v[0]);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p)
                *reinterpret_cast<b8*>(s + p * S::kHalves + b / kPer * S::kLd + b % kPer * 8) = planes[p];
        }
    };
    auto store = [&](int64_t k) {
        if constexpr (kSlopeP) put(P{}, sp, rp, std::true_type{}, r0, k);
        else if (product) put(P{}, sp, rp, std::false_type{}, 0, 0);
        if constexpr (kSlopeQ) put(Q{}, sq, rq, std::true_type{}, k, c0);
        else put(Q{}, sq, rq, std::false_type{}, 0, 0);
    };

    f16v acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[x][y][q] = 0.0f;
    const int wm = wave / 2 * WM, wn = wave % 2 * WN;
    auto multiply = [&]() {
#pragma unroll
        for (int ks = 0; ks < kBK; ks += 16) {
            b8 fp[FM][P::NP], fq[FN][Q::NP];
#pragma unroll
            for (int p = 2; p >= 0; --p) {
#pragma unroll
                for (int x = 0; x < FM; ++x)
                    if (p < P::NP) fp[x][p] = P::read(sp, p, wm + 32 * x, ks, lane);
#pragma unroll
                for (int y = 0; y < FN; ++y)
                    if (p < Q::NP) fq[y][p] = Q::read(sq, p, wn + 32 * y, ks, lane);
            }
            each_product<P::NP, Q::NP>([&](int i, int j) {
#pragma unroll
                for (int x = 0; x < FM; ++x)
#pragma unroll
                    for (int y = 0; y < FN; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fq[y][j], fp[x][i], acc[x][y], 0, 0, 0);
            });
        }
    };

    load(k0);
    for (int64_t k = k0; k < k1; k += kBK) {
        store(k);
        __syncthreads();
        if (k + kBK < k1) load(k + kBK);
        if (product) multiply();
        __syncthreads();
    }

    if (KIND == kDw && sums) {
        // the threads of one column block, in order
        constexpr int kPer = BN / 8;
        double* s = reinterpret_cast<double*>(mem);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j * kThreads + tid] = sum[j];
        __syncthreads();
        if (tid < BN) {
            double t = 0.0;
            for (int i = 0; i < kThreads / kPer; ++i) t += s[tid % 8 * kThreads + i * kPer + tid / 8];
            if (c0 + tid < a.cols) {
                if (a.splits > 1) a.db_part[part * a.cols + c0 + tid] = t;
                else a.db[c0 + tid] = (float)(t * (double)a.drop.scale);
            }
        }
        __syncthreads();
    }
    if (!product) return;

    // A lane holds row lane % 32 and columns 8 g + 4 (lane / 32) + 0 .. 3 of each tile of 32:
    // through LDS, so that rows leave in whole lines; a thread keeps to its eight columns.
    constexpr int kPer = BN / 8, kRows = kThreads / kPer, kG = kHalf / kRows < 4 ? kHalf / kRows : 4;
    const int64_t c = c0 + tid % kPer * 8;
    const int w = a.cols - c < 8 ? (int)(a.cols - c) : 8;
    float bias[8] = {};
    if (KIND == kFwd && c < a.cols) bias8<VEC>(a, c, w, bias);
    float* s = reinterpret_cast<float*>(mem);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h) __syncthreads();
        if (wave / 2 == h) {
#pragma unroll
            for (int x = 0; x < FM; ++x)
#pragma unroll
                for (int y = 0; y < FN; ++y)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float4 v{acc[x][y][4 * g], acc[x][y][4 * g + 1], acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
                        *reinterpret_cast<float4*>(&s[(32 * x + (lane & 31)) * kLdS + wn + 32 * y + 8 * g + 4 * (lane >> 5)]) = v;
                    }
        }
        __syncthreads();
        for (int i0 = 0; i0 < kHalf; i0 += kG * kRows) {
            float v[kG][8];
            int64_t n[kG];
            bool on[kG];
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                const int i = i0 + g * kRows + tid / kPer;
                n[g] = r0 + h * kHalf + i;
                on[g] = n[g] < a.rows && c < a.cols;
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4*>(&v[g][e]) = *reinterpret_cast<const float4*>(&s[i * kLdS + tid % kPer * 8 + e]);
            }
            leave8<T, KIND, VEC, kG>(a, offset, part, v, bias, n, on, c, w);
        }
    }
}

// The parts' sums in fp64 and the epilogue: G threads share eight results, each adds every
// G-th part in order (G = 8 where there are many: one thread's loads would wait for each
// other, 128 parts of 128 x 128 34 us), then one adds the eight.  The gradient of the bias by
// the blocks behind the others, eight threads to a column.
template <class T, int KIND, bool VEC, int G>
__global__ void __launch_bounds__(kThreads) k_linear_join(GemmArgs a, int64_t blocks)
{
    constexpr int kEach = kThreads / G;
    __shared__ double s[G > 1 ? kThreads * 8 : kThreads];
    const int tid = threadIdx.x, g = tid / kEach;
    if ((int64_t)blockIdx.x >= blocks) {
        constexpr int kCols = kThreads / 8;
        const int64_t c = ((int64_t)blockIdx.x - blocks) * kCols + tid % kCols;
        double t = 0.0;
        if (c < a.cols) {
#pragma unroll 4
            for (int64_t i = tid / kCols; i < a.db_splits; i += 8) t += a.db_part[i * a.cols + c];
        }
        s[tid] = t;
        __syncthreads();
        if (tid >= kCols || c >= a.cols) return;
        for (int i = 1; i < 8; ++i) t += s[i * kCols + tid];
        a.db[c] = (float)(t * (double)a.drop.scale);
        return;
    }
    const int64_t per = (a.cols + 7) / 8, q = (int64_t)blockIdx.x * kEach + tid % kEach;
    const bool on = q < a.rows * per;
    const int64_t n = on ? q / per : 0, c = on ? q % per * 8 : 0;
    const int w = a.cols - c < 8 ? (int)(a.cols - c) : 8;
    double t[8] = {};
    if (on) {
        const float* p = a.part + (g * a.rows + n) * a.cols + c;
#pragma unroll 4
        for (int64_t i = g; i < a.splits; i += G, p += G * a.rows * a.cols) {
            Raw8<float> v;
            v.load_some(p, VEC ? 8 : w);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] += (double)v[j];
        }
    }
    if constexpr (G > 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j * kThreads + tid] = t[j];
        __syncthreads();
        if (g) return;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            for (int i = 1; i < G; ++i) t[j] += s[j * kThreads + i * kEach + tid];
    }
    if (!on) return;
    float v[1][8], bias[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[0][j] = (float)t[j];
    if (KIND == kFwd) bias8<VEC>(a, c, w, bias);
    finish8<T, KIND, VEC, 1>(a, drop_offset(a.drop), v, bias, {n}, {true}, c, w);
}

// out[0 .. bytes) = 0, two at a time (a kernel: a captured graph may hold it)
__global__ void __launch_bounds__(kThreads) k_linear_zero(int64_t bytes, char* __restrict__ out)
{
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 2;
    for (int64_t q = i; q < bytes; q += (int64_t)gridDim.x * kThreads * 2) *reinterpret_cast<uint16_t*>(out + q) = 0;
}

// ---- choice of tiles and parts ------------------------------------------------------------
struct Plan {
    int bm, bn;
    int64_t tr, tc, splits, run;
};

constexpr int64_t kManySplits = 16;  // eight threads to a result from here on

// the three products' result and contraction
struct Dims {
    int64_t rows, cols, depth;
};

Dims dims_of(const LinShape& n, int kind)
{
    return kind == kFwd ? Dims{n.N, n.M, n.K} : kind == kDx ? Dims{n.N, n.K, n.M} : Dims{n.K, n.M, n.N};
}

// Tiles of 128 where they fill the chip or the result is that wide; the contraction is cut
// where tiles alone leave compute units idle, into parts of at least four steps (twelve where half of
// the compute units have a tile) and some four blocks to a compute unit.  (970 x 151 x 4092 bf16 gradients
// 60 us and 83 with SiLU, with eight steps and two blocks 64 and 91, uncut 153 and 297; 345 x 794 x 2198 fp32, 210
// tiles, 32 against 44 uncut.)
Plan plan_tiles(const Dims& d)
{
    Plan p{};
    auto side = [](int64_t n) { return n > 64 ? 128 : 64; };
    p.bm = side(d.rows);
    p.bn = side(d.cols);
    auto tiles = [&]() { return cdiv64(d.rows, p.bm) * cdiv64(d.cols, p.bn); };
    if (tiles() < 256) p.bm = 64;
    if (tiles() < 256) p.bn = 64;
    p.tr = cdiv64(d.rows, p.bm);
    p.tc = cdiv64(d.cols, p.bn);
    const int64_t n = p.tr * p.tc, most = d.depth / (n < 128 ? 4 * kBK : 12 * kBK);
    int64_t s = n >= 256 ? 1 : 1024 / n;
    s = s < most ? s : most;
    s = s < 1 ? 1 : s;
    p.run = cdiv64(cdiv64(d.depth, s), kBK) * kBK;
    p.splits = cdiv64(d.depth, p.run);
    return p;
}

// Tiles of 256 where they, with the parts of a contraction of at least 512, fill the chip once; else of 128,
// three blocks to a compute unit.
Plan plan_wide(const Dims& d)
{
    Plan p{};
    p.bm = p.bn = 256;
    auto tiles = [&]() { return cdiv64(d.rows, p.bm) * cdiv64(d.cols, p.bn); };
    const int64_t most = cdiv64(d.depth, 512);
    if (tiles() * most < 256) p.bm = p.bn = 128;
    p.tr = cdiv64(d.rows, p.bm);
    p.tc = cdiv64(d.cols, p.bn);
    int64_t s = (p.bm == 256 ? 256 : 768) / (p.tr * p.tc);
    s = s < most ? s : most;
    s = s < 1 ? 1 : s;
    p.run = cdiv64(cdiv64(d.depth, s), kBK) * kBK;
    p.splits = cdiv64(d.depth, p.run);
    return p;
}

// Rows behind the last whole tile that go by themselves: up to 64 of them, where without
// them the tiles take a turn of the chip less.  (16385 x 1024 x 4096: one turn for dx instead of
// two, four for y instead of five, for one or two launches of 64 x 64 tiles more.)
int64_t rest_of(const Dims& d)
{
    const Plan p = plan_wide(d);
    const int64_t rest = d.rows % p.bm, turn = p.bm == 256 ? 256 : 768, n = p.tr * p.tc;
    return rest <= 64 && d.rows > p.bm && cdiv64(n, turn) > cdiv64(n - p.tc, turn) ? rest : 0;
}

constexpr int64_t kMaxWideLd = int64_t(1) << 22;  // row strides: a tile's byte offsets stay in 32 bits

// Planes where the products bound the call, not memory or launches: forward and gradients of fp32 2048 x 1024 x
// 512 (1.07e9) 43 and 72 us, by tiles 30 and 66; 1500 x 1024 x 1024 (1.57e9) 46 and 91, by tiles 42 and 132.
// bf16 1000 x 256 x 512 (1.3e8) 7.1 and 17.9, by tiles 5.9 and 19.7; 800 x 512 x 512 (2.1e8) 8.5 and
// 16.8, by tiles 10.4 and 21.7.  bf16 gradients with a slope, whose dz is three planes in memory, replayed from a
// graph: 800 x 512 x 512 38, by tiles 30; 8000 x 256 x 256 (5.2e8) 38 and 36; 1500 x 1024 x 512 (7.9e8) 50
// and 56; 1500 x 1024 x 1024 61 and 109.
bool wide_shape(const LinShape& n, bool backward)
{
    const double least = n.dtype == kF32 ? 1.1e9 : backward && n.act != kNone ? 6e8 : 2e8;
    return n.K % 8 == 0 && n.M % 8 == 0 && n.N >= 256 && n.K >= 256 && n.M >= 256 &&
           (double)n.N * (double)n.K * (double)n.M >= least;
}

// Few rows: one pass over W on the vector units.  Replayed from a graph, us: 1, 4 and 16 rows x
// 1024 x 4096 bf16 3.8, 5.4 and 6.7, by tiles 7.6 to 8.0; fp32 3.9, 5.5 and 7.0, by tiles 12.4.
// Where W is small tiles are as quick from three rows on (128 x 128 bf16: 4.1).
bool few_rows(int64_t rows, int64_t depth) { return rows <= 2 || (rows <= 16 && depth >= 512); }

// Rows that registers hold whole, and enough of them: 105730 x 64 x 1920 fp32 217 to 241 us, by tiles 264 to
// 279, bf16 98 and 135; 105730 x 8 x 64 14.8 and 20; 2000 x 128 x 128 7.7 and 7.2.
bool rows_whole(const LinShape& n) { return n.K <= 128 && n.N >= 256; }

// Gradients in one pass: up to 128 outputs.  With tanh, replayed from a graph: 2000 x 128 x 128 fp32 17.3 us, by
// tiles 27.7; 25000 x 128 x 128 bf16 29.7 and 37.0; 20000 x 1024 x 128 fp32 107 and 153.
bool one_pass(const LinShape& n) { return n.M <= 128; }

// dx of few inputs over many outputs, from rows of g in registers: where its blocks, which go through all
// outputs, fill the chip.  Replayed from a graph, over 1920 outputs, us (by tiles): above 64 inputs, blocks of 128
// rows, 72 x 40000 rows fp32 149 (180), with SiLU 257 (273), bf16 50 (65) and 136 (195), 128 x 105730 345 (380),
// 528 (507), 151 (155) and 301 (363); 128 x 24576 with SiLU fp32 149 (131).  Up to 64 inputs, blocks of 256
// rows, fp32 without a slope: 64 x 40000 120 (138), 105730 243 (264), 32768 96 (85); with SiLU 64 x 65536
// 255 (230), 160000 678 (516), bf16 without a slope 8 x 160000 187 (131).  With few blocks tiles cut the
// contraction instead: 64 x 4096 rows over 4096 outputs fp32 with SiLU 404 (33).
bool dx_rows(const LinShape& n)
{
    if (n.K > 128 || n.M <= 128 || n.M % 8 != 0) return false;
    return n.K > 64 ? n.N >= 32768 : n.dtype == kF32 && n.act == kNone && n.N >= 40000;
}

// dW of few inputs, from columns of x and g in registers, with their join: 64 x 1920 of 105730 rows 211 us, by
// tiles 299; 8 x 4096 of 8192 38 and 45 (where dz is g: z would not find room there, and a mask would be
// formed eight times).
bool dw_columns(const LinShape& n) { return n.dtype == kF32 && n.K <= 64 && n.M > 128 && n.N >= 8192; }

Plan plan_columns(const LinShape& n)
{
    Plan p{};
    p.tr = 1;
    p.tc = cdiv64(n.M, 128);
    const int64_t s = p.tc < 512 ? 512 / p.tc : 1;
    p.run = cdiv64(cdiv64(n.N, s), 64) * 64;
    p.splits = cdiv64(n.N, p.run);
    return p;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

size_t part_bytes(const Plan& p, const Dims& d, bool bias)
{
    if (p.splits <= 1) return 0;
    return round256((size_t)(p.splits * d.rows * d.cols) * 4) + (bias ? (size_t)(p.splits * d.cols) * 8 : 0);
}

Plan plan_of(const LinShape& n, int kind) { return plan_tiles(dims_of(n, kind)); }

// rows of a block that forms planes, and how many blocks that makes
int64_t plane_run(int64_t rows, int64_t cols)
{
    const int64_t across = cdiv64(cols, 256);
    int64_t run = cdiv64(rows * across, 2048);
    run = cdiv64(run < 8 ? 8 : run, 8) * 8;
    return run;
}

// workspace of the narrow form: parts of dW, parts of db
size_t back_bytes(int64_t splits, const LinShape& n)
{
    return round256((size_t)(splits * n.K * n.M) * 4) + (size_t)(splits * n.M) * 8;
}

// workspace of the wide form, by arrays
struct WideSpace {
    size_t dz, x, W, db, part, bytes;
    WideSpace(const LinShape& n, bool backward)
    {
        const int np = n.dtype == kF32 ? 3 : 1;
        size_t at = 0;
        auto take = [&](size_t b) {
            const size_t was = at;
            at += round256(b);
            return was;
        };
        dz = take(backward ? (size_t)(3 * n.N * n.M) * 2 : 0);
        x = take(np > 1 ? (size_t)(np * n.N * n.K) * 2 : 0);
        W = take(np > 1 ? (size_t)(np * n.K * n.M) * 2 : 0);
        db = take(backward ? (size_t)(cdiv64(n.N, plane_run(n.N, n.M)) * n.M) * 8 : 0);
        size_t most = 0;
        for (int kind : {kFwd, kDx, kDw}) {
            if ((kind != kFwd) != backward) continue;
            Dims d = dims_of(n, kind);
            const int64_t rest = kind == kDw ? 0 : rest_of(d);
            d.rows -= rest;
            const size_t b = part_bytes(plan_wide(d), d, false);
            most = most > b ? most : b;
            d.rows = rest;
            const size_t c = rest ? part_bytes(plan_tiles(d), d, false) : 0;
            most = most > c ? most : c;
        }
        part = take(most);
        bytes = at;
    }
};

template <class T, int KIND, bool VEC>
hipError_t join(const GemmArgs& a, hipStream_t s)
{
    const dim3 block(kThreads);
    const bool many = a.splits >= kManySplits;
    const int64_t blocks = KIND != kDw || a.want ? cdiv64(a.rows * cdiv64(a.cols, 8), many ? kThreads / 8 : kThreads) : 0;
    const int64_t more = KIND == kDw && a.db ? cdiv64(a.cols, kThreads / 8) : 0;
    const dim3 grid((unsigned)(blocks + more));
    if (many) hipLaunchKernelGGL((k_linear_join<T, KIND, VEC, 8>), grid, block, 0, s, a, blocks);
    else hipLaunchKernelGGL((k_linear_join<T, KIND, VEC, 1>), grid, block, 0, s, a, blocks);
    return hipGetLastError();
}

template <class T, int KIND, bool VEC>
hipError_t run(GemmArgs& a, const Plan& p, void* ws, hipStream_t s)
{
    a.tr = p.tr;
    a.tc = p.tc;
    a.splits = p.splits;
    a.run = p.run;
    if (p.splits > 1) {
        a.part = (float*)ws;
        a.db_part = (double*)((char*)ws + round256((size_t)(p.splits * a.rows * a.cols) * 4));
        a.db_splits = p.splits;
    }
    auto tiles = [&](auto z) {
        constexpr bool HZ = decltype(z)::value;
        const dim3 grid((unsigned)(p.tr * p.tc * p.splits)), block(kThreads);
        if (p.bm == 128 && p.bn == 128) hipLaunchKernelGGL((k_linear<T, KIND, 128, 128, VEC, HZ>), grid, block, 0, s, a);
        else if (p.bm == 128) hipLaunchKernelGGL((k_linear<T, KIND, 128, 64, VEC, HZ>), grid, block, 0, s, a);
        else if (p.bn == 128) hipLaunchKernelGGL((k_linear<T, KIND, 64, 128, VEC, HZ>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_linear<T, KIND, 64, 64, VEC, HZ>), grid, block, 0, s, a);
    };
    // (fp32 operands have three planes either way)
    if constexpr (KIND == kFwd) tiles(std::false_type{});
    else if (kPlanes<T> == 3 || a.Z) tiles(std::true_type{});
    else tiles(std::false_type{});
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || p.splits <= 1 ? e : join<T, KIND, VEC>(a, s);
}

template <class T, int KIND>
hipError_t run(GemmArgs& a, const Plan& p, bool vec, void* ws, hipStream_t s)
{
    return vec ? run<T, KIND, true>(a, p, ws, s) : run<T, KIND, false>(a, p, ws, s);
}

// one product of planes
template <class T, int KIND>
hipError_t run_wide(const LinShape& n, int64_t rest, GemmArgs a, const uint16_t* P, int64_t ldp, const uint16_t* Q,
                    int64_t ldq, float* part, hipStream_t s)
{
    Dims d = dims_of(n, KIND);
    d.rows -= rest;
    const Plan p = plan_wide(d);
    WideArgs w{};
    a.rows = d.rows;
    a.cols = d.cols;
    a.depth = d.depth;
    a.tr = p.tr;
    a.tc = p.tc;
    a.splits = p.splits;
    a.run = p.run;
    a.part = part;
    w.g = a;
    w.P = P;
    w.Q = Q;
    w.ldp = ldp;
    w.ldq = ldq;
    w.planeP = KIND == kDx ? n.N * n.M : n.N * n.K;
    w.planeQ = KIND == kDw ? n.N * n.M : n.K * n.M;
    w.side = p.bm;
    const hipError_t e = launch_linear_wide(n.dtype, KIND, w, s);
    if (e != hipSuccess || (p.splits <= 1 && !(KIND == kDw && a.db))) return e;
    if (p.splits <= 1) w.g.want = false;  // dW is there
    return join<T, KIND, true>(w.g, s);
}

// x or W as planes: as it is for bf16, else formed at `to`
template <class T>
hipError_t planes_of(const void* v, int64_t ld, int64_t rows, int64_t cols, void* to, const uint16_t*& p, int64_t& ldp,
                     hipStream_t s)
{
    if (kPlanes<T> == 1) {
        p = (const uint16_t*)v;
        ldp = ld;
        return hipSuccess;
    }
    PlaneArgs a{};
    a.x = v;
    a.ld = ld;
    a.rows = rows;
    a.cols = cols;
    a.run = plane_run(rows, cols);
    a.out = (uint16_t*)to;
    p = a.out;
    ldp = cols;
    return launch_linear_planes(kF32, false, a, s);
}

template <class T>
hipError_t fwd(const LinShape& n, const void* x, const void* W, const float* bias, const void* R, void* z, void* y,
               void* ws, hipStream_t s)
{
    GemmArgs a{};
    a.A = x;
    a.B = W;
    a.lda = n.ldx;
    a.ldb = n.M;
    a.rows = n.N;
    a.cols = n.M;
    a.depth = n.K;
    a.act = n.act;
    a.drop = n.drop;
    a.bias = bias;
    a.R = R;
    a.out = y;
    a.zout = z;
    a.ldr = n.ldr;
    a.ldo = n.ldy;
    constexpr int64_t es = sizeof(T);
    const bool vec = n.K % 8 == 0 && n.M % 8 == 0 && aligned_rows(x, n.ldx, es) && aligned_rows(W, n.M, es) &&
                     aligned_rows(y, n.ldy, es) && (!z || aligned_rows(z, n.M, es)) &&
                     (!R || aligned_rows(R, n.ldr, es));
    if (vec && wide_shape(n, false) && n.ldx < kMaxWideLd) {
        const WideSpace at(n, false);
        char* w = (char*)ws;
        const uint16_t *P, *Q;
        int64_t ldp, ldq;
        hipError_t e = planes_of<T>(x, n.ldx, n.N, n.K, w + at.x, P, ldp, s);
        if (e == hipSuccess) e = planes_of<T>(W, n.M, n.K, n.M, w + at.W, Q, ldq, s);
        const int64_t rest = rest_of(dims_of(n, kFwd));
        if (e == hipSuccess) e = run_wide<T, kFwd>(n, rest, a, P, ldp, Q, ldq, (float*)(w + at.part), s);
        if (e != hipSuccess || !rest) return e;
        a.first = n.N - rest;
        a.rows = rest;
        a.A = (const T*)x + a.first * n.ldx;
        if (R) a.R = (const T*)R + a.first * n.ldr;
        a.out = (T*)y + a.first * n.ldy;
        if (z) a.zout = (T*)z + a.first * n.M;
        if (few_rows(rest, n.K)) return launch_linear_few(n.dtype, true, a, s);
        return run<T, kFwd>(a, plan_tiles(Dims{rest, n.M, n.K}), true, w + at.part, s);
    }
    if (rows_whole(n)) return launch_linear_rows(n.dtype, vec, a, s);
    if (few_rows(n.N, n.K)) return launch_linear_few(n.dtype, vec, a, s);
    return run<T, kFwd>(a, plan_of(n, kFwd), vec, ws, s);
}

template <class T>
hipError_t bwd_wide(const LinShape& n, GemmArgs a, const void* x, const void* W, const void* g, void* dx, void* dW,
                    float* db, void* ws, hipStream_t s)
{
    const WideSpace at(n, true);
    char* w = (char*)ws;
    // dz: g itself where it is a plane already
    const bool plain = kPlanes<T> == 1 && a.act == kNone && a.drop.thr == 0 && n.ldg < kMaxWideLd;
    const uint16_t* dz = plain ? (const uint16_t*)g : (const uint16_t*)(w + at.dz);
    const int64_t ldz = plain ? n.ldg : n.M;
    hipError_t e = hipSuccess;
    a.db = db;
    a.db_part = (double*)(w + at.db);
    if (!plain || db) {
        PlaneArgs p{};
        p.g = a;
        p.x = g;
        p.ld = n.ldg;
        p.rows = n.N;
        p.cols = n.M;
        p.run = plane_run(n.N, n.M);
        p.out = plain || !(dx || dW) ? nullptr : (uint16_t*)(w + at.dz);
        a.db_splits = cdiv64(p.rows, p.run);
        e = launch_linear_planes(n.dtype, true, p, s);
        if (e != hipSuccess) return e;
    }
    float* part = (float*)(w + at.part);
    const uint16_t *P, *Q;
    int64_t ldp, ldq;
    if (dx) {
        GemmArgs b = a;
        b.out = dx;
        b.ldo = n.ldd;
        b.db = nullptr;
        const int64_t rest = rest_of(dims_of(n, kDx));
        e = planes_of<T>(W, n.M, n.K, n.M, w + at.W, Q, ldq, s);
        if (e == hipSuccess) e = run_wide<T, kDx>(n, rest, b, dz, ldz, Q, ldq, part, s);
        if (e == hipSuccess && rest) {
            b.first = n.N - rest;
            b.A = (const T*)g + b.first * n.ldg;
            if (b.Z) b.Z = (const T*)b.Z + b.first * n.M;
            b.B = W;
            b.lda = n.ldg;
            b.ldb = n.M;
            b.rows = rest;
            b.cols = n.K;
            b.depth = n.M;
            b.out = (T*)dx + b.first * n.ldd;
            e = run<T, kDx>(b, plan_tiles(Dims{rest, n.K, n.M}), true, part, s);
        }
        if (e != hipSuccess) return e;
    }
    a.out = dW;
    a.ldo = n.M;
    a.want = dW != nullptr;
    if (dW) {
        e = planes_of<T>(x, n.ldx, n.N, n.K, w + at.x, P, ldp, s);
        return e != hipSuccess ? e : run_wide<T, kDw>(n, 0, a, P, ldp, dz, ldz, part, s);
    }
    if (db) {
        a.rows = n.K;
        a.cols = n.M;
        return join<T, kDw, true>(a, s);
    }
    return hipSuccess;
}

template <class T>
hipError_t bwd(const LinShape& n, const void* x, const void* W, const void* z, const void* g, void* dx, void* dW,
               float* db, void* ws, hipStream_t s)
{
    constexpr int64_t es = sizeof(T);
    GemmArgs a{};
    a.Z = n.act == kNone ? nullptr : z;
    a.ldz = n.M;
    a.act = n.act;
    a.drop = n.drop;
    const bool vec = n.K % 8 == 0 && n.M % 8 == 0 && aligned_rows(g, n.ldg, es) && (!a.Z || aligned_rows(z, n.M, es));
    const bool vec_x = vec && aligned_rows(W, n.M, es) && aligned_rows(dx, n.ldd, es);
    const bool vec_w = vec && aligned_rows(x, n.ldx, es) && aligned_rows(dW, n.M, es);
    // parts of dW and db, and what is needed to add them
    auto parts = [&](int64_t tr, int64_t tc, int64_t splits) {
        GemmArgs b = a;
        b.A = x;
        b.B = g;
        b.lda = n.ldx;
        b.ldb = n.ldg;
        b.rows = n.K;
        b.cols = n.M;
        b.depth = n.N;
        b.tr = tr;
        b.tc = tc;
        b.splits = b.db_splits = splits;
        b.part = (float*)ws;
        b.db_part = (double*)((char*)ws + round256((size_t)(splits * n.K * n.M) * 4));
        b.out = dW;
        b.ldo = n.M;
        b.db = db;
        b.want = dW != nullptr;
        return b;
    };
    auto add = [&](const GemmArgs& b) { return vec_w ? join<T, kDw, true>(b, s) : join<T, kDw, false>(b, s); };
    if (one_pass(n)) {
        const BackPlan p = back_plan(n.N, n.K, n.M);
        const GemmArgs b = parts(p.tr, 1, p.splits);
        const hipError_t e = launch_linear_back(n.dtype, vec && (!dW || vec_w) && (!dx || vec_x), b, p, W, dx, n.ldd, s);
        return e != hipSuccess || (!dW && !db) ? e : add(b);
    }
    if (dx && vec_x && dx_rows(n) && n.ldg < kMaxWideLd) {
        WideArgs w{};
        w.g = a;
        w.g.A = g;
        w.g.lda = n.ldg;
        w.g.rows = n.N;
        w.g.cols = n.K;
        w.g.depth = n.M;
        w.g.out = dx;
        w.g.ldo = n.ldd;
        w.planeQ = n.K * n.M;
        hipError_t e = planes_of<T>(W, n.M, n.K, n.M, ws, w.Q, w.ldq, s);
        if (e == hipSuccess) e = launch_linear_dx(n.dtype, w, s);
        if (e != hipSuccess) return e;
        dx = nullptr;
    }
    if (dW && n.act == kNone && n.drop.thr == 0 && dw_columns(n) && n.ldx < kMaxWideLd && n.ldg < kMaxWideLd) {
        const Plan p = plan_columns(n);
        GemmArgs b = parts(1, p.tc, p.splits);
        b.run = p.run;
        const hipError_t e = launch_linear_dw(b, s);
        if (e != hipSuccess) return e;
        const hipError_t f = add(b);
        if (f != hipSuccess) return f;
        dW = nullptr;
        db = nullptr;
    }
    if ((!dx || vec_x) && (!dW || vec_w) && vec && wide_shape(n, true) && (!dW || n.ldx < kMaxWideLd))
        return bwd_wide<T>(n, a, x, W, g, dx, dW, db, ws, s);
    if (dx) {
        GemmArgs b = a;
        b.A = g;
        b.B = W;
        b.lda = n.ldg;
        b.ldb = n.M;
        b.rows = n.N;
        b.cols = n.K;
        b.depth = n.M;
        b.out = dx;
        b.ldo = n.ldd;
        const hipError_t e = run<T, kDx>(b, plan_of(n, kDx), vec_x, ws, s);
        if (e != hipSuccess) return e;
    }
    if (dW || db) {
        a.A = x;  // not read where only the bias is wanted
        a.B = g;
        a.lda = n.ldx;
        a.ldb = n.ldg;
        a.rows = n.K;
        a.cols = n.M;
        a.depth = n.N;
        a.out = dW;
        a.ldo = n.M;
        a.db = db;
        a.want = dW != nullptr;
        return run<T, kDw>(a, plan_of(n, kDw), dW ? vec_w : vec, ws, s);
    }
    return hipSuccess;
}

hipError_t zero(void* p, int64_t bytes, hipStream_t s)
{
    int64_t blocks = cdiv64(bytes, kThreads * 8);
    blocks = blocks < 4096 ? blocks : 4096;
    hipLaunchKernelGGL(k_linear_zero, dim3((unsigned)blocks), dim3(kThreads), 0, s, bytes, (char*)p);
    return hipGetLastError();
}

}  // namespace

bool linear_fits(const LinShape& n)
{
    if (n.N == 0) return true;
    // (the rows' form takes 64 to a block of 256 threads where their registers have no room for more)
    if (rows_whole(n) && n.dtype == kF32 && n.K > 64 && cdiv64(n.N, 64) >= 16777216) return false;
    for (int kind : {kFwd, kDx, kDw}) {
        const Dims d = dims_of(n, kind);
        const Plan p = plan_tiles(d);
        const double blocks = (double)p.tr * (double)p.tc * (double)p.splits;
        const double join = p.splits > 1 ? (double)d.rows * ((double)d.cols / 8 + 1) / 32 : 0.0;
        if (blocks >= 16777216.0 || join >= 8388608.0) return false;
    }
    return true;
}

size_t linear_workspace_bytes(const LinShape& n, bool backward)
{
    if (n.N == 0) return 0;
    if (backward && one_pass(n)) return back_bytes(back_plan(n.N, n.K, n.M).splits, n);
    // (The activation is not known here: none, with which the forms have their widest ranges.  Rows without
    // 16-byte alignment take the tiles where others take planes.)
    size_t most = wide_shape(n, backward) ? WideSpace(n, backward).bytes : 0;
    if (backward && dx_rows(n) && n.dtype == kF32) most = (size_t)(3 * n.K * n.M) * 2;
    if (backward && dw_columns(n)) {
        const size_t b = back_bytes(plan_columns(n).splits, n);
        most = most > b ? most : b;
    }
    for (int kind : {kFwd, kDx, kDw}) {
        if ((kind != kFwd) != backward) continue;
        if (kind == kFwd && (few_rows(n.N, n.K) || rows_whole(n))) continue;
        const size_t b = part_bytes(plan_of(n, kind), dims_of(n, kind), kind == kDw);
        most = most > b ? most : b;
    }
    return most;
}

hipError_t launch_linear_fwd(const LinShape& n, const void* x, const void* W, const float* bias, const void* residual,
                             void* z, void* y, void* ws, hipStream_t s)
{
    if (n.N == 0) return hipSuccess;
    return n.dtype == kF32 ? fwd<float>(n, x, W, bias, residual, z, y, ws, s)
                           : fwd<bf16_t>(n, x, W, bias, residual, z, y, ws, s);
}

hipError_t launch_linear_bwd(const LinShape& n, const void* x, const void* W, const void* z, const void* grad_y,
                             void* grad_x, void* grad_W, float* grad_bias, void* ws, hipStream_t s)
{
    if (n.N == 0) {
        hipError_t e = hipSuccess;
        if (grad_W) e = zero(grad_W, n.K * n.M * dtype_size(n.dtype), s);
        if (e == hipSuccess && grad_bias) e = zero(grad_bias, n.M * 4, s);
        return e;
    }
    return n.dtype == kF32 ? bwd<float>(n, x, W, z, grad_y, grad_x, grad_W, grad_bias, ws, s)
                           : bwd<bf16_t>(n, x, W, z, grad_y, grad_x, grad_W, grad_bias, ws, s);
}

}  // namespace cgtp
