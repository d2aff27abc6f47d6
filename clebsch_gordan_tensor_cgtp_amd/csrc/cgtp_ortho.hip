// cgtp_ortho.hip -- orthogonalised updates by Newton-Schulz products on the
// fp16 matrix cores.
//
//   X = G / (||G||_F + eps), then `steps` times
//   A = X X^T,  B = b A + c A A,  X <- a X + B X
// on the orientation whose rows are the shorter side (s <= t), so that every
// singular value x of X becomes a x + b x^3 + c x^5.
//
// Precision.  Each operand v is kept as two fp16 numbers, h = fp16(v k) and
// l = fp16(v k - h), with a power of two k that places the operand's bound at
// 2^14..2^15: the spectral norm is at most ||X||_F = ||G||_F / (||G||_F + eps) at
// the start and follows the polynomial's maximum from step to step.  h + l holds 23
// bits (eleven each and l's sign) of every value down to 2^-16 of the bound, one
// fewer than fp32, and
//   u v = (hu hv + hu lv + lu hv) / k^2
// leaves out lu lv only, at most 2^-22 of the product and of either sign.  Three fp16
// products with fp32 accumulation so give what an fp32 product gives (the result of
// five steps is off by 0.8 to 1.1 times what fp32 products give, from 20 rows up), at
// a third of the fp16 rate instead of the sixteenth that fp32 matrix instructions
// reach.  Below 17 rows sums are too short to hide the missing bit (up to twice the
// fp32 error), and there is little to multiply: those matrices run in fp64, up to the
// 32768 elements that a block holds.
//
// bf16 matrices take the same three products.  A step carries the error of the steps
// before on, and steeper coefficients magnify it: with hu hv alone in A = X X^T the
// result was off by 4e-4 to 8e-4 after five steps of the usual quintic, 2e-3 after twenty
// and 4e-3 after five of (4.0848, -6.8946, 2.9270).
//
// Layout.  An operand of `rows` rows is cut along k into blocks of 32: a row's
// piece of a block is 32 h, then their 32 l, one 128-byte line, and a block's
// lines lie one after the other, so that what a tile loads for one block of k
// is one run of memory (plain rows measured the same).  All products are "rows times
// rows": D[i][j] = sum_k P[i][k] Q[j][k] with k contiguous in both; A and B are
// symmetric, and X is kept as it is and transposed.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "cgtp_internal.h"
#include "cgtp_train_internal.h"
#include "cgtp_vec.h"

namespace cgtp {
namespace {

constexpr int kThreads = 256;
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// offset of element (row, k) of a split operand (its low half is 32 further on)
__device__ __forceinline__ int64_t split_at(int64_t row, int64_t k, int64_t rows)
{
    return ((k >> 5) * rows + row) * 64 + (k & 31);
}

__device__ __forceinline__ void split(float v, _Float16& h, _Float16& l)
{
    h = (_Float16)v;
    l = (_Float16)(v - (float)h);
}

// ---- units ------------------------------------------------------------------------------
// Bounds of a step: |x| <= M for every singular value gives |a x + b x^3 + c x^5|
// <= next, and |b y + c y^2| <= poly for y = x^2.
struct Bounds {
    double next, poly;
};

__host__ __device__ inline Bounds step_bounds(double a, double b, double c, double M)
{
    auto p = [&](double x) { return fabs(x * (a + x * x * (b + c * x * x))); };
    auto q = [&](double y) { return fabs(y * (b + c * y)); };
    Bounds r{p(M), q(M * M)};
    // p' = a + 3 b y + 5 c y^2 at y = x^2; q' = b + 2 c y
    auto at = [&](double y) {
        if (y > 0.0 && y < M * M) r.next = fmax(r.next, p(sqrt(y)));
    };
    if (c != 0.0) {
        const double disc = 9.0 * b * b - 20.0 * a * c;
        if (disc >= 0.0) {
            at((-3.0 * b + sqrt(disc)) / (10.0 * c));
            at((-3.0 * b - sqrt(disc)) / (10.0 * c));
        }
        const double y = -b / (2.0 * c);
        if (y > 0.0 && y < M * M) r.poly = fmax(r.poly, q(y));
    } else if (b != 0.0) {
        at(-a / (3.0 * b));
    }
    return r;
}

// the power of two that takes `bound` to 2^14 .. 2^15 (1 for a zero or NaN bound)
__host__ __device__ inline double unit_of(double bound)
{
    if (!(bound > 0.0) || !(bound < 1e300)) return 1.0;
    int e;
    frexp(bound, &e);  // bound = f 2^e, f in [0.5, 1)
    return ldexp(1.0, 15 - e);
}

// Factors of one step's three products, from its operands' units to its results':
// A = gram * XX, B = sq * AA + lin * A, X' = mul * BX + add * X.
struct Units {
    float gram, sq, lin, mul, add;
};

// The steps' factors for a matrix whose first iterate's norm is at most r
// (below 1 only where eps exceeds the norm).
__host__ __device__ inline void step_units(const OrthoPoly& p, double r, Units* __restrict__ u)
{
    double M = r, kx = unit_of(r);
    for (int k = 0; k < p.steps; ++k) {
        const Bounds bd = step_bounds(p.a, p.b, p.c, M);
        const double ka = unit_of(M * M), kb = unit_of(bd.poly);
        const double kn = k + 1 < p.steps ? unit_of(bd.next) : (double)p.scale;
        u[k] = Units{(float)(ka / kx / kx), (float)(p.c * kb / ka / ka), (float)(p.b * kb / ka),
                     (float)(kn / kb / kx), (float)(p.a * kn / kx)};
        M = bd.next;
        kx = kn;
    }
}

// The factors for the bound 1, formed on the host: they serve every matrix
// whose norm is not below eps, so that the kernels need not wait for the fp64
// chain above (about 4 us).
struct UnitTable {
    Units u[kMaxOrthoSteps];
};

// A factor as a power of two and the rest, for elements whose magnitude and
// factor together stay in fp32's range although the factor alone may not.
struct Scale {
    float two, rest;
};

__device__ __forceinline__ Scale scale_of(double f)
{
    int e;
    frexp(f, &e);
    e = e < -120 ? -120 : e > 120 ? 120 : e;
    const double two = ldexp(1.0, e);
    return Scale{(float)two, (float)(f / two)};
}

// the bound that a matrix of norm r, at most 1, goes by
__device__ __forceinline__ double start_bound(double r) { return r > 0.5 ? 1.0 : r; }

// ---- norms and the first X ---------------------------------------------------------------
constexpr int kNormBlocks = 256;    // partial sums per matrix, at most
constexpr int kNormElems = 8192;    // elements per partial sum, about

// 2048 x 2048 fp32 5.6 us (3 TB/s), 4096 x 4096 22 us: one pass over G
template <class T>
__global__ void __launch_bounds__(kThreads) k_ortho_norm(int64_t size, int32_t per, bool wide,
                                                         const T* __restrict__ G, double* __restrict__ part)
{
    __shared__ double s[kThreads];
    constexpr int V = kWide<T>;
    const int64_t b = blockIdx.x / per, k = blockIdx.x % per;
    const int64_t each = ((size + per - 1) / per + V - 1) / V * V;
    const int64_t i0 = k * each, i1 = i0 + each < size ? i0 + each : size;
    const T* p = G + b * size;
    double t = 0.0;
    int64_t i = i0 + threadIdx.x * V;
    if (wide) {
#pragma unroll 4
        for (; i + V <= i1; i += kThreads * V) {
            float v[V];
            load_vec<T, V>(v, p + i);
#pragma unroll
            for (int j = 0; j < V; ++j) t += (double)v[j] * (double)v[j];
        }
    }
    for (; i < i1; i += kThreads * V)
        for (int64_t j = i; j < i + V && j < i1; ++j) t += (double)to_f32(p[j]) * (double)to_f32(p[j]);
    s[threadIdx.x] = t;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d /= 2) {
        if ((int)threadIdx.x < d) s[threadIdx.x] += s[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) part[blockIdx.x] = s[0];
}

// Frobenius norm of matrix b, by every wave
__device__ __forceinline__ double norm_of(const double* __restrict__ part, int64_t b, int32_t per)
{
    double t = 0.0;
    for (int32_t q = threadIdx.x & 63; q < per; q += 64) t += part[b * per + q];
#pragma unroll
    for (int d = 32; d > 0; d /= 2) t += __shfl_xor(t, d, 64);
    return sqrt(t);
}

// X and X^T of one 64 x 64 tile, split, zero outside the matrix; the first tile
// of a matrix leaves its steps' factors.  4096 x 4096 fp32 35 us: 67 MB read, 134 MB
// written (5.7 TB/s); 2048 x 2048 12.7 us
template <class T>
__global__ void __launch_bounds__(kThreads) k_ortho_first(OrthoDims d, OrthoPoly poly, UnitTable table,
                                                          int32_t per, const double* __restrict__ part,
                                                          const T* __restrict__ G, _Float16* __restrict__ X,
                                                          _Float16* __restrict__ Xt, Units* __restrict__ units)
{
    __shared__ float tile[64][65];
    const int64_t ti = d.sp / 64, tj = d.tp / 64;
    const int64_t b = blockIdx.x / (ti * tj), r = blockIdx.x % (ti * tj);
    const int64_t i0 = r / tj * 64, j0 = r % tj * 64;
    const double norm = norm_of(part, b, per), den = norm + (double)poly.eps;
    const double bound = start_bound(norm / den);
    const Scale inv = scale_of(unit_of(bound) / den);
    if (r == 0) {
        if (bound == 1.0) {
            if ((int)threadIdx.x < poly.steps) units[b * poly.steps + threadIdx.x] = table.u[threadIdx.x];
        } else if (threadIdx.x == 0) {
            step_units(poly, bound, units + b * poly.steps);
        }
    }
    const T* g = G + b * d.s * d.t;
    // the loads stand outside any condition (outside the matrix at its first element)
    constexpr int kEach = 64 * 64 / kThreads;
    T v[kEach];
    auto row_col = [&](int k, int64_t& i, int64_t& j, int& a, int& c) {  // c runs along G's rows
        const int q = k * kThreads + (int)threadIdx.x;
        a = q / 64;
        c = q % 64;
        i = i0 + (d.tall ? c : a);
        j = j0 + (d.tall ? a : c);
        return i < d.s && j < d.t;
    };
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        int64_t i, j;
        int a, c;
        const bool in = row_col(k, i, j, a, c);
        v[k] = g[in ? (d.tall ? j * d.s + i : i * d.t + j) : 0];
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        int64_t i, j;
        int a, c;
        const bool in = row_col(k, i, j, a, c);
        tile[d.tall ? c : a][d.tall ? a : c] = in ? to_f32(v[k]) * inv.two * inv.rest : 0.0f;
    }
    __syncthreads();
    X += b * d.sp * d.tp * 2;
    Xt += b * d.sp * d.tp * 2;
    // eight k of a row at a time, both orientations
    for (int q = threadIdx.x; q < 64 * 64 / 8; q += kThreads) {
        const int c = q % 4 * 8 + q / 256 * 32, a = q / 4 % 64;
        h8 h, l, ht, lt;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            _Float16 u, v;
            split(tile[a][c + e], u, v);
            h[e] = u;
            l[e] = v;
            split(tile[c + e][a], u, v);
            ht[e] = u;
            lt[e] = v;
        }
        _Float16* p = X + split_at(i0 + a, j0 + c, d.sp);
        *reinterpret_cast<h8*>(p) = h;
        *reinterpret_cast<h8*>(p + 32) = l;
        p = Xt + split_at(j0 + a, i0 + c, d.tp);
        *reinterpret_cast<h8*>(p) = ht;
        *reinterpret_cast<h8*>(p + 32) = lt;
    }
}

// ---- products ----------------------------------------------------------------------------
enum : int { kGram = 0, kPoly = 1, kNext = 2, kLast = 3 };

struct ProdArgs {
    OrthoDims d;
    int64_t K;          // contraction length (padded)
    int64_t ti, tj;     // tiles along i and j; tj = 0: the upper triangle of ti x ti
    const _Float16 *P, *Q;
    const _Float16* E;  // kPoly: A; kNext, kLast: X^T (rows j)
    _Float16 *R, *Rt;   // results, [i][j] and [j][i]
    void* out;          // kLast: O in G's layout
    const Units* units; // this step's factors, `steps` apart for each matrix
    int32_t steps;
};

// Tile `r` of a product of ti x tj tiles (tj = 0: the upper triangle, bi <= bj),
// counted through bands of four columns, row by row within a band, so that
// consecutive tiles share operands.
__device__ __forceinline__ void tile_at(int64_t r, int64_t ti, int64_t tj, int64_t& bi, int64_t& bj)
{
    constexpr int64_t kBand = 4;
    const bool upper = tj == 0;
    const int64_t cols = upper ? ti : tj;
    int64_t c0 = 0, w = 0, n = 0;
    for (;; c0 += kBand, r -= n) {
        w = cols - c0 < kBand ? cols - c0 : kBand;
        n = upper ? w * c0 + w * (w + 1) / 2 : w * ti;
        if (r < n) break;
    }
    const int64_t full = upper ? c0 : ti;  // rows with all w columns
    if (r < full * w) {
        bi = r / w;
        bj = c0 + r % w;
        return;
    }
    r -= full * w;  // the band's own triangle
    bi = c0;
    while (r >= c0 + w - bi) {
        r -= c0 + w - bi;
        ++bi;
    }
    bj = bi + r;
}

// Blocks go to the XCDs in turn: block x works on tile (x % kXcds) * (n / kXcds)
// + x / kXcds (the first n % kXcds XCDs one more), so that an XCD's tiles are
// neighbours and share its L2.
__device__ __forceinline__ int64_t xcd_order(int64_t x, int64_t n)
{
    const int64_t q = n / kXcds, rest = n % kXcds, c = x % kXcds;
    return c * q + (c < rest ? c : rest) + x / kXcds;
}

// All but the last N of this wave's loads have arrived, its LDS reads are done,
// and every wave of the block is here.  (The counters' wait as a builtin, so that
// the compiler knows of it; the barrier holds memory accesses on their side.)
template <int N>
__device__ __forceinline__ void wait_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);  // vmcnt(N) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
}

// One TILE x TILE tile of D = P Q^T, each wave WX x WY tiles of 32 x 32, 32 k at
// a time through a ring of kStages LDS buffers that loads fill directly, kStages
// blocks of k ahead.  Two waves per SIMD (TILE 128) keep the matrix cores busy
// across the barriers of a block of k.  Bound by the matrix cores: a full product of
// 4096 x 4096 x 4096 (X') takes 404 us, 1.02 PFLOP/s of fp16 products where a library's
// large fp16 product reaches 1.15; A and B, by their upper triangle, 255 and 260 us.
// At 2048 X' fills the 256 compute units once (57 us, 0.90 PFLOP/s), and the 136 tiles
// of A and B leave half of them idle (45 us): equal shares of all 136 tiles' blocks of k
// for 256 blocks, joined by a tile's last to arrive, were slower all the same (five steps
// 733 against 698 us, at 4096 4.72 against 4.32 ms).  Two stages instead of four: 477
// against 382 us a product at 4096.
template <int TILE>
struct TileShape;
template <>
struct TileShape<128> {
    static constexpr int WX = 2, WY = 1;
};
template <>
struct TileShape<64> {
    static constexpr int WX = 1, WY = 1;
};
template <int TILE>
constexpr int kProdThreads = 64 * (TILE / 32 / TileShape<TILE>::WX) * (TILE / 32 / TileShape<TILE>::WY);

template <int TILE, int KIND, class T>
__global__ void __launch_bounds__(kProdThreads<TILE>) k_ortho_prod(ProdArgs a)
{
    constexpr int WX = TileShape<TILE>::WX, WY = TileShape<TILE>::WY, kThr = kProdThreads<TILE>;
    constexpr int kRowHalves = 64, kStages = 4;
    constexpr int kPieces = TILE * 8 / kThr;  // 16-byte pieces per thread, operand and stage
    constexpr int kLd = TILE + 4;             // row stride of the result in LDS
    constexpr int kRing = kStages * 2 * TILE * kRowHalves * 2, kResult = TILE * kLd * 4;
    __shared__ __attribute__((aligned(16))) char mem[kRing > kResult ? kRing : kResult];
    auto lds = reinterpret_cast<_Float16(*)[2][TILE * kRowHalves]>(mem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t tiles = a.tj == 0 ? a.ti * (a.ti + 1) / 2 : a.ti * a.tj;
    const int64_t x = xcd_order(blockIdx.x, gridDim.x), b = x / tiles;
    int64_t bi, bj;
    tile_at(x % tiles, a.ti, a.tj, bi, bj);
    const OrthoDims& d = a.d;
    const int64_t rowsP = d.sp, rowsQ = KIND == kNext || KIND == kLast ? d.tp : d.sp;
    const _Float16* P = a.P + b * rowsP * a.K * 2 + bi * TILE * kRowHalves;
    const _Float16* Q = a.Q + b * rowsQ * a.K * 2 + bj * TILE * kRowHalves;

    f16v acc[WX][WY];
#pragma unroll
    for (int x = 0; x < WX; ++x)
#pragma unroll
        for (int y = 0; y < WY; ++y)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[x][y][q] = 0.0f;

    // Thread p of a stage fills piece p % 8 of row p / 8, with the row's piece
    // (p % 8) ^ (row / 2 % 8): a wave's LDS destination is one run of 1 KB, and
    // the reads of sixteen rows at one k spread over all 64 banks.
    const uint32_t mine = (uint32_t)((tid / 8) * 128 + (((tid % 8) ^ ((tid / 16) & 7)) * 16));
    auto fill = [&](int64_t kb) {
        _Float16(*to)[TILE * kRowHalves] = lds[kb % kStages];
        const char* pp = (const char*)(P + kb * rowsP * kRowHalves);
        const char* qq = (const char*)(Q + kb * rowsQ * kRowHalves);
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int at = (q * kThr + wave * 64) * 8;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void*)(pp + (uint32_t)(mine + q * kThr * 16)),
                (__attribute__((address_space(3))) void*)&to[0][at], 16, 0, 0);
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void*)(qq + (uint32_t)(mine + q * kThr * 16)),
                (__attribute__((address_space(3))) void*)&to[1][at], 16, 0, 0);
        }
    };
    constexpr int kAcross = TILE / 32 / WY;  // waves along j
    const int wi = wave / kAcross * 32 * WX, wj = wave % kAcross * 32 * WY;
    const int64_t nk = a.K / 32;
    // operands of one block of k in registers
    struct Frag {
        h8 ph[2][WX], pl[2][WX], qh[2][WY], ql[2][WY];
    };
    auto read = [&](Frag& f, int64_t kb) {
        const _Float16(*from)[TILE * kRowHalves] = lds[kb % kStages];
        auto at = [&](int op, int row, int piece) {
            return *reinterpret_cast<const h8*>(&from[op][row * kRowHalves + ((piece ^ ((row >> 1) & 7)) * 8)]);
        };
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int piece = ks * 2 + (lane >> 5);
#pragma unroll
            for (int x = 0; x < WX; ++x) f.ph[ks][x] = at(0, wi + 32 * x + (lane & 31), piece);
#pragma unroll
            for (int y = 0; y < WY; ++y) f.ql[ks][y] = at(1, wj + 32 * y + (lane & 31), piece + 4);
#pragma unroll
            for (int x = 0; x < WX; ++x) f.pl[ks][x] = at(0, wi + 32 * x + (lane & 31), piece + 4);
#pragma unroll
            for (int y = 0; y < WY; ++y) f.qh[ks][y] = at(1, wj + 32 * y + (lane & 31), piece);
        }
    };
    auto multiply = [&](const Frag& f) {
        auto add = [&](const h8(&p)[WX], const h8(&q)[WY]) {
#pragma unroll
            for (int x = 0; x < WX; ++x)
#pragma unroll
                for (int y = 0; y < WY; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(p[x], q[y], acc[x][y], 0, 0, 0);
        };
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            add(f.ph[ks], f.ql[ks]);
            add(f.pl[ks], f.qh[ks]);
            add(f.ph[ks], f.qh[ks]);
        }
        // first the next block's LDS reads, then the loads, between the products
        constexpr int kReads = 4 * (WX + WY), kMul = 6 * WX * WY;
#pragma unroll
        for (int g = 0; g < kMul / 2; ++g) {
            __builtin_amdgcn_sched_group_barrier(0x100, (kReads + kMul / 2 - 1) / (kMul / 2), 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
#pragma unroll
        for (int g = 0; g < kMul / 2; ++g) {
            __builtin_amdgcn_sched_group_barrier(0x010, (2 * kPieces + kMul / 2 - 1) / (kMul / 2), 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
    };
    // Step kb multiplies block kb, already in registers, while it reads block
    // kb + 1 from LDS and starts the loads of block kb + kStages into the buffer
    // that block kb has left.  Block kb + 1 is in when at most the kStages - 2
    // blocks after it are out; behind the barrier every wave has read block kb.
    auto main_step = [&](int64_t kb, const Frag& cur, Frag& next) {
        wait_barrier<2 * kPieces*(kStages - 2)>();
        read(next, kb + 1);
        fill(kb + kStages);
        multiply(cur);
    };
    auto tail_step = [&](int64_t kb, const Frag& cur, Frag& next) {
        if (kb + 1 < nk) {
            wait_barrier<0>();
            read(next, kb + 1);
            if (kb + kStages < nk) fill(kb + kStages);
        }
        multiply(cur);
    };
    Frag f0, f1;
    for (int64_t kb = 0; kb < kStages && kb < nk; ++kb) fill(kb);
    wait_barrier<0>();
    read(f0, 0);
    int64_t kb = 0;
    for (; kb + 1 + kStages < nk; kb += 2) {
        main_step(kb, f0, f1);
        main_step(kb + 1, f1, f0);
    }
    for (; kb < nk; kb += 2) {
        tail_step(kb, f0, f1);
        if (kb + 1 < nk) tail_step(kb + 1, f1, f0);
    }

    // The result goes through LDS as s[j][i], so that both orientations leave in
    // whole lines.  A lane holds column j = lane % 32, rows 8 (q / 4) + 4 (lane /
    // 32) + q % 4 of each tile of 32.
    const Units u = a.units[b * a.steps];
    const float alpha = KIND == kGram ? u.gram : KIND == kPoly ? u.sq : u.mul;
    const float beta = KIND == kPoly ? u.lin : u.add;
    float* s = reinterpret_cast<float*>(mem);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < WX; ++x)
#pragma unroll
        for (int y = 0; y < WY; ++y)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float4 v;
                v.x = alpha * acc[x][y][4 * g];
                v.y = alpha * acc[x][y][4 * g + 1];
                v.z = alpha * acc[x][y][4 * g + 2];
                v.w = alpha * acc[x][y][4 * g + 3];
                *reinterpret_cast<float4*>(
                    &s[(wj + 32 * y + (lane & 31)) * kLd + wi + 32 * x + 8 * g + 4 * (lane >> 5)]) = v;
            }
    __syncthreads();
    const int64_t of = b * rowsP * rowsQ * 2;  // this matrix in E, R and Rt
    constexpr int kEights = TILE * TILE / 8;
    // rows j, eight i at a time: add E and write R^T
    if constexpr (KIND != kGram) {
        for (int q = tid; q < kEights; q += kThr) {
            const int c = q % 4, j = q / 4 % TILE, i = q / (4 * TILE) * 32 + 8 * c;
            float* v = &s[j * kLd + i];
            const int64_t at = of + split_at(bj * TILE + j, bi * TILE + i, rowsQ);
            const h8 eh = *reinterpret_cast<const h8*>(a.E + at), el = *reinterpret_cast<const h8*>(a.E + at + 32);
            h8 vh, vl;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] += beta * ((float)eh[e] + (float)el[e]);
                _Float16 h, l;
                split(v[e], h, l);
                vh[e] = h;
                vl[e] = l;
            }
            // the diagonal tile of a symmetric result is written below
            if (KIND == kNext || (KIND == kPoly && bi != bj)) {
                *reinterpret_cast<h8*>(a.Rt + at) = vh;
                *reinterpret_cast<h8*>(a.Rt + at + 32) = vl;
            }
        }
        __syncthreads();
    }
    if constexpr (KIND == kLast) {
        T* o = (T*)a.out + b * d.s * d.t;
        for (int q = tid; q < TILE * TILE; q += kThr) {
            // the output's own rows
            const int i = d.tall ? q % TILE : q / TILE, j = d.tall ? q / TILE : q % TILE;
            const int64_t gi = bi * TILE + i, gj = bj * TILE + j;
            if (gi < d.s && gj < d.t) o[d.tall ? gj * d.s + gi : gi * d.t + gj] = from_f32<T>(s[j * kLd + i]);
        }
    } else {
        // rows i, eight j at a time: write R; of a symmetric result's diagonal
        // tile the upper triangle decides, and off the diagonal its mirror too
        for (int q = tid; q < kEights; q += kThr) {
            const int c = q % 4, i = q / 4 % TILE, j = q / (4 * TILE) * 32 + 8 * c;
            h8 vh, vl;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool flip = KIND != kNext && bi == bj && i > j + e;
                _Float16 h, l;
                split(flip ? s[i * kLd + j + e] : s[(j + e) * kLd + i], h, l);
                vh[e] = h;
                vl[e] = l;
            }
            const int64_t at = of + split_at(bi * TILE + i, bj * TILE + j, rowsP);
            *reinterpret_cast<h8*>(a.R + at) = vh;
            *reinterpret_cast<h8*>(a.R + at + 32) = vl;
        }
        if constexpr (KIND == kGram) {
            if (bi != bj)
                for (int q = tid; q < kEights; q += kThr) {
                    const int c = q % 4, j = q / 4 % TILE, i = q / (4 * TILE) * 32 + 8 * c;
                    h8 vh, vl;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        _Float16 h, l;
                        split(s[j * kLd + i + e], h, l);
                        vh[e] = h;
                        vl[e] = l;
                    }
                    const int64_t at = of + split_at(bj * TILE + j, bi * TILE + i, rowsQ);
                    *reinterpret_cast<h8*>(a.Rt + at) = vh;
                    *reinterpret_cast<h8*>(a.Rt + at + 32) = vl;
                }
        }
    }
}

// ---- short sides of at most 16 -------------------------------------------------------------
// A block holds a matrix as fp32 in LDS, s rows of `ld` elements, and works in fp64
// (v_mfma_f64_16x16x4: A[i][k] in lane i + 16 k, B[k][j] in lane j + 16 k, D[i][j] in
// element i / 4 of lane j + 16 (i % 4)).  A wave keeps to its own tiles of 16 columns:
// the next X of a tile needs B and that tile alone, and the operand element m of a
// lane, X[4 m + lane / 16][lane % 16], is the element that its D element m replaces.
// Only the sum of A crosses waves.  No units: fp64 and fp32 hold every magnitude.
// Bound by the chain of dependent products and barriers: 200 of 12 x 50, five steps, 16 us.
constexpr int kTinySide = 16, kTinyWaves = 8, kTinyElems = 32768;
typedef double d4 __attribute__((ext_vector_type(4)));

struct TinyArgs {
    OrthoDims d;  // sp, tp unused
    OrthoPoly poly;
    int32_t ld;
    const void* G;
    void* out;
};

extern __shared__ __attribute__((aligned(16))) float tiny_lds[];

template <class T>
__global__ void __launch_bounds__(64 * kTinyWaves) k_ortho_tiny(TinyArgs a)
{
    __shared__ double parts[kTinyWaves][256], A[256], norms[kTinyWaves];
    float* X = tiny_lds;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int s = (int)a.d.s, t = (int)a.d.t, ld = a.ld, c = lane & 15, r4 = lane >> 4;
    const T* g = (const T*)a.G + (int64_t)blockIdx.x * s * t;
    double sum = 0.0;
    for (int q = tid; q < s * t; q += 64 * kTinyWaves) {
        const float v = to_f32(g[q]);
        sum += (double)v * (double)v;
        X[a.d.tall ? q % s * ld + q / s : q / t * ld + q % t] = v;
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) norms[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kTinyWaves; ++w) sum += norms[w];
    const double inv = 1.0 / (sqrt(sum) + (double)a.poly.eps);
    // a row or column outside the matrix reads its first element and counts as zero
    auto at = [&](int row, int col) { return (double)X[row < s && col < t ? row * ld + col : 0]; };
    auto in = [&](int row, int col) { return row < s && col < t; };
    for (int j0 = 16 * wave; j0 < t; j0 += 16 * kTinyWaves)  // the first X
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int row = 4 * m + r4, col = j0 + c;
            const double v = at(row, col) * inv;
            if (in(row, col)) X[row * ld + col] = (float)v;
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int k = 0; k < a.poly.steps; ++k) {
        const bool last = k + 1 == a.poly.steps;
        d4 acc = {0.0, 0.0, 0.0, 0.0};
        for (int j0 = 16 * wave; j0 < t; j0 += 16 * kTinyWaves)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int col = j0 + 4 * m + r4;
                const double v = in(c, col) ? at(c, col) : 0.0;
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(v, v, acc, 0, 0, 0);
            }
#pragma unroll
        for (int m = 0; m < 4; ++m) parts[wave][(4 * m + r4) * 16 + c] = acc[m];
        __syncthreads();
        if (tid < 256) {
            double v = 0.0;
#pragma unroll
            for (int w = 0; w < kTinyWaves; ++w) v += parts[w][tid];
            A[tid] = v;
        }
        __syncthreads();
        // every wave forms B, each for itself: in D's layout, then as an operand by way of its part
        acc = d4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int m = 0; m < 4; ++m)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64(A[c * 16 + 4 * m + r4], A[(4 * m + r4) * 16 + c], acc, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int e = (4 * m + r4) * 16 + c;
            parts[wave][e] = a.poly.b * A[e] + a.poly.c * acc[m];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        double bk[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) bk[m] = parts[wave][c * 16 + 4 * m + r4];
        T* o = (T*)a.out + (int64_t)blockIdx.x * s * t;
        for (int j0 = 16 * wave; j0 < t; j0 += 16 * kTinyWaves) {
            double x[4];
            acc = d4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                x[m] = in(4 * m + r4, j0 + c) ? at(4 * m + r4, j0 + c) : 0.0;
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(bk[m], x[m], acc, 0, 0, 0);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int row = 4 * m + r4, col = j0 + c;
                const double v = a.poly.a * x[m] + acc[m];
                if (!in(row, col)) continue;
                if (last) o[a.d.tall ? col * s + row : row * t + col] = from_f64<T>(v * (double)a.poly.scale);
                else X[row * ld + col] = (float)v;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// ---- short sides of at most 128 ------------------------------------------------------------
// One block holds a matrix (or its chunk of TP columns, s <= SP) in LDS through
// all three products of a step: X split in 64 KB at most, A and then B in another
// 64 KB.  A step is 3 x 2 SP^2 TP flops and five barriers instead of three launches.
// The next X is formed transposed, D[t][s] = sum_k X[k][t] B[s][k], so that a
// lane ends with four consecutive t of a row of X and writes them back at once;
// X^T is read from X's rows by transposing LDS reads.  Bound by one compute unit's matrix
// cores and its LDS: 15 of 128 x 128 fp32, five steps, 42.8 us (8.5 us a step, of which the
// products take 3.9 us at the cores' peak); 100 of 64 x 64 15.4 us.
template <int SP, int TP>
struct Small {
    static constexpr int WC = SP / 32, NW = SP == 128 ? 8 : 4, WR = NW / WC;  // waves along the columns and rows
    static constexpr int GX = SP / 32 / WR, NX = TP / 32 / WR;               // 32 x 32 tiles per wave, A and X
    static constexpr int kThr = 64 * NW;
    static constexpr int kX = SP * TP * 2, kA = SP * SP * 2;  // halves
    static constexpr int kTileFloats = GX * 16 * kThr;          // A by threads: SP * SP
};

struct SmallArgs {
    OrthoDims d;  // sp, tp unused
    OrthoPoly poly;
    UnitTable table;
    bool wide;
    const void* G;
    void* out;
};

typedef short s4v __attribute__((ext_vector_type(4)));
typedef _Float16 h4v __attribute__((ext_vector_type(4)));

template <int SP, int TP>
struct SmallOps {
    using S = Small<SP, TP>;
    _Float16 *X, *A;
    int lane, wi, wj, wt;  // wave's first row of A, column, first t
    // The lane's offsets (halves), formed once: rows begin at multiples of 32, so
    // that the swizzle depends on the lane alone.
    int at[4];  // pieces 2 ks + lane / 32 (+ 4) of row lane % 32, by ks + 2 low
    int tr[4];  // transposing reads, by first row 0 or 4, + 2 low

    __device__ __forceinline__ SmallOps(_Float16* x, _Float16* a) : X(x), A(a)
    {
        lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wi = wave / S::WC * 32 * S::GX;
        wt = wave / S::WC * 32 * S::NX;
        wj = wave % S::WC * 32;
        const int r = lane & 31, hf = lane >> 5, l = lane & 15, half16 = (lane >> 4) & 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            at[q] = place_of(0, 0, r, ((q & 1) * 2 + hf) + (q >> 1) * 4);
            // lanes of 16 hold rows t0 + lane % 16, four k each; each lane points
            // at 8 bytes of row k + lane % 16 / 4 of X
            tr[q] = place_of(0, 0, 8 * hf + 4 * (q & 1) + (l >> 2), 2 * half16 + ((l & 3) >> 1) + (q >> 1) * 4) + 4 * (l & 1);
        }
    }
    // halves offset of 16-byte piece c (0..7) of row r in block kb; an operand of `rows` rows
    static __device__ __forceinline__ int place_of(int rows, int kb, int r, int c)
    {
        return (kb * rows + r) * 64 + ((c ^ ((r >> 1) & 7)) * 8);
    }
    template <int N>
    static __device__ __forceinline__ void clear(f16v (&acc)[N])
    {
#pragma unroll
        for (int x = 0; x < N; ++x)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[x][q] = 0.0f;
    }
    // acc[x] += three products of p[x] and q
    template <int N>
    static __device__ __forceinline__ void multiply(const h8 (&ph)[N], const h8 (&pl)[N], h8 qh, h8 ql, f16v (&acc)[N])
    {
#pragma unroll
        for (int x = 0; x < N; ++x) acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[x], ql, acc[x], 0, 0, 0);
#pragma unroll
        for (int x = 0; x < N; ++x) acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[x], qh, acc[x], 0, 0, 0);
#pragma unroll
        for (int x = 0; x < N; ++x) acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[x], qh, acc[x], 0, 0, 0);
    }
    // acc[x] += sum_k p[row wi + 32 x ..][k] p[row wj ..][k], k over blocks of 32
    template <int BLOCKS, int N>
    __device__ __forceinline__ void square(const _Float16* p, f16v (&acc)[N]) const
    {
        const _Float16 *pi = p + wi * 64, *pj = p + wj * 64;
#pragma unroll
        for (int kb = 0; kb < BLOCKS; ++kb)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const h8 qh = *reinterpret_cast<const h8*>(pj + at[ks] + kb * SP * 64);
                const h8 ql = *reinterpret_cast<const h8*>(pj + at[ks + 2] + kb * SP * 64);
                h8 ph[N], pl[N];
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    ph[x] = *reinterpret_cast<const h8*>(pi + at[ks] + (kb * SP + 32 * x) * 64);
                    pl[x] = *reinterpret_cast<const h8*>(pi + at[ks + 2] + (kb * SP + 32 * x) * 64);
                }
                multiply(ph, pl, qh, ql, acc);
            }
    }
    // four k of X^T's rows
    __device__ __forceinline__ h4v transposed(const _Float16* p) const
    {
        const s4v v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4v*)const_cast<_Float16*>(p));
        return __builtin_bit_cast(h4v, v);
    }
    // acc[x][..] = sum_k X[k][wt + 32 x ..] B[wj ..][k], B in A's place
    __device__ __forceinline__ void next(f16v (&acc)[S::NX]) const
    {
        clear(acc);
        const _Float16 *pt = X + (wt >> 5) * SP * 64, *pj = A + wj * 64;
#pragma unroll
        for (int kb = 0; kb < SP / 32; ++kb)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const h8 qh = *reinterpret_cast<const h8*>(pj + at[ks] + kb * SP * 64);
                const h8 ql = *reinterpret_cast<const h8*>(pj + at[ks + 2] + kb * SP * 64);
                h8 ph[S::NX], pl[S::NX];
#pragma unroll
                for (int x = 0; x < S::NX; ++x) {
                    const _Float16* p = pt + (x * SP + kb * 32 + ks * 16) * 64;
                    ph[x] = __builtin_shufflevector(transposed(p + tr[0]), transposed(p + tr[1]), 0, 1, 2, 3, 4, 5, 6, 7);
                    pl[x] = __builtin_shufflevector(transposed(p + tr[2]), transposed(p + tr[3]), 0, 1, 2, 3, 4, 5, 6, 7);
                }
                multiply(ph, pl, qh, ql, acc);
            }
    }
    // the lane's four values g of block kb (low half: + 4) in row wj + lane % 32
    __device__ __forceinline__ int four_at(int kb, int g) const
    {
        return place_of(SP, kb, lane & 31, g) + 4 * (lane >> 5);
    }
    // rows v[x][4 g .. 4 g + 3] at first + 32 x + 8 g + 4 (lane / 32) of column wj + lane % 32,
    // written as that row of p
    template <int N>
    __device__ __forceinline__ void put(_Float16* p, const f16v (&v)[N], int first) const
    {
        p += (wj + (first >> 5) * SP) * 64;
#pragma unroll
        for (int x = 0; x < N; ++x)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                h4v h, l;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    _Float16 a, b;
                    split(v[x][4 * g + q], a, b);
                    h[q] = a;
                    l[q] = b;
                }
                *reinterpret_cast<h4v*>(p + four_at(x, g)) = h;
                *reinterpret_cast<h4v*>(p + four_at(x, g + 4)) = l;
            }
    }
    // the lane's values of X, as put() left them
    __device__ __forceinline__ void get(f16v (&v)[S::NX]) const
    {
        const _Float16* p = X + (wj + (wt >> 5) * SP) * 64;
#pragma unroll
        for (int x = 0; x < S::NX; ++x)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const h4v h = *reinterpret_cast<const h4v*>(p + four_at(x, g));
                const h4v l = *reinterpret_cast<const h4v*>(p + four_at(x, g + 4));
#pragma unroll
                for (int q = 0; q < 4; ++q) v[x][4 * g + q] = (float)h[q] + (float)l[q];
            }
    }
    // A (its values in ar) to B in A's place; two barriers inside, one owed after
    __device__ __forceinline__ void poly(f16v (&ar)[S::GX], const Units& u) const
    {
        put(A, ar, wi);
        __syncthreads();
        f16v acc[S::GX];
        clear(acc);
        square<SP / 32>(A, acc);
#pragma unroll
        for (int x = 0; x < S::GX; ++x)
#pragma unroll
            for (int q = 0; q < 16; ++q) ar[x][q] = u.sq * acc[x][q] + u.lin * ar[x][q];
        __syncthreads();
        put(A, ar, wi);
    }
    // columns t0 .. t0 + TP of matrix g, zero outside: the thread's elements,
    // eight along G's rows each (wide: G's rows are whole 16-byte accesses)
    static constexpr int kEights = SP * TP / 8 / S::kThr;
    // row i of X and column j of the thread's k-th eight's first element
    static __device__ __forceinline__ int row_of(const OrthoDims& d, int k)
    {
        const int q = k * S::kThr + (int)threadIdx.x;
        return d.tall ? q % (SP / 8) * 8 : q / (TP / 8);
    }
    static __device__ __forceinline__ int col_of(const OrthoDims& d, int k)
    {
        const int q = k * S::kThr + (int)threadIdx.x;
        return d.tall ? q / (SP / 8) : q % (TP / 8) * 8;
    }
    static __device__ __forceinline__ int64_t offset(const OrthoDims& d, int64_t t0, int k)
    {
        const int64_t i = row_of(d, k), j = t0 + col_of(d, k);
        return d.tall ? j * d.s + i : i * d.t + j;
    }
    // whether the eight's element e is in the matrix
    static __device__ __forceinline__ bool inside(const OrthoDims& d, int64_t t0, int k, int e)
    {
        const int64_t i = row_of(d, k), j = t0 + col_of(d, k);
        return d.tall ? j < d.t && i + e < d.s : i < d.s && j + e < d.t;
    }
    template <class T>
    __device__ __forceinline__ void fetch(const OrthoDims& d, const T* __restrict__ g, int64_t t0, bool wide,
                                          float (&v)[kEights][8]) const
    {
        // loads stand outside any condition (outside the matrix at its first
        // element), so that all of them are in flight together
        if (wide) {
            constexpr int V = kWide<T>;
            float f[kEights][8 / V][V];
#pragma unroll
            for (int k = 0; k < kEights; ++k)
#pragma unroll
                for (int e = 0; e < 8 / V; ++e)
                    load_vec<T, V>(f[k][e], g + (inside(d, t0, k, e * V) ? offset(d, t0, k) + e * V : 0));
#pragma unroll
            for (int k = 0; k < kEights; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k][e] = inside(d, t0, k, e / V * V) ? f[k][e / V][e % V] : 0.0f;
        } else {
#pragma unroll
            for (int k = 0; k < kEights; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k][e] = to_f32(g[inside(d, t0, k, e) ? offset(d, t0, k) + e : 0]);
#pragma unroll
            for (int k = 0; k < kEights; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k][e] = inside(d, t0, k, e) ? v[k][e] : 0.0f;
        }
    }
    // those elements times the scale, split, to X
    __device__ __forceinline__ void place(const OrthoDims& d, const float (&v)[kEights][8], Scale k) const
    {
#pragma unroll
        for (int e8 = 0; e8 < kEights; ++e8) {
            const int i = row_of(d, e8), j = col_of(d, e8);
            h8 h, l;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                _Float16 a, b;
                split(v[e8][e] * k.two * k.rest, a, b);
                h[e] = a;
                l[e] = b;
            }
            if (!d.tall) {
                *reinterpret_cast<h8*>(X + place_of(SP, j >> 5, i, (j & 31) >> 3)) = h;
                *reinterpret_cast<h8*>(X + place_of(SP, j >> 5, i, ((j & 31) >> 3) + 4)) = l;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    X[place_of(SP, j >> 5, i + e, (j & 31) >> 3) + (j & 7)] = h[e];
                    X[place_of(SP, j >> 5, i + e, ((j & 31) >> 3) + 4) + (j & 7)] = l[e];
                }
            }
        }
    }
    // the lane's values of the last X to the output
    template <class T>
    __device__ __forceinline__ void store(const OrthoDims& d, T* __restrict__ o, int64_t t0, bool wide,
                                          const f16v (&v)[S::NX]) const
    {
        const int64_t i = wj + (lane & 31);
        if (i >= d.s) return;
#pragma unroll
        for (int x = 0; x < S::NX; ++x)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int64_t j = t0 + wt + 32 * x + 8 * g + 4 * (lane >> 5);
                if (wide && !d.tall) {  // t is a multiple of four
                    struct alignas(4 * sizeof(T)) Four {
                        T e[4];
                    } w;
#pragma unroll
                    for (int q = 0; q < 4; ++q) w.e[q] = from_f32<T>(v[x][4 * g + q]);
                    if (j < d.t) *reinterpret_cast<Four*>(o + i * d.t + j) = w;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (j + q < d.t) o[d.tall ? (j + q) * d.s + i : i * d.t + j + q] = from_f32<T>(v[x][4 * g + q]);
                }
            }
    }
};

// A whole matrix per block (t <= TP), norm to output.
template <int SP, int TP, class T>
__global__ void __launch_bounds__((Small<SP, TP>::kThr)) k_ortho_small(SmallArgs a)
{
    using S = Small<SP, TP>;
    __shared__ __attribute__((aligned(16))) _Float16 X[S::kX], A[S::kA];
    __shared__ Units units[kMaxOrthoSteps];
    __shared__ double norms[S::NW];
    const SmallOps<SP, TP> ops(X, A);
    const int64_t size = a.d.s * a.d.t;
    const T* g = (const T*)a.G + blockIdx.x * size;
    float v[SmallOps<SP, TP>::kEights][8];
    ops.fetch(a.d, g, 0, a.wide, v);
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < SmallOps<SP, TP>::kEights; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)v[k][e] * (double)v[k][e];
#pragma unroll
    for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d, 64);
    if ((threadIdx.x & 63) == 0) norms[threadIdx.x >> 6] = sum;
    if ((int)threadIdx.x < a.poly.steps) units[threadIdx.x] = a.table.u[threadIdx.x];
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < S::NW; ++w) sum += norms[w];
    const double norm = sqrt(sum), den = norm + (double)a.poly.eps, bound = start_bound(norm / den);
    if (bound != 1.0 && threadIdx.x == 0) step_units(a.poly, bound, units);
    ops.place(a.d, v, scale_of(unit_of(bound) / den));
    __syncthreads();
    f16v xr[S::NX], ar[S::GX], acc[S::NX];
    ops.get(xr);
    for (int k = 0; k < a.poly.steps; ++k) {
        const Units u = units[k];
        ops.clear(ar);
        ops.template square<TP / 32>(X, ar);
#pragma unroll
        for (int x = 0; x < S::GX; ++x)
#pragma unroll
            for (int q = 0; q < 16; ++q) ar[x][q] *= u.gram;
        ops.poly(ar, u);
        __syncthreads();
        ops.next(acc);
#pragma unroll
        for (int x = 0; x < S::NX; ++x)
#pragma unroll
            for (int q = 0; q < 16; ++q) xr[x][q] = u.mul * acc[x][q] + u.add * xr[x][q];
        if (k + 1 == a.poly.steps) break;
        __syncthreads();
        ops.put(X, xr, ops.wt);
        __syncthreads();
    }
    ops.store(a.d, (T*)a.out + blockIdx.x * size, 0, a.wide, xr);
}

// ---- a short side of at most 128, the other longer -------------------------------------------
// A matrix's chunks of TP columns are dealt to `blocks` blocks.  A launch per step, and
// one that adds the partial A where they are many (15 of 128 x 1024 bf16: 16.3 and 4.3 us,
// bound by launches and by each block's own three products; the first X with its A takes
// 12.2 us): every block adds the partial A = X X^T of all blocks, forms B (the same
// work in each, in parallel), takes its chunks of X, held in memory as they lie
// in LDS, through X <- a X + B X, and leaves its partial A of the new X.
struct WideArgs {
    OrthoDims d;  // sp, tp unused
    OrthoPoly poly;
    int64_t chunks;     // of a matrix
    int32_t blocks;     // per matrix
    bool wide;
    const void* G;
    void* out;
    Units* units;       // [batch][steps]
    _Float16* image;    // [batch][chunks] X as in LDS
    const float* sums;  // [batch][nsums] partial A, by threads
    float* osums;       // [batch][blocks]
    int32_t nsums, step;
};

// A's values by threads: four at a time, the block's threads in a row
template <int SP, int TP>
__device__ __forceinline__ void put_sums(float* __restrict__ p, const f16v (&v)[Small<SP, TP>::GX])
{
    using S = Small<SP, TP>;
    float4* o = reinterpret_cast<float4*>(p) + threadIdx.x;
#pragma unroll
    for (int x = 0; x < S::GX; ++x)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            o[(x * 4 + g) * S::kThr] = make_float4(v[x][4 * g], v[x][4 * g + 1], v[x][4 * g + 2], v[x][4 * g + 3]);
}

template <int SP, int TP>
__device__ __forceinline__ void add_sums(const float* __restrict__ p, f16v (&v)[Small<SP, TP>::GX])
{
    using S = Small<SP, TP>;
    const float4* o = reinterpret_cast<const float4*>(p) + threadIdx.x;
#pragma unroll
    for (int x = 0; x < S::GX; ++x)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 f = o[(x * 4 + g) * S::kThr];
            v[x][4 * g] += f.x;
            v[x][4 * g + 1] += f.y;
            v[x][4 * g + 2] += f.z;
            v[x][4 * g + 3] += f.w;
        }
}

template <int SP, int TP>
__device__ __forceinline__ void put_image(_Float16* __restrict__ to, const _Float16* X)
{
    using S = Small<SP, TP>;
#pragma unroll
    for (int q = 0; q < S::kX / 8 / S::kThr; ++q) {
        const int at = (q * S::kThr + (int)threadIdx.x) * 8;
        *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(X + at);
    }
}

// starts the loads of a chunk's image; in when vmcnt says so
template <int SP, int TP>
__device__ __forceinline__ void load_image(const _Float16* __restrict__ from, _Float16* X)
{
    using S = Small<SP, TP>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int q = 0; q < S::kX / 8 / S::kThr; ++q)
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(from + (q * S::kThr + (int)threadIdx.x) * 8),
            (__attribute__((address_space(3))) void*)(X + (q * S::kThr + wave * 64) * 8), 16, 0, 0);
}

// the first X, split, and its partial A
template <int SP, int TP, class T>
__global__ void __launch_bounds__((Small<SP, TP>::kThr)) k_ortho_wide_first(WideArgs a, UnitTable table, int32_t per,
                                                                            const double* __restrict__ part)
{
    using S = Small<SP, TP>;
    __shared__ __attribute__((aligned(16))) _Float16 X[S::kX];
    const SmallOps<SP, TP> ops(X, nullptr);
    const int64_t b = blockIdx.x / a.blocks, k = blockIdx.x % a.blocks;
    const double norm = norm_of(part, b, per), den = norm + (double)a.poly.eps, bound = start_bound(norm / den);
    if (k == 0) {
        if (bound == 1.0) {
            if ((int)threadIdx.x < a.poly.steps) a.units[b * a.poly.steps + threadIdx.x] = table.u[threadIdx.x];
        } else if (threadIdx.x == 0) {
            step_units(a.poly, bound, a.units + b * a.poly.steps);
        }
    }
    const Scale inv = scale_of(unit_of(bound) / den);
    const T* g = (const T*)a.G + b * a.d.s * a.d.t;
    f16v ar[S::GX];
    ops.clear(ar);
    for (int64_t c = k; c < a.chunks; c += a.blocks) {
        float v[SmallOps<SP, TP>::kEights][8];
        ops.fetch(a.d, g, c * TP, a.wide, v);
        __syncthreads();  // the chunk before is read
        ops.place(a.d, v, inv);
        __syncthreads();
        put_image<SP, TP>(a.image + (b * a.chunks + c) * S::kX, X);
        ops.template square<TP / 32>(X, ar);
    }
    put_sums<SP, TP>(a.osums + blockIdx.x * (int64_t)(SP * SP), ar);
}

// one step; the last one writes the output
template <int SP, int TP, class T>
__global__ void __launch_bounds__((Small<SP, TP>::kThr)) k_ortho_wide_step(WideArgs a)
{
    using S = Small<SP, TP>;
    __shared__ __attribute__((aligned(16))) _Float16 X[S::kX], A[S::kA];
    const SmallOps<SP, TP> ops(X, A);
    const int64_t b = blockIdx.x / a.blocks, k = blockIdx.x % a.blocks;
    const bool last = a.step + 1 == a.poly.steps;
    const Units u = a.units[b * a.poly.steps + a.step];
    _Float16* image = a.image + b * a.chunks * S::kX;
    load_image<SP, TP>(image + k * S::kX, X);
    f16v ar[S::GX];
    ops.clear(ar);
#pragma unroll 2
    for (int32_t p = 0; p < a.nsums; ++p) add_sums<SP, TP>(a.sums + (b * a.nsums + p) * (int64_t)(SP * SP), ar);
#pragma unroll
    for (int x = 0; x < S::GX; ++x)
#pragma unroll
        for (int q = 0; q < 16; ++q) ar[x][q] *= u.gram;
    ops.poly(ar, u);
    ops.clear(ar);
    for (int64_t c = k; c < a.chunks; c += a.blocks) {
        if (c != k) {
            __syncthreads();  // the chunk before is read
            load_image<SP, TP>(image + c * S::kX, X);
        }
        wait_barrier<0>();
        f16v xr[S::NX], acc[S::NX];
        ops.get(xr);
        ops.next(acc);
#pragma unroll
        for (int x = 0; x < S::NX; ++x)
#pragma unroll
            for (int q = 0; q < 16; ++q) xr[x][q] = u.mul * acc[x][q] + u.add * xr[x][q];
        if (last) {
            ops.store(a.d, (T*)a.out + b * a.d.s * a.d.t, c * TP, a.wide, xr);
        } else {
            __syncthreads();
            ops.put(X, xr, ops.wt);
            __syncthreads();
            put_image<SP, TP>(image + c * S::kX, X);
            ops.template square<TP / 32>(X, ar);
        }
    }
    if (!last) put_sums<SP, TP>(a.osums + blockIdx.x * (int64_t)(SP * SP), ar);
}

// sums of the blocks' partial A, where they are many
__global__ void __launch_bounds__(kThreads) k_ortho_add(int64_t size, int32_t n, const float4* __restrict__ p,
                                                        float4* __restrict__ o)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (i >= size) return;
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int32_t k = 0; k < n; ++k) {
        const float4 f = p[(b * n + k) * size + i];
        t.x += f.x;
        t.y += f.y;
        t.z += f.z;
        t.w += f.w;
    }
    o[b * size + i] = t;
}

// ---- host ----------------------------------------------------------------------------------

// Wide tiles read less of LDS per product, small ones fill the chip: wide ones where
// they are on more than half of the 256 compute units (five steps, wide from 100 and
// from 129 tiles: 1408 x 1408, 121 and 66 tiles, 329 and 306 us; 1792 x 1792, 196 and 105,
// 558 and 510; 2048 x 2048, 256 and 136, 687 us, and 726 with the 136 as small tiles).
constexpr int64_t kFill = 129;

// Forms: a whole matrix per block, chunks of columns per block, tiles, or a matrix
// of few rows per block in fp64.
enum : int { kWhole = 0, kChunks = 1, kTiles = 2, kTiny = 3 };

struct OrthoLayout {
    OrthoDims d;
    int form, side;  // side: the padded short side of the first two forms
    int pad;
    int32_t per, blocks;
    int64_t chunks;
    size_t part, units, image, sums[2], total, X, Xt[2], A, B, bytes;
};

constexpr int kChunk = 128;    // columns
constexpr int kAddBlocks = 2;  // partial sums that every block adds by itself; more are added first

OrthoLayout ortho_layout(const OrthoShape& o)
{
    OrthoLayout w{};
    w.d.tall = o.m > o.n;
    w.d.s = w.d.tall ? o.n : o.m;
    w.d.t = w.d.tall ? o.m : o.n;
    w.form = w.d.t <= kChunk ? kWhole : w.d.s <= 128 ? kChunks : kTiles;
    w.side = w.d.s <= 64 ? 64 : 128;
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t at = off;
        off += align256((size_t)bytes);
        return at;
    };
    if (w.d.s <= kTinySide && w.d.s * w.d.t <= kTinyElems) w.form = kTiny;
    if (w.form == kWhole || w.form == kTiny) return w;  // no workspace
    const int64_t sums = cdiv64(o.m * o.n, kNormElems);
    w.per = (int32_t)(sums < kNormBlocks ? sums : kNormBlocks);
    w.part = take(8 * o.batch * w.per);
    w.units = take((int64_t)sizeof(Units) * o.batch * kMaxOrthoSteps);
    if (w.form == kChunks) {
        // about one block per compute unit (two of the small ones)
        w.chunks = cdiv64(w.d.t, kChunk);
        const int64_t want = (w.side == 128 ? 256 : 512) / (o.batch > 0 ? o.batch : 1);
        w.blocks = (int32_t)(want < 1 ? 1 : want < w.chunks ? want : w.chunks);
        w.image = take(4 * o.batch * w.chunks * w.side * kChunk);
        for (int k = 0; k < 2; ++k) w.sums[k] = take(4 * o.batch * w.blocks * w.side * w.side);
        w.total = take(4 * o.batch * w.side * w.side);
    } else {
        // whole wide tiles where there are enough of them and they add little padding
        const int64_t s64 = cdiv64(w.d.s, 64), t64 = cdiv64(w.d.t, 64), s128 = cdiv64(s64, 2), t128 = cdiv64(t64, 2);
        w.pad = s128 * t128 * o.batch >= kFill && 40 * s128 * t128 <= 11 * s64 * t64 ? 128 : 64;
        w.d.sp = cdiv64(w.d.s, w.pad) * w.pad;
        w.d.tp = cdiv64(w.d.t, w.pad) * w.pad;
        w.X = take(4 * o.batch * w.d.sp * w.d.tp);
        for (int k = 0; k < 2; ++k) w.Xt[k] = take(4 * o.batch * w.d.sp * w.d.tp);
        w.A = take(4 * o.batch * w.d.sp * w.d.sp);
        w.B = take(4 * o.batch * w.d.sp * w.d.sp);
    }
    w.bytes = off;
    return w;
}

template <int KIND, class T>
void prod(const OrthoLayout& w, const OrthoShape& o, ProdArgs a, hipStream_t s)
{
    constexpr bool upper = KIND == kGram || KIND == kPoly;
    auto tiles = [&](int64_t tile) {
        a.ti = w.d.sp / tile;
        a.tj = upper ? 0 : w.d.tp / tile;
        return (upper ? a.ti * (a.ti + 1) / 2 : a.ti * a.tj) * o.batch;
    };
    if (w.pad == 128 && tiles(128) >= kFill)
        hipLaunchKernelGGL((k_ortho_prod<128, KIND, T>), dim3((unsigned)tiles(128)), dim3(kProdThreads<128>), 0, s,
                           a);
    else
        hipLaunchKernelGGL((k_ortho_prod<64, KIND, T>), dim3((unsigned)tiles(64)), dim3(kProdThreads<64>), 0, s, a);
}

bool wide_rows(const OrthoShape& o, const void* G, const void* out)
{
    return (o.n * dtype_size(o.dtype)) % 16 == 0 && (((uintptr_t)G | (uintptr_t)out) & 15u) == 0;
}

template <int SP, int TP, class T>
hipError_t whole(const OrthoLayout& w, const OrthoShape& o, const OrthoPoly& poly, const UnitTable& table,
                 const void* G, void* out, hipStream_t s)
{
    SmallArgs a{};
    a.d = w.d;
    a.poly = poly;
    a.table = table;
    a.wide = wide_rows(o, G, out);
    a.G = G;
    a.out = out;
    hipLaunchKernelGGL((k_ortho_small<SP, TP, T>), dim3((unsigned)o.batch), dim3(Small<SP, TP>::kThr), 0, s, a);
    return hipGetLastError();
}

template <int SP, class T>
hipError_t chunks(const OrthoLayout& w, const OrthoShape& o, const OrthoPoly& poly, const UnitTable& table,
                  const void* G, void* out, char* base, hipStream_t s)
{
    constexpr int TP = kChunk;
    using S = Small<SP, TP>;
    const dim3 grid((unsigned)(o.batch * w.blocks)), thr(S::kThr);
    float *sums[2] = {(float*)(base + w.sums[0]), (float*)(base + w.sums[1])}, *total = (float*)(base + w.total);
    WideArgs a{};
    a.d = w.d;
    a.poly = poly;
    a.chunks = w.chunks;
    a.blocks = w.blocks;
    a.wide = wide_rows(o, G, out);
    a.G = G;
    a.out = out;
    a.units = (Units*)(base + w.units);
    a.image = (_Float16*)(base + w.image);
    a.osums = sums[0];
    hipLaunchKernelGGL((k_ortho_wide_first<SP, TP, T>), grid, thr, 0, s, a, table, w.per,
                       (const double*)(base + w.part));
    const bool add = w.blocks > kAddBlocks;
    for (int step = 0; step < o.steps; ++step) {
        a.step = step;
        a.sums = sums[step & 1];
        a.osums = sums[(step & 1) ^ 1];
        a.nsums = w.blocks;
        if (add) {
            const int64_t size = SP * SP / 4;
            hipLaunchKernelGGL(k_ortho_add, dim3((unsigned)cdiv64(size, kThreads), (unsigned)o.batch), dim3(kThreads), 0,
                               s, size, w.blocks, (const float4*)a.sums, (float4*)total);
            a.sums = total;
            a.nsums = 1;
        }
        hipLaunchKernelGGL((k_ortho_wide_step<SP, TP, T>), grid, thr, 0, s, a);
    }
    return hipGetLastError();
}

template <class T>
hipError_t tiles(const OrthoLayout& w, const OrthoShape& o, const OrthoPoly& poly, const UnitTable& table,
                 const void* G, void* out, char* base, hipStream_t s)
{
    _Float16 *X = (_Float16*)(base + w.X), *Xt[2] = {(_Float16*)(base + w.Xt[0]), (_Float16*)(base + w.Xt[1])};
    _Float16 *A = (_Float16*)(base + w.A), *B = (_Float16*)(base + w.B);
    Units* units = (Units*)(base + w.units);
    hipLaunchKernelGGL(k_ortho_first<T>, dim3((unsigned)(o.batch * (w.d.sp / 64) * (w.d.tp / 64))), dim3(kThreads), 0,
                       s, w.d, poly, table, w.per, (const double*)(base + w.part), (const T*)G, X, Xt[0], units);
    for (int step = 0; step < o.steps; ++step) {
        ProdArgs a{};
        a.d = w.d;
        a.units = units + step;
        a.steps = o.steps;
        a.K = w.d.tp;
        a.P = a.Q = X;
        a.R = a.Rt = A;
        prod<kGram, T>(w, o, a, s);
        a.K = w.d.sp;
        a.P = a.Q = a.E = A;
        a.R = a.Rt = B;
        prod<kPoly, T>(w, o, a, s);
        a.P = B;
        a.Q = a.E = Xt[step & 1];
        a.R = X;
        a.Rt = Xt[(step & 1) ^ 1];
        a.out = out;
        if (step + 1 == o.steps) prod<kLast, T>(w, o, a, s);
        else prod<kNext, T>(w, o, a, s);
    }
    return hipGetLastError();
}

template <class T>
hipError_t tiny(const OrthoLayout& w, const OrthoShape& o, const OrthoPoly& poly, const void* G, void* out,
                hipStream_t s)
{
    TinyArgs a{};
    a.d = w.d;
    a.poly = poly;
    // rows begin 4 modulo 16 banks apart: sixteen rows at four columns meet in no bank
    a.ld = (int32_t)(cdiv64(w.d.t, 16) * 16 + 4);
    a.G = G;
    a.out = out;
    hipLaunchKernelGGL(k_ortho_tiny<T>, dim3((unsigned)o.batch), dim3(64 * kTinyWaves), (unsigned)(w.d.s * a.ld * 4), s, a);
    return hipGetLastError();
}

template <class T>
hipError_t orthogonalize(const OrthoShape& o, const void* G, void* out, void* ws, hipStream_t s)
{
    const OrthoLayout w = ortho_layout(o);
    char* base = (char*)ws;
    const OrthoPoly poly{o.steps, o.a, o.b, o.c, o.eps, o.scale};
    if (w.form == kTiny) return tiny<T>(w, o, poly, G, out, s);
    UnitTable table{};
    step_units(poly, 1.0, table.u);
    if (w.form == kWhole) {
        if (w.d.t <= 64) return whole<64, 64, T>(w, o, poly, table, G, out, s);
        if (w.side == 64) return whole<64, 128, T>(w, o, poly, table, G, out, s);
        return whole<128, 128, T>(w, o, poly, table, G, out, s);
    }
    hipLaunchKernelGGL(k_ortho_norm<T>, dim3((unsigned)(o.batch * w.per)), dim3(kThreads), 0, s, o.m * o.n, w.per,
                       o.m * o.n % kWide<T> == 0 && ((uintptr_t)G & 15u) == 0, (const T*)G, (double*)(base + w.part));
    if (w.form == kTiles) return tiles<T>(w, o, poly, table, G, out, base, s);
    return w.side == 64 ? chunks<64, T>(w, o, poly, table, G, out, base, s)
                        : chunks<128, T>(w, o, poly, table, G, out, base, s);
}

}  // namespace

bool ortho_bounded(double a, double b, double c, int steps)
{
    double M = 1.0;
    for (int k = 0; k < steps; ++k) {
        const Bounds r = step_bounds(a, b, c, M);
        // no product at all, or beyond what the fp32 factors hold
        if (!(r.next >= 1e-6) || !(r.next <= 1e6) || !(r.poly >= 1e-6) || !(r.poly <= 1e6)) return false;
        M = r.next;
    }
    return true;
}

size_t ortho_workspace_bytes(const OrthoShape& o) { return ortho_layout(o).bytes; }

hipError_t launch_orthogonalize(const OrthoShape& o, const void* G, void* out, void* ws, hipStream_t s)
{
    return o.dtype == kF32 ? orthogonalize<float>(o, G, out, ws, s) : orthogonalize<bf16_t>(o, G, out, ws, s);
}

}  // namespace cgtp
