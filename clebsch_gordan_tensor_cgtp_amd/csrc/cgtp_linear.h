// cgtp_linear.h -- what the kernels of the product with its epilogue share (device code of
// cgtp_linear.hip and cgtp_linear_{wide,few,rows,back}.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "cgtp_act.h"
#include "cgtp_drop.h"
#include "cgtp_internal.h"
#include "cgtp_train_internal.h"
#include "cgtp_vec.h"

namespace cgtp {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4 __attribute__((ext_vector_type(4)));

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// block x of n works on tile `xcd_order`: blocks go to the XCDs in turn, so that an XCD's
// tiles are neighbours and share its L2
__device__ __forceinline__ int64_t xcd_order(int64_t x, int64_t n)
{
    const int64_t q = n / kXcds, rest = n % kXcds, c = x % kXcds;
    return c * q + (c < rest ? c : rest) + x / kXcds;
}

enum : int { kFwd = 0, kDx = 1, kDw = 2 };

struct GemmArgs {
    const void *A, *B;        // kFwd: x, W; kDx: g, W; kDw: x, g
    const void* Z;            // z [N][M], or nullptr: act none
    int64_t lda, ldb, ldz;
    int64_t rows, cols, depth;  // of the result, of the contraction
    int64_t first;            // row of the caller's that the first one here is, for the mask
    int64_t tr, tc;           // tiles along rows and columns
    int64_t splits, run;      // parts of the contraction and their length
    int act;
    Drop drop;
    // epilogue
    const float* bias;
    const void* R;
    void *out, *zout;
    int64_t ldr, ldo;
    float* part;       // [splits][rows][cols] where splits > 1
    float* db;         // kDw: the gradient of the bias, or nullptr
    double* db_part;   // [db_splits][cols]
    int64_t db_splits;
    bool want;         // kDw: the product itself is wanted
};

// planes that an operand of type T is cut into
template <class T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;

// and dz = mask g act'(z): an fp32 number whatever g's type, so three, but those of g where there is no
// slope (HZ: there may be a z), which the mask alone leaves as it is
template <class T, bool HZ>
constexpr int kSlopePlanes = HZ ? 3 : kPlanes<T>;

// The products of operands of NA and NB planes, the smallest first: f(i, j) for plane i of the one and
// j of the other, i + j below the larger number.
template <int NA, int NB, class F>
__device__ __forceinline__ void each_product(F&& f)
{
    constexpr int N = NA > NB ? NA : NB;
#pragma unroll
    for (int o = N - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i <= o; ++i)
            if (i < NA && o - i < NB) f(i, o - i);
}

// v as NP bf16 vectors
template <int NP>
__device__ __forceinline__ void cut(f8 v, b8 (&p)[NP])
{
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        p[i] = __builtin_convertvector(v, b8);
        if (i + 1 < NP) v -= __builtin_convertvector(p[i], f8);
    }
}

// The same for eight elements in a row of the contraction: the remainder of each element of a pair comes
// from one product with (-1, 0) or (0, -1), exact and cheaper than taking the pair apart (3.5 operations
// an element instead of 5.5).  An infinity spoils its neighbour too, which reaches the same results.
template <int NP>
__device__ __forceinline__ void cut_along(f8 v, b8 (&p)[NP])
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    uint32_t first = 0x0000bf80u, second = 0xbf800000u;
    // (not as a constant: the compiler takes the first for the inline constant -1.0, which is the second)
    asm("" : "+s"(first));
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const b2 h = __builtin_convertvector(f2{v[j], v[j + 1]}, b2);
            p[i][j] = h[0];
            p[i][j + 1] = h[1];
            if (i + 1 < NP) {
                v[j] = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(b2, first), v[j], false);
                v[j + 1] = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(b2, second), v[j + 1], false);
            }
        }
}

// act'(z) and the mask of eight elements of g at (n, 8 q); HZ: there may be a z
template <bool HZ = true>
__device__ __forceinline__ void slope8(const GemmArgs& a, uint64_t offset, f8& v, const float (&z)[8], int64_t n, int32_t q)
{
    if (HZ && a.Z) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= act_slope(a.act, z[j]);
    }
    if (a.drop.thr) {
        const Drawn f = philox((uint32_t)q, (uint32_t)(a.first + n), offset, a.drop.seed);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f[j] >= a.drop.thr ? v[j] : 0.0f;
    }
}

// Operand fragment of the matrix instruction whose contraction runs across the rows of LDS, ld halves
// apart: p is this lane's place, row 8 (lane / 32) + lane % 16 / 4 and column (lane & 16) + 4 (lane % 4)
// of the 16 x 32 block.
__device__ __forceinline__ b8 read_across(const uint16_t* p, int ld)
{
    auto tr = [](const uint16_t* q) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4*)(const __attribute__((address_space(3))) void*)q);
    };
    struct Two {
        s4 a, b;
    } t{tr(p), tr(p + 4 * ld)};
    return __builtin_bit_cast(b8, t);
}

// the bias of eight channels, of which w are inside (VEC: all)
template <bool VEC>
__device__ __forceinline__ void bias8(const GemmArgs& a, int64_t c, int w, float (&b)[8])
{
    if (VEC && a.bias) {
        struct __attribute__((packed, aligned(4))) Four {
            float v[4];
        };
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const Four f = *reinterpret_cast<const Four*>(a.bias + c + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) b[j + e] = f.v[e];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = a.bias && j < w ? a.bias[c + j] : 0.0f;
    }
}

// Eight results from channel c on, of which w are inside, of each of G rows n (none where on is
// not set).  The conditions stand outside the loops over the rows, so that the rows' loads and
// chains of operations overlap.
template <class T, int KIND, bool VEC, int G>
__device__ __forceinline__ void finish8(const GemmArgs& a, uint64_t offset, float (&v)[G][8], const float (&b)[8],
                                        const int64_t (&n)[G], const bool (&on)[G], int64_t c, int w)
{
    auto put = [&](T* p, const float(&v)[8]) { store8<T>(p, v, VEC ? 8 : w); };
    if constexpr (KIND == kFwd) {
        float r[G][8];
        if (a.R) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                Raw8<T> t;
                t.load_some((const T*)a.R + n[g] * a.ldr + c, !on[g] ? 0 : VEC ? 8 : w);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[g][j] = t[j];
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[g][j] += b[j];
        if (a.zout) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (on[g]) put((T*)a.zout + n[g] * a.cols + c, v[g]);
        }
        if (a.act == kSilu) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[g][j] = act_of<kSilu>(v[g][j]);
        } else if (a.act == kTanh) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[g][j] = act_of<kTanh>(v[g][j]);
        }
        if (a.drop.thr) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const Drawn f = philox((uint32_t)c / 8, (uint32_t)(a.first + n[g]), offset, a.drop.seed);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[g][j] = f[j] >= a.drop.thr ? v[g][j] * a.drop.scale : 0.0f;
            }
        }
        if (a.R) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[g][j] += r[g][j];
        }
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[g][j] *= a.drop.scale;
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (on[g]) put((T*)a.out + n[g] * a.ldo + c, v[g]);
}

// The same, or the sums of one part of the contraction where that is cut.
template <class T, int KIND, bool VEC, int G>
__device__ __forceinline__ void leave8(const GemmArgs& a, uint64_t offset, int64_t part, float (&v)[G][8],
                                       const float (&b)[8], const int64_t (&n)[G], const bool (&on)[G], int64_t c, int w)
{
    if (a.splits > 1) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float* p = a.part + (part * a.rows + n[g]) * a.cols + c;
            if (on[g]) store8<float>(p, v[g], VEC ? 8 : w);
        }
    } else {
        finish8<T, KIND, VEC, G>(a, offset, v, b, n, on, c, w);
    }
}

}  // namespace cgtp
