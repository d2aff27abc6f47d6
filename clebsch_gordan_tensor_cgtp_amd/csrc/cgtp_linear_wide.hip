// cgtp_linear_wide.hip -- large products of bf16 planes: y, dx and dW where the matrix
// cores bound them.
//
// The operands are bf16 in memory: x, W and g as the caller has them, or as planes that a
// pass of their own has written to the workspace -- the three numbers of an fp32 operand
// (cgtp_linear.hip), dz with its mask and slope (formed once instead of in every tile
// that needs it, three numbers with a slope for either type; its columns' sums on the way).  A product of
// three planes each goes through the contraction six times, of three with one three times, the smallest
// products first, into one accumulator.
//
// A block computes a BM x BN tile, each wave WM x WN of it, through a ring of LDS buffers of 32 k that
// loads fill directly; one barrier to a step, whose operands are in registers when it begins.  The 16-byte
// pieces of a buffer are swapped about (by the address that each lane loads from), so that
// what a read instruction takes spreads over all banks: an operand whose rows run along k has
// the pieces of row r at piece ^ (r / 4 % 4) of its 64 bytes, the other kind its 32-byte pieces
// of row k at piece ^ 2 (k % 4).  Each wave takes its results through LDS by itself, 32 rows at a
// time, so that they leave in whole lines.
//
// 16384 x 1024 x 4096 bf16: dx and dW 111 and 112 us where dz is g (1.23 PFLOP/s; a library's plain product of
// these operands takes 142 us), 346 and 310 with SiLU, three products each (1.19 and 1.33 PFLOP/s), the matrix cores
// busy 65 and 78 % of the cycles at the clock that the power leaves.  y, whose tiles each have an epilogue of
// 13 us (mask, SiLU, two arrays out) that nothing covers, 165 to 170.  Tiles of 256 x 128, two blocks to a
// compute unit, whose epilogues can be covered: 211 (half again as much comes from L2, 48 bytes a cycle and
// compute unit).  Tiles of 128 x 128 serve results that have few.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "cgtp_linear.h"
#include "cgtp_linear_wide.h"

namespace cgtp {
namespace {

constexpr int kStep = 32;

// all but the last N of this wave's loads have arrived, its LDS reads are done, and every
// wave of the block is here
template <int N>
__device__ __forceinline__ void wait_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);  // vmcnt(N) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
}

// Sixteen bytes per lane from base + offset (of each lane) to LDS, from `to` on in the lanes' order,
// without the compiler's knowledge: where it knows of such loads, every transposing read
// waits for all of them.  Their arrival is what wait_barrier counts; nothing reads `to` before,
// and nothing else in these kernels uses m0.
__device__ __forceinline__ void load_lds(uint16_t* to, const uint16_t* base, uint32_t offset)
{
    const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t*)to;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(offset), "s"(base));
}

// One operand's tile: WIDTH rows (or columns) of the result by kStep of the contraction.
template <int WIDTH, int THR, bool ALONG>
struct Tile {
    static constexpr bool kAlong = ALONG;
    static constexpr int kPieces = WIDTH * kStep / 8 / THR;
    static_assert(WIDTH * kStep % (8 * THR) == 0, "whole pieces per thread");

    // row (ALONG) or k and the source piece of 8 halves of this thread's piece i
    __device__ static __forceinline__ void place(int i, int& row, int& col)
    {
        const int p = i * THR + (int)threadIdx.x;
        if constexpr (ALONG) {
            row = p / 4;
            col = ((p & 3) ^ ((row >> 2) & 3)) * 8;
        } else {
            constexpr int kPer = WIDTH / 8;
            row = p / kPer;
            col = (((p % kPer) >> 1) ^ (2 * (row & 3))) * 16 + (p & 1) * 8;
        }
    }
    // the 32 x 16 operand from row (column) r0 and k = 16 ks on
    __device__ static __forceinline__ b8 read(const uint16_t* s, int r0, int ks, int lane)
    {
        if constexpr (ALONG) {
            const int row = r0 + (lane & 31), piece = ks * 2 + (lane >> 5);
            return *reinterpret_cast<const b8*>(s + row * kStep + ((piece ^ ((row >> 2) & 3)) * 8));
        } else {
            const int l = lane & 15, k = ks * 16 + 8 * (lane >> 5) + l / 4, col = r0 + (lane & 16);
            const uint16_t* p = s + k * WIDTH + (((col >> 4) ^ (2 * (k & 3))) << 4) + 4 * (l % 4);
            return read_across(p, WIDTH);
        }
    }
};

// tile r of tr x tc: bands of four columns, row by row within a band
__device__ __forceinline__ void tile_at(int64_t r, int64_t tr, int64_t tc, int64_t& i, int64_t& j)
{
    const int64_t band = r / (4 * tr), c0 = band * 4, w = tc - c0 < 4 ? tc - c0 : 4;
    r -= band * 4 * tr;
    i = r / w;
    j = c0 + r % w;
}

template <class T, int KIND, bool HZ, int BM, int BN, int WM, int WN, int kStages>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN)) __attribute__((amdgpu_waves_per_eu(BM == 256 ? 2 : 3)))
k_linear_wide(WideArgs w)
{
    constexpr int kThr = 64 * (BM / WM) * (BN / WN), FM = WM / 32, FN = WN / 32;
    constexpr bool kAlongP = KIND != kDw, kAlongQ = KIND == kDx;
    using P = Tile<BM, kThr, kAlongP>;
    using Q = Tile<BN, kThr, kAlongQ>;
    // planes of dz times the one of the other operand, or all products of two fp32 numbers
    constexpr int kPasses = kPlanes<T> == 3 ? 6 : KIND == kFwd ? 1 : kSlopePlanes<T, HZ>;
    constexpr int kStage = (BM + BN) * kStep;  // halves
    constexpr int kLd = WN + 4, kPatch = 32 * kLd * 4;
    constexpr int kRing = kStages * kStage * 2, kOut = kPatch * (kThr / 64);
    __shared__ __attribute__((aligned(16))) char mem[kRing > kOut ? kRing : kOut];
    uint16_t* ring = reinterpret_cast<uint16_t*>(mem);
    const GemmArgs& a = w.g;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t at = xcd_order(blockIdx.x, gridDim.x), tiles = a.tr * a.tc;
    const int64_t part = at / tiles;
    int64_t ti, tj;
    tile_at(at % tiles, a.tr, a.tc, ti, tj);
    const int64_t r0 = ti * BM, c0 = tj * BN;
    const int64_t k0 = part * a.run, k1 = k0 + a.run < a.depth ? k0 + a.run : a.depth;
    const int32_t full = (int32_t)((k1 - k0) / kStep), tail = (int32_t)((k1 - k0) % kStep);

    // byte offsets of the thread's pieces from the step's first element; outside the result
    // the last row or column is loaded again
    uint32_t op[P::kPieces], oq[Q::kPieces];
    auto offsets = [&](auto side, uint32_t* o, int64_t ld, int64_t first, int64_t lim) {
        using S = decltype(side);
#pragma unroll
        for (int i = 0; i < S::kPieces; ++i) {
            int row, col;
            S::place(i, row, col);
            const int64_t left = lim - first;
            if constexpr (S::kAlong) row = row < left ? row : (int)left - 1;
            else col = col < left ? col : (int)left - 8;
            o[i] = (uint32_t)((uint32_t)row * (uint32_t)ld + (uint32_t)col) * 2u;
        }
    };
    offsets(P{}, op, w.ldp, r0, a.rows);
    offsets(Q{}, oq, w.ldq, c0, a.cols);
    const uint16_t* p0 = w.P + (kAlongP ? r0 * w.ldp + k0 : k0 * w.ldp + r0);
    const uint16_t* q0 = w.Q + (kAlongQ ? c0 * w.ldq + k0 : k0 * w.ldq + c0);
    const int64_t stepP = kAlongP ? kStep : kStep * w.ldp, stepQ = kAlongQ ? kStep : kStep * w.ldq;
    // planes of pass j of six: h l, m m, l h, h m, m h, h h (h, m, l = 0, 1, 2); of three: l, m, h of dz
    auto plane = [&](int j, const uint16_t*& p, const uint16_t*& q) {
        const int ip = kPasses == 6 ? (0x010210 >> (4 * j)) & 15 : KIND == kDx ? kPasses - 1 - j : 0;
        const int iq = kPasses == 6 ? (0x001012 >> (4 * j)) & 15 : KIND == kDw ? kPasses - 1 - j : 0;
        p = p0 + ip * w.planeP;
        q = q0 + iq * w.planeQ;
    };

    f16v acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
    struct Frag {  // of one step
        b8 p[2][FM], q[2][FN];
    };
    auto read = [&](Frag& f, int slot) {
        const uint16_t* s = ring + slot * kStage;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int y = 0; y < FN; ++y) f.q[ks][y] = Q::read(s + BM * kStep, wn + 32 * y, ks, lane);
#pragma unroll
            for (int x = 0; x < FM; ++x) f.p[ks][x] = P::read(s, wm + 32 * x, ks, lane);
        }
    };
    auto multiply = [&](const Frag& f) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int x = 0; x < FM; ++x)
#pragma unroll
                for (int y = 0; y < FN; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.q[ks][y], f.p[ks][x], acc[x][y], 0, 0, 0);
    };
    // the next step's LDS reads between the first half of the products
    auto in_turn = [&]() {
        constexpr int kReads = 2 * (FM * (kAlongP ? 1 : 2) + FN * (kAlongQ ? 1 : 2)), kMul = 2 * FM * FN;
#pragma unroll
        for (int g = 0; g < kMul / 2; ++g) {
            __builtin_amdgcn_sched_group_barrier(0x100, (kReads + kMul / 2 - 1) / (kMul / 2), 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kMul / 2, 0);
    };
    Frag f0, f1;

    // What is left of the contraction beyond whole steps goes through registers, zeros behind it.
    if (tail) {
        for (int j = 0; j < kPasses; ++j) {
            const uint16_t *p, *q;
            plane(j, p, q);
            auto some = [&](auto side, const uint16_t* from, const uint32_t* o, uint16_t* to) {
                using S = decltype(side);
#pragma unroll
                for (int i = 0; i < S::kPieces; ++i) {
                    int row, col;
                    S::place(i, row, col);
                    const uint16_t* e = reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(from) + o[i]);
                    uint16_t* t = to + (i * kThr + tid) * 8;
                    for (int c = 0; c < 8; ++c) t[c] = (S::kAlong ? col + c : row) < tail ? e[c] : (uint16_t)0;
                }
            };
            some(P{}, p + full * stepP, op, ring);
            some(Q{}, q + full * stepQ, oq, ring + BM * kStep);
            __syncthreads();
            read(f0, 0);
            multiply(f0);
            __syncthreads();
        }
    }

    // the loads' place: the next step's operands
    const uint16_t *pp, *qq;
    plane(0, pp, qq);
    auto fill = [&](int slot) {
        uint16_t* to = ring + slot * kStage + wave * 512;
#pragma unroll
        for (int i = 0; i < P::kPieces; ++i) load_lds(to + i * kThr * 8, pp, op[i]);
#pragma unroll
        for (int i = 0; i < Q::kPieces; ++i) load_lds(to + BM * kStep + i * kThr * 8, qq, oq[i]);
        pp += stepP;
        qq += stepQ;
    };
    constexpr int kLoads = P::kPieces + Q::kPieces;
    const int32_t nk = full * kPasses;
    // Step k multiplies block k, which is in registers, while it reads block k + 1 from LDS and
    // starts the loads of block k + kStages into the buffer that block k has left.  Block k + 1 is in
    // when at most the kStages - 2 blocks after it are out; behind the barrier every wave has read block k.
    int slot = 0;  // of block k
    auto after = [](int i) { return i + 1 == kStages ? 0 : i + 1; };
    auto main_step = [&](const Frag& cur, Frag& next) {
        wait_barrier<kLoads*(kStages - 2)>();
        const int to = slot;
        slot = after(slot);
        read(next, slot);
        fill(to);
        multiply(cur);
        in_turn();
    };
    auto tail_step = [&](bool more, const Frag& cur, Frag& next) {
        if (more) {
            wait_barrier<0>();
            slot = after(slot);
            read(next, slot);
        }
        multiply(cur);
    };
    if (nk > 0) {
        int pass = 0;
        int32_t left = full;  // of the pass, for the loads
        const int ahead = nk < kStages ? nk : kStages;
        auto next_pass = [&]() {
            left = full;
            if (++pass < kPasses) plane(pass, pp, qq);
        };
        for (int i = 0; i < ahead; ++i) {
            fill(i);
            if (--left == 0) next_pass();
        }
        if (nk >= kStages) wait_barrier<kLoads*(kStages - 1)>();
        else wait_barrier<0>();
        read(f0, 0);
        int32_t k = 0;
        while (k + kStages < nk) {  // (no condition inside a pass' steps: it would wait for what it reads)
            k += left;
            if (left & 1) {
                main_step(f0, f1);
                f0 = f1;
            }
            for (int32_t i = left >> 1; i > 0; --i) {
                main_step(f0, f1);
                main_step(f1, f0);
            }
            next_pass();
        }
        for (; k < nk; k += 2) {
            tail_step(k + 1 < nk, f0, f1);
            if (k + 1 < nk) tail_step(k + 2 < nk, f1, f0);
        }
    }
    __syncthreads();

    // a lane holds row lane % 32, columns 8 g + 4 (lane / 32) + 0 .. 3 of each tile of 32
    float* s = reinterpret_cast<float*>(mem) + wave * (kPatch / 4);
    const uint64_t offset = drop_offset(a.drop);
    constexpr int kPer = WN / 8, kRows = 64 / kPer, kG = 2;
    const int64_t c = c0 + wn + lane % kPer * 8;
    float bias[8] = {};
    if (KIND == kFwd && c < a.cols) bias8<true>(a, c, 8, bias);
#pragma unroll
    for (int x = 0; x < FM; ++x) {
#pragma unroll
        for (int y = 0; y < FN; ++y)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 v{acc[x][y][4 * g], acc[x][y][4 * g + 1], acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
                *reinterpret_cast<float4*>(&s[(lane & 31) * kLd + 32 * y + 8 * g + 4 * (lane >> 5)]) = v;
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += kG * kRows) {
            float v[kG][8];
            int64_t n[kG];
            bool on[kG];
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                const int row = i0 + g * kRows + lane / kPer;
                n[g] = r0 + wm + 32 * x + row;
                on[g] = n[g] < a.rows && c < a.cols;
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4*>(&v[g][e]) = *reinterpret_cast<const float4*>(&s[row * kLd + lane % kPer * 8 + e]);
            }
            leave8<T, KIND, true, kG>(a, offset, part, v, bias, n, on, c, 8);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// dx of up to KC inputs over many outputs: memory bounds it, g (and z) being read once, and the six
// products with the cutting of g come close (105730 x 1920 x 64 fp32 230 to 240 us, 3.6 TB/s; 413 blocks of
// 256 rows leave a fifth of the chip's places empty; by tiles 264; 128 inputs 332, by tiles 380).  Each wave
// loads its 32 FR rows of dz straight into matrix operands (a lane has eight outputs of one row),
// forms and cuts them there; the planes of W come to LDS by direct loads, 32 outputs to a step, for the
// block's four waves.  Both are fetched one step ahead: W's behind the one barrier of a step, dz's into
// the registers that have just been cut.  HZ: with z.
template <class T, int KC, int FR, bool HZ>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) k_linear_dx(WideArgs w)
{
    constexpr int NP = kPlanes<T>, NZ = kSlopePlanes<T, HZ>, FC = KC / 32, kThr = 256;
    using Q = Tile<KC, kThr, true>;
    constexpr int kPlane = KC * kStep, kLdS = 36;  // halves; floats
    __shared__ __attribute__((aligned(16))) uint16_t ring[2][NP * kPlane];
    __shared__ __attribute__((aligned(16))) float patch[4][32 * kLdS];
    const GemmArgs& a = w.g;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t r0 = xcd_order(blockIdx.x, gridDim.x) * (128 * FR) + wave * (32 * FR);
    const uint64_t offset = drop_offset(a.drop);

    // W's pieces: rows behind the last input are that one again, outputs behind the last the last eight
    // (dz is zero there)
    auto fill = [&](int slot, int64_t k) {
#pragma unroll
        for (int i = 0; i < Q::kPieces; ++i) {
            int row, col;
            Q::place(i, row, col);
            row = row < a.cols ? row : (int)a.cols - 1;
            col = k + col < a.depth ? col : (int)(a.depth - k) - 8;
#pragma unroll
            for (int p = 0; p < NP; ++p)
                load_lds(&ring[slot][p * kPlane + (i * kThr + wave * 64) * 8], w.Q + p * w.planeQ + k, (uint32_t)(row * (int)w.ldq + col) * 2u);
        }
    };
    // rows outside are the last one again; byte offsets from the wave's first row
    int64_t n[FR];
    uint32_t og[FR], oz[FR];
    const int64_t base = r0 < a.rows ? r0 : a.rows - 1;
#pragma unroll
    for (int x = 0; x < FR; ++x) {
        const int64_t m = r0 + 32 * x + (lane & 31);
        n[x] = m < a.rows ? m : a.rows - 1;
        og[x] = ((uint32_t)(n[x] - base) * (uint32_t)a.lda + 8u * (uint32_t)(lane >> 5)) * (uint32_t)sizeof(T);
        oz[x] = ((uint32_t)(n[x] - base) * (uint32_t)a.ldz + 8u * (uint32_t)(lane >> 5)) * (uint32_t)sizeof(T);
    }
    const char* pg = (const char*)((const T*)a.A + base * a.lda);
    const char* pz = HZ ? (const char*)((const T*)a.Z + base * a.ldz) : nullptr;
    Raw8<T> rg[2][FR], rz[HZ ? 2 : 1][HZ ? FR : 1];
    // outputs k + 16 ks + 8 (lane / 32) + 0 .. 7; those behind the last are others of the row
    auto fetch = [&](int ks, int x, int64_t k) {
        const uint32_t back = k + 16 * ks + 8 * (lane >> 5) < a.depth ? 0 : (uint32_t)(16 * ks + 8 * (lane >> 5)) * (uint32_t)sizeof(T);
        const int64_t at = (k + 16 * ks) * (int64_t)sizeof(T);
        rg[ks][x].load((const T*)(pg + at + og[x] - back));
        if constexpr (HZ) rz[ks][x].load((const T*)(pz + at + oz[x] - back));
    };
    auto fetch_in = [&](int ks, int x, int64_t k) {
        const int64_t at = (k + 16 * ks) * (int64_t)sizeof(T);
        rg[ks][x].load((const T*)(pg + at + og[x]));
        if constexpr (HZ) rz[ks][x].load((const T*)(pz + at + oz[x]));
    };
    constexpr int kFetches = 2 * FR * (HZ ? 2 : 1) * (int)sizeof(T) / 2;  // loads of a step
    f16v acc[FR][FC];
#pragma unroll
    for (int x = 0; x < FR; ++x)
#pragma unroll
        for (int y = 0; y < FC; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;
    // one step; `then`: the next one's first output, or k again behind the last (not used)
    auto step = [&](int slot, int64_t k, int64_t then, auto last, auto next) {
        constexpr bool LAST = decltype(last)::value;
        wait_barrier<kFetches>();  // W's loads were started before the step's
        fill(slot ^ 1, then);
        asm volatile("" ::: "memory");  // (and stay so)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            b8 p[FR][NZ], q[FC][NP];
            const int64_t e = k + 16 * ks + 8 * (lane >> 5);
#pragma unroll
            for (int x = 0; x < FR; ++x) {
                f8 v;
                float z[8] = {};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = rg[ks][x][j];
                    if constexpr (HZ) z[j] = rz[ks][x][j];
                }
                next(ks, x, then);
                slope8<HZ>(a, offset, v, z, n[x], (int32_t)(e / 8));
                if constexpr (LAST) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = e < a.depth ? v[j] : 0.0f;
                }
                cut_along(v, p[x]);
            }
#pragma unroll
            for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                for (int y = 0; y < FC; ++y) q[y][o] = Q::read(&ring[slot][o * kPlane], 32 * y, ks, lane);
            each_product<NZ, NP>([&](int i, int j) {
#pragma unroll
                for (int x = 0; x < FR; ++x)
#pragma unroll
                    for (int y = 0; y < FC; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[y][j], p[x][i], acc[x][y], 0, 0, 0);
            });
        }
    };
    fill(0, 0);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int x = 0; x < FR; ++x) fetch(ks, x, 0);
    int slot = 0;
    int64_t k = 0;
    for (; k + 2 * kStep <= a.depth; k += kStep, slot ^= 1) step(slot, k, k + kStep, std::false_type{}, fetch_in);
    for (; k < a.depth; k += kStep, slot ^= 1) step(slot, k, k + kStep < a.depth ? k + kStep : k, std::true_type{}, fetch);
    wait_barrier<0>();  // no load to LDS is left
    // a lane holds row lane % 32, inputs 8 g + 4 (lane / 32) + 0 .. 3
    float* s = patch[wave];
    const float none[8] = {};
#pragma unroll
    for (int x = 0; x < FR; ++x)
#pragma unroll
        for (int y = 0; y < FC; ++y) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 v{acc[x][y][4 * g], acc[x][y][4 * g + 1], acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
                *reinterpret_cast<float4*>(&s[(lane & 31) * kLdS + 8 * g + 4 * (lane >> 5)]) = v;
            }
            __builtin_amdgcn_wave_barrier();
            float v[2][8];
            int64_t m[2];
            bool in[2];
            const int64_t c = 32 * y + lane % 4 * 8;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int row = 16 * g + lane / 4;
                m[g] = r0 + 32 * x + row;
                in[g] = m[g] < a.rows && c < a.cols;
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4*>(&v[g][j]) = *reinterpret_cast<const float4*>(&s[row * kLdS + lane % 4 * 8 + j]);
            }
            finish8<T, kDx, true, 2>(a, offset, v, none, m, in, c, 8);
            __builtin_amdgcn_wave_barrier();
        }
}

// dW of fp32 rows with dz = g, up to 64 inputs: memory and the matrix cores bound it alike (64 x 1920
// of 105730 rows 183 to 197 us, 4.4 TB/s and 0.8 PFLOP/s of bf16 products; by tiles 299 with the join).  A wave
// owns 64 inputs x 128 outputs and a run of rows, and needs no LDS: a lane has one column of x or g
// and eight rows in a row, which is what eight loads of whole lines bring (a row's 32 columns to
// each half of the wave).  The next rows' loads go to the registers that have just been cut.  The four
// waves of a block add their sums at the end, in order.  HB: db too.
template <bool HB>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) k_linear_dw(GemmArgs a)
{
    constexpr int FP = 2, FQ = 4;
    __shared__ float s[64][128 + 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // blocks with the same rows of x are neighbours; the last 128 outputs may reach into those before
    const int64_t at = xcd_order(blockIdx.x, gridDim.x), part = at / a.tc, own = at % a.tc * 128;
    const int64_t c0 = own + 128 < a.cols ? own : a.cols - 128;
    const int64_t n0 = part * a.run + wave * (a.run / 4), end = n0 + a.run / 4 < a.depth ? n0 + a.run / 4 : a.depth;
    // byte offsets of the lane's column and rows from those of the wave; inputs outside are the last again
    uint32_t op[FP];
#pragma unroll
    for (int x = 0; x < FP; ++x) {
        const int c = 32 * x + (lane & 31);
        op[x] = ((uint32_t)(lane >> 5) * 8u * (uint32_t)a.lda + (uint32_t)(c < a.rows ? c : (int)a.rows - 1)) * 4u;
    }
    const uint32_t oq = ((uint32_t)(lane >> 5) * 8u * (uint32_t)a.ldb + (uint32_t)(lane & 31)) * 4u;
    f16v acc[FP][FQ];
#pragma unroll
    for (int x = 0; x < FP; ++x)
#pragma unroll
        for (int y = 0; y < FQ; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;
    // rows n .. n + 15, the lane's eight from n + 8 (lane / 32) on
    float rx[FP][8], rg[FQ][8];
    auto fetch = [&](float(&r)[8], const void* base, int64_t ld, int64_t c, uint32_t offset, int64_t n) {
        const char* p = (const char*)((const float*)base + n * ld + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = *(const float*)(p + j * ld * 4 + offset);
    };
    // the last rows, fewer than 16: behind the end the last one again
    auto fetch_end = [&](float(&r)[8], const void* base, int64_t ld, int64_t c, int64_t n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t m = n + 8 * (lane >> 5) + j;
            r[j] = ((const float*)base)[(m < end ? m : end - 1) * ld + c];
        }
    };
    double sum[HB ? FQ : 1] = {};
    auto step = [&](int64_t n, auto last, auto next_x, auto next_g) {
        constexpr bool LAST = decltype(last)::value;
        b8 p[FP][3], q[3];
        const int64_t m = n + 8 * (lane >> 5);
#pragma unroll
        for (int x = 0; x < FP; ++x) {
            f8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = !LAST || m + j < end ? rx[x][j] : 0.0f;
            cut_along(v, p[x]);
            next_x(x);
        }
#pragma unroll
        for (int y = 0; y < FQ; ++y) {
            f8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = rg[y][j];
                if constexpr (LAST) v[j] = m + j < end ? v[j] : 0.0f;
            }
            next_g(y);
            if constexpr (HB) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[y] += (double)v[j];
            }
            cut_along(v, q);
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
                for (int i = 0; i <= o; ++i)
#pragma unroll
                    for (int x = 0; x < FP; ++x)
                        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[o - i], p[x][i], acc[x][y], 0, 0, 0);
        }
    };
    int64_t n = n0;
    if (n + 16 <= end) {
        auto next_x = [&](int x, int64_t n) { fetch(rx[x], a.A, a.lda, 0, op[x], n); };
        auto next_g = [&](int y, int64_t n) { fetch(rg[y], a.B, a.ldb, c0 + 32 * y, oq, n); };
#pragma unroll
        for (int x = 0; x < FP; ++x) next_x(x, n);
#pragma unroll
        for (int y = 0; y < FQ; ++y) next_g(y, n);
        for (; n + 16 <= end; n += 16) {
            const int64_t then = n + 32 <= end ? n + 16 : n;  // (behind the last whole step: that again, not used)
            step(n, std::false_type{}, [&](int x) { next_x(x, then); }, [&](int y) { next_g(y, then); });
        }
    }
    if (n < end) {
#pragma unroll
        for (int x = 0; x < FP; ++x) {
            const int64_t c = 32 * x + (lane & 31);
            fetch_end(rx[x], a.A, a.lda, c < a.rows ? c : a.rows - 1, n);
        }
#pragma unroll
        for (int y = 0; y < FQ; ++y) fetch_end(rg[y], a.B, a.ldb, c0 + 32 * y + (lane & 31), n);
        step(n, std::true_type{}, [](int) {}, [](int) {});
    }
    // a lane holds input lane % 32, outputs 8 g + 4 (lane / 32) + 0 .. 3 of each tile of 32
    for (int v = 0; v < 4; ++v) {
        if (v) __syncthreads();
        if (wave == v) {
#pragma unroll
            for (int x = 0; x < FP; ++x)
#pragma unroll
                for (int y = 0; y < FQ; ++y)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float4* to = reinterpret_cast<float4*>(&s[32 * x + (lane & 31)][32 * y + 8 * g + 4 * (lane >> 5)]);
                        float4 t{acc[x][y][4 * g], acc[x][y][4 * g + 1], acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
                        if (v) {
                            const float4 b = *to;
                            t.x += b.x;
                            t.y += b.y;
                            t.z += b.z;
                            t.w += b.w;
                        }
                        *to = t;
                    }
        }
    }
    __syncthreads();
    for (int b = tid; b < 64 * 128; b += 256) {
        const int64_t i = b / 128, c = c0 + b % 128;
        if (i < a.rows && c >= own) a.part[(part * a.rows + i) * a.cols + c] = s[i][b % 128];
    }
    if constexpr (HB) {
        __shared__ double sd[4][2][128];
#pragma unroll
        for (int y = 0; y < FQ; ++y) sd[wave][lane >> 5][32 * y + (lane & 31)] = sum[y];
        __syncthreads();
        if (tid < 128 && c0 + tid >= own) {
            double t = 0.0;
            for (int v = 0; v < 8; ++v) t += sd[v / 2][v % 2][tid];
            a.db_part[part * a.cols + c0 + tid] = t;
        }
    }
}

// Planes of rows: as they are, or dz = mask g act'(z) with its columns' sums.  A block takes
// 256 columns of a run of rows, eight rows at a time.  Bound by memory: dz of 16385 x 4096 bf16 with SiLU and
// dropout 124 to 132 us (671 MB, three planes of them, 5.2 TB/s); formed in the tiles of both products
// instead one number of it alone took 1.3 ms more.
template <class T, bool DZ, bool HZ>
__global__ void __launch_bounds__(256) k_linear_planes(PlaneArgs p)
{
    constexpr int NP = DZ ? kSlopePlanes<T, HZ> : kPlanes<T>;
    __shared__ double s[DZ ? 8 * 256 : 1];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t c = ((int64_t)blockIdx.x * 32 + lane) * 8;
    const int64_t n1 = ((int64_t)blockIdx.y + 1) * p.run < p.rows ? ((int64_t)blockIdx.y + 1) * p.run : p.rows;
    const uint64_t offset = drop_offset(p.g.drop);
    double sum[8] = {};
    if (c < p.cols) {
#pragma unroll 2
        for (int64_t n = (int64_t)blockIdx.y * p.run + tid / 32; n < n1; n += 8) {
            Raw8<T> r;
            r.load((const T*)p.x + n * p.ld + c);
            f8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = r[j];
            if constexpr (DZ) {
                float z[8] = {};
                if (HZ && p.g.Z) {
                    Raw8<T> q;
                    q.load((const T*)p.g.Z + n * p.g.ldz + c);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] = q[j];
                }
                slope8<HZ>(p.g, offset, v, z, n, (int32_t)(c / 8));
                if (p.g.db) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += (double)v[j];
                }
            }
            if (p.out) {
                b8 planes[NP];
                cut(v, planes);
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    *reinterpret_cast<b8*>(p.out + i * p.rows * p.cols + n * p.cols + c) = planes[i];
            }
        }
    }
    if constexpr (DZ) {
        if (!p.g.db) return;
#pragma unroll
        for (int j = 0; j < 8; ++j) s[tid / 32 * 256 + lane * 8 + j] = sum[j];
        __syncthreads();
        double t = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i * 256 + tid];
        const int64_t at = (int64_t)blockIdx.x * 256 + tid;
        if (at < p.cols) p.g.db_part[(int64_t)blockIdx.y * p.cols + at] = t;
    }
}

template <class T, int KIND, bool HZ>
hipError_t wide(const WideArgs& w, hipStream_t s)
{
    const dim3 grid((unsigned)(w.g.tr * w.g.tc * w.g.splits));
    if (w.side == 256) hipLaunchKernelGGL((k_linear_wide<T, KIND, HZ, 256, 256, 128, 64, 4>), grid, dim3(512), 0, s, w);
    else hipLaunchKernelGGL((k_linear_wide<T, KIND, HZ, 128, 128, 64, 64, 3>), grid, dim3(256), 0, s, w);
    return hipGetLastError();
}

template <class T, bool HZ>
hipError_t wide(int kind, const WideArgs& w, hipStream_t s)
{
    return kind == kFwd ? wide<T, kFwd, false>(w, s) : kind == kDx ? wide<T, kDx, HZ>(w, s) : wide<T, kDw, HZ>(w, s);
}

}  // namespace

hipError_t launch_linear_wide(int dtype, int kind, const WideArgs& w, hipStream_t s)
{
    // (fp32 operands have three planes either way)
    if (dtype == kF32) return wide<float, true>(kind, w, s);
    return w.g.Z ? wide<bf16_t, true>(kind, w, s) : wide<bf16_t, false>(kind, w, s);
}

hipError_t launch_linear_dx(int dtype, const WideArgs& w, hipStream_t s)
{
    auto go = [&](auto kernel, int rows) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv64(w.g.rows, rows)), dim3(256), 0, s, w);
    };
    const bool z = w.g.Z;
    if (w.g.cols <= 64) go(k_linear_dx<float, 64, 2, false>, 256);
    else if (dtype == kF32) z ? go(k_linear_dx<float, 128, 1, true>, 128) : go(k_linear_dx<float, 128, 1, false>, 128);
    else z ? go(k_linear_dx<bf16_t, 128, 1, true>, 128) : go(k_linear_dx<bf16_t, 128, 1, false>, 128);
    return hipGetLastError();
}

hipError_t launch_linear_dw(const GemmArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)(a.tc * a.splits));
    if (a.db) hipLaunchKernelGGL(k_linear_dw<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_linear_dw<false>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_linear_planes(int dtype, bool dz, const PlaneArgs& p, hipStream_t s)
{
    const dim3 grid((unsigned)cdiv64(p.cols, 256), (unsigned)cdiv64(p.rows, p.run));
    if (dtype == kF32) {
        if (dz) hipLaunchKernelGGL((k_linear_planes<float, true, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_linear_planes<float, false, false>), grid, dim3(256), 0, s, p);
    } else if (p.g.Z) {  // (bf16 rows are planes)
        hipLaunchKernelGGL((k_linear_planes<bf16_t, true, true>), grid, dim3(256), 0, s, p);
    } else {
        hipLaunchKernelGGL((k_linear_planes<bf16_t, true, false>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace cgtp
