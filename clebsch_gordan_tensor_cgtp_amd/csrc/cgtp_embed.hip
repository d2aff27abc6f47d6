// cgtp_embed.hip -- embedding of species (token) ids with a scale, and the
// gradient of its table by sorted ids.
//
//   out[n][c]   = s * T[ids[n]][c]                      (0 for an id outside the table)
//   dT[v][c]    = s * sum_{n: ids[n] = v} g[n][c]       (0 for a row without ids)
//
// Both are bound by memory.  The gradient sums rows that lie anywhere: the ids
// are sorted (stable radix sort, least significant digit first, integers
// only), the sorted positions are cut into runs of equal length, every run is
// summed in registers (fp64) by the lanes that own its channels, and rows
// whose ids span several runs are joined from the runs' partial sums in order.
// Nothing depends on the order in which blocks run.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "cgtp_internal.h"
#include "cgtp_train_internal.h"
#include "cgtp_vec.h"

namespace cgtp {
namespace {

constexpr int kThreads = 256;

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Blocks of a launch over `n` units of work: the kernels stride over what is
// left, so a launch stays below 2^32 threads.
constexpr int64_t kMaxBlocks = 1 << 22;
inline unsigned grid_of(int64_t n) { return (unsigned)(n < kMaxBlocks ? n : kMaxBlocks); }

// ---- forward ---------------------------------------------------------------------
// L lanes per row (CV = C / VEC accesses per row, at most 256 lanes), the rest
// of the block on further rows; kRows rows per lane so that the gathers of
// several rows are in flight behind their ids.
constexpr int kRows = 4;

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_fwd(int64_t N, int32_t V, int64_t CV, int32_t L, int64_t C,
                                                        const int32_t* __restrict__ ids, const T* __restrict__ table,
                                                        float scale, T* __restrict__ out, int64_t ld)
{
    const int32_t rl = (int32_t)threadIdx.x / L, lane = (int32_t)threadIdx.x - rl * L, RL = kThreads / L;
    if (rl >= RL) return;
    for (int64_t n0 = (int64_t)blockIdx.x * RL * kRows + rl; n0 < N; n0 += (int64_t)gridDim.x * RL * kRows) {
        int32_t id[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t n = n0 + (int64_t)k * RL;
            id[k] = ids[n < N ? n : n0];
            if (id[k] >= V) id[k] = -1;
        }
        for (int64_t q = lane; q < CV; q += L) {
            // loads stand outside any condition (row 0 for an id outside the table),
            // so that all of them are in flight together
            Raw<T, VEC> v[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) v[k].load(table + (int64_t)(id[k] >= 0 ? id[k] : 0) * C + q * VEC);
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int64_t n = n0 + (int64_t)k * RL;
                if (n >= N) continue;
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) o[j] = id[k] >= 0 ? v[k][j] * scale : 0.0f;
                store_vec<T, VEC>(out + n * ld + q * VEC, o);
            }
        }
    }
}

// ---- stable radix sort of (id, row) pairs, least significant digit first --------------
// kBits bits at a time.  Ids outside the table sort as the value V.
constexpr int kBits = 9, kDigits = 1 << kBits;

// p[0 .. n16) and t[0 .. tail) = 0, by blocks first .. first + blocks - 1
struct Clear {
    uint4* p;
    int64_t n16, tail;
    uint16_t* t;
    uint32_t blocks;
};

__device__ __forceinline__ void clear(const Clear& c, uint32_t block)
{
    const int64_t i = (int64_t)block * blockDim.x + threadIdx.x, step = (int64_t)c.blocks * blockDim.x;
    for (int64_t k = i; k < c.n16; k += step) c.p[k] = uint4{0, 0, 0, 0};
    for (int64_t k = i; k < c.tail; k += step) c.t[k] = 0;
}

__global__ void __launch_bounds__(kThreads) k_clear(Clear c) { clear(c, blockIdx.x); }

__device__ __forceinline__ int32_t key_of(int32_t id, int32_t V) { return id >= 0 && id < V ? id : V; }

// The wave's LDS accesses before this come before those after it (the hardware
// keeps a wave's LDS accesses in order; the compiler has to as well).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Rank of a key among its wave's keys of the same digit so far (cnt: the wave's
// counts, raised here).  The lanes with one digit find each other by setting their
// bits in mask[digit] (zero before and after): three LDS accesses, where comparing
// bit by bit takes seven vector instructions for each bit (a scatter of 50000 ids
// 7.0 us, bit by bit 7.8 us).
__device__ __forceinline__ int32_t rank_in_wave(int32_t d, bool in, unsigned long long* mask, int32_t* cnt)
{
    const int lane = threadIdx.x & 63;
    if (in) __hip_atomic_fetch_or(&mask[d], 1ull << lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
    wave_fence();
    const unsigned long long same = in ? mask[d] : 0ull;
    const unsigned long long below = same & ((1ull << lane) - 1);
    const int32_t r = in ? cnt[d] + (int32_t)__popcll(below) : 0;
    wave_fence();
    if (in && below == 0) {
        cnt[d] += (int32_t)__popcll(same);
        mask[d] = 0ull;
    }
    wave_fence();
    return r;
}

// exclusive sum over the block's THR threads; *all: the total.  s: [THR / 64]
template <int THR>
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* s, int32_t* all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    if (lane == 63) s[wave] = x;
    __syncthreads();
    int32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < THR / 64; ++w) {
        if (w < wave) before += s[w];
        sum += s[w];
    }
    __syncthreads();
    *all = sum;
    return before + x - v;
}

// -- up to kOneKeys keys: one block, key and row in one word, all passes in LDS, while
// the launch's other blocks clear the table
constexpr int kOneThreads = 1024, kOneWaves = kOneThreads / 64, kOnePer = 24;
constexpr int64_t kOneKeys = (int64_t)kOneThreads * kOnePer;

struct OneArgs {
    int32_t N, V, key_bits, row_bits;
    const int32_t* ids;
    int32_t *okey, *oval;
    Clear c;
};

template <int PER>
__global__ void __launch_bounds__(kOneThreads) k_sort_one(OneArgs a)
{
    // the exchanged words, and while ranks are formed the waves' masks
    constexpr int kWords = kOneThreads * PER, kMasks = 2 * kOneWaves * kDigits;
    __shared__ __attribute__((aligned(8))) uint32_t word[kWords > kMasks ? kWords : kMasks];
    __shared__ int32_t cnt[kOneWaves][kDigits];
    __shared__ int32_t s[kOneWaves];
    if (blockIdx.x > 0) {
        clear(a.c, blockIdx.x - 1);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t first = wave * 64 * PER + lane;  // a wave owns 64 PER keys in a row
    uint32_t w[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int32_t p = first + 64 * k;
        w[k] = (uint32_t)key_of(a.ids[p < a.N ? p : 0], a.V) << a.row_bits | (uint32_t)p;
    }
    for (int shift = 0; shift < a.key_bits; shift += kBits) {
        const int bits = a.key_bits - shift < kBits ? a.key_bits - shift : kBits;
        unsigned long long* mask = reinterpret_cast<unsigned long long*>(word) + wave * kDigits;
        if (shift > 0) __syncthreads();  // the words of the pass before are read
        for (int d = lane; d < kDigits; d += 64) {
            cnt[wave][d] = 0;
            mask[d] = 0ull;
        }
        wave_fence();
        int32_t rank[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k)
            rank[k] = rank_in_wave((int32_t)(w[k] >> (a.row_bits + shift)) & ((1 << bits) - 1), first + 64 * k < a.N, mask,
                                   cnt[wave]);
        __syncthreads();
        // first place of each digit, then of each wave in it
        int32_t sum = 0, all;
        if (tid < kDigits)
            for (int v = 0; v < kOneWaves; ++v) sum += cnt[v][tid];
        int32_t at = block_scan<kOneThreads>(tid < kDigits ? sum : 0, s, &all);
        if (tid < kDigits)
            for (int v = 0; v < kOneWaves; ++v) {
                const int32_t c = cnt[v][tid];
                cnt[v][tid] = at;
                at += c;
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (first + 64 * k < a.N)
                word[cnt[wave][(int32_t)(w[k] >> (a.row_bits + shift)) & ((1 << bits) - 1)] + rank[k]] = w[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (first + 64 * k < a.N) w[k] = word[first + 64 * k];
        // cnt is cleared by its own wave only, word written after two barriers
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int32_t p = first + 64 * k;
        if (p < a.N) {
            a.okey[p] = (int32_t)(w[k] >> a.row_bits);
            a.oval[p] = (int32_t)(w[k] & ((1u << a.row_bits) - 1));
        }
    }
}

// -- more keys: tiles of kTile keys, a block each; per pass the tiles' counts, their
// sums over earlier tiles (by each scattering block where the tiles are few, else by a
// launch of their own), and the scatter
constexpr int kWaves = kThreads / 64, kPer = 4, kTile = kThreads * kPer, kFewTiles = 64;

struct SortArgs {
    int64_t N;
    int32_t V, shift, tiles;
    const int32_t* ids;          // first pass: keys from here, values are the positions
    const int32_t *key, *val;    // later passes
    int32_t *okey, *oval;
    int32_t *hist, *total;       // [tiles][kDigits] (few tiles) or [kDigits][tiles]; [kDigits]
    Clear c;                     // first pass: the blocks beyond the tiles clear the table
};

__device__ __forceinline__ int32_t sort_key(const SortArgs& a, int64_t p)
{
    return a.ids ? key_of(a.ids[p], a.V) : a.key[p];
}

__device__ __forceinline__ int32_t& hist_at(const SortArgs& a, int32_t d, int32_t t)
{
    return a.hist[a.tiles <= kFewTiles ? (int64_t)t * kDigits + d : (int64_t)d * a.tiles + t];
}

__global__ void __launch_bounds__(kThreads) k_sort_hist(SortArgs a)
{
    __shared__ int32_t h[kDigits];
    if ((int32_t)blockIdx.x >= a.tiles) {
        clear(a.c, blockIdx.x - a.tiles);
        return;
    }
    for (int d = threadIdx.x; d < kDigits; d += kThreads) h[d] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kTile;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t p = t0 + k * kThreads + threadIdx.x;
        if (p < a.N) atomicAdd(&h[(sort_key(a, p) >> a.shift) & (kDigits - 1)], 1);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += kThreads) hist_at(a, d, blockIdx.x) = h[d];
}

// block d: exclusive sums of digit d's counts over the tiles, and their total
__global__ void __launch_bounds__(kThreads) k_sort_scan(SortArgs a)
{
    __shared__ int32_t s[kWaves];
    int32_t* h = a.hist + (int64_t)blockIdx.x * a.tiles;
    int32_t base = 0;
    for (int32_t t = 0; t < a.tiles; t += kThreads) {
        const int32_t i = t + (int32_t)threadIdx.x;
        const int32_t v = i < a.tiles ? h[i] : 0;
        int32_t all;
        const int32_t x = block_scan<kThreads>(v, s, &all);
        if (i < a.tiles) h[i] = base + x;
        base += all;
    }
    if (threadIdx.x == 0) a.total[blockIdx.x] = base;
}

__global__ void __launch_bounds__(kThreads) k_sort_scatter(SortArgs a)
{
    __shared__ int32_t cnt[kWaves][kDigits];  // keys of each digit met by each wave so far
    __shared__ unsigned long long mask[kWaves][kDigits];
    __shared__ int32_t s[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t p0 = (int64_t)blockIdx.x * kTile + (int64_t)wave * (kTile / kWaves) + lane;
    int32_t key[kPer], val[kPer], rank[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t p = p0 + 64 * k, q = p < a.N ? p : 0;
        key[k] = sort_key(a, q);
        val[k] = a.ids ? (int32_t)p : a.val[q];
    }
    // thread: digits 2 tid and 2 tid + 1, their counts in earlier tiles and in all
    constexpr int kEach = kDigits / kThreads;
    int32_t early[kEach], sum[kEach];
    if (a.tiles <= kFewTiles) {
        static_assert(kEach == 2, "two counts in one load");
        early[0] = early[1] = sum[0] = sum[1] = 0;
#pragma unroll 16
        for (int32_t t = 0; t < a.tiles; ++t) {
            const int2 c = *reinterpret_cast<const int2*>(&hist_at(a, 2 * tid, t));
            const bool before = t < (int32_t)blockIdx.x;
            sum[0] += c.x;
            sum[1] += c.y;
            early[0] += before ? c.x : 0;
            early[1] += before ? c.y : 0;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            early[e] = hist_at(a, kEach * tid + e, blockIdx.x);
            sum[e] = a.total[kEach * tid + e];
        }
    }
    for (int d = lane; d < kDigits; d += 64) {
        cnt[wave][d] = 0;
        mask[wave][d] = 0ull;
    }
    wave_fence();
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        rank[k] = rank_in_wave((key[k] >> a.shift) & (kDigits - 1), p0 + 64 * k < a.N, mask[wave], cnt[wave]);
    __syncthreads();
    {
        int32_t mine = 0, all;
#pragma unroll
        for (int e = 0; e < kEach; ++e) mine += sum[e];
        int32_t first = block_scan<kThreads>(mine, s, &all);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            int32_t at = first + early[e];
            first += sum[e];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int32_t c = cnt[w][kEach * tid + e];
                cnt[w][kEach * tid + e] = at;
                at += c;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (p0 + 64 * k >= a.N) continue;
        const int64_t to = cnt[wave][(key[k] >> a.shift) & (kDigits - 1)] + rank[k];
        a.okey[to] = key[k];
        a.oval[to] = val[k];
    }
}

// ---- sums over the sorted rows --------------------------------------------------------
// A block's run is RL R consecutive sorted positions, R for each group of L lanes.  A
// group writes a stretch of equal ids that lies inside its positions to its table row;
// the first and the last stretch, which may reach over the ends, meet those of the
// other groups in LDS, and what reaches over the run's ends goes to part[run][0] (it
// began before this run) or part[run][1] (it begins here and goes on).
struct SumArgs {
    int64_t N, C, CV, runs, ld;
    int32_t V, L, R, RL;
    float scale;
    const int32_t *key, *val;  // sorted ids and their rows
    double* part;              // [runs][2][C]
};

constexpr int kBatch = 8;  // rows in flight per lane

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_sum(SumArgs a, const T* __restrict__ grad, T* __restrict__ gtab)
{
    __shared__ double ends[2][VEC][kThreads];     // sums of the groups' first and last stretches
    __shared__ int32_t ids[2][kThreads];          // their ids; -1: the group has no positions
    __shared__ bool whole[kThreads];              // one stretch: the first
    const int32_t rl = (int32_t)threadIdx.x / a.L, lane = (int32_t)threadIdx.x - rl * a.L;
    const int64_t q = (int64_t)blockIdx.y * a.L + lane;
    const bool on = rl < a.RL && q < a.CV;
    for (int64_t run = blockIdx.x; run < a.runs; run += gridDim.x) {
        const int64_t b0 = run * a.R * a.RL, b1 = b0 + (int64_t)a.R * a.RL < a.N ? b0 + (int64_t)a.R * a.RL : a.N;
        const int32_t before = b0 > 0 ? a.key[b0 - 1] : -1, after = b1 < a.N ? a.key[b1] : -1;
        auto store = [&](int32_t id, const double (&acc)[VEC]) {
            if (id >= a.V) return;
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = (float)(acc[j] * (double)a.scale);
            store_vec<T, VEC>(gtab + (int64_t)id * a.C + q * VEC, v);
        };
        const int64_t p0 = b0 + (int64_t)rl * a.R, p1 = p0 + a.R < b1 ? p0 + a.R : b1;
        if (on) {
            int32_t cur = -1;
            bool first = true;
            double acc[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
            auto keep = [&](int which) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) ends[which][j][threadIdx.x] = acc[j];
                if (lane == 0) ids[which][rl] = cur;
            };
            if (p0 < p1) cur = a.key[p0];
            for (int64_t p = p0; p < p1; p += kBatch) {
                int32_t k[kBatch], row[kBatch];
                Raw<T, VEC> v[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int64_t at = p + u < p1 ? p + u : p;
                    k[u] = a.key[at];
                    row[u] = a.val[at];
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) v[u].load(grad + (int64_t)row[u] * a.ld + q * VEC);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (p + u >= p1) continue;
                    if (k[u] != cur) {
                        if (first) keep(0);
                        else store(cur, acc);
                        first = false;
                        cur = k[u];
#pragma unroll
                        for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
                    }
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[j] += (double)v[u][j];
                }
            }
            keep(first ? 0 : 1);
            if (lane == 0) whole[rl] = first;
        }
        __syncthreads();
        if (on && rl == 0) {
            int32_t open = -1;   // the stretch under way
            bool start = true;   // it began with the run
            double acc[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
            auto flush = [&](bool last) {
                const bool from = start && open == before, to = last && open == after;
                if (open >= 0 && open < a.V && (from || to)) {
                    double* d = a.part + (run * 2 + (from ? 0 : 1)) * a.C + q * VEC;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) d[j] = acc[j];
                } else if (open >= 0) {
                    store(open, acc);
                }
            };
            for (int32_t g = 0; g < a.RL; ++g) {
                const int32_t id = ids[0][g];
                if (id < 0) break;
                if (id != open) {
                    flush(false);
                    start = g == 0;
                    open = id;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[j] += ends[0][j][g * a.L + lane];
                if (!whole[g]) {
                    flush(false);
                    start = false;
                    open = ids[1][g];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[j] = ends[1][j][g * a.L + lane];
                }
            }
            flush(true);
        }
        __syncthreads();
    }
}

// Block (run, slice): if a stretch begins in this run and goes on after it, its
// partial sums from here to its end.
constexpr int kJoin = 256;

template <class T, int VEC>
__global__ void __launch_bounds__(kJoin) k_embed_join(SumArgs a, T* __restrict__ gtab)
{
    __shared__ double s[kJoin * VEC];
    const int64_t rows = (int64_t)a.R * a.RL;
    for (int64_t run = blockIdx.x; run + 1 < a.runs; run += gridDim.x) {  // conditions are the same for the whole block
        const int64_t p0 = run * rows, p1 = p0 + rows;
        const int32_t k = a.key[p1 - 1];
        if (k >= a.V || a.key[p1] != k) continue;
        if (a.key[p0] == k && p0 > 0 && a.key[p0 - 1] == k) continue;
        // the last run that begins with k: every round counts the probes that do
        // among kJoin spread over what is left
        int64_t last = run + 1, n = a.runs - last;
        while (n > 1) {
            const int64_t step = (n + kJoin - 1) / kJoin, at = threadIdx.x * step;
            const int c = __syncthreads_count(at < n && a.key[(last + at) * rows] == k);
            const int64_t left = n - (c - 1) * step;
            last += (c - 1) * step;
            n = step < left ? step : left;
        }
        const int32_t rl = (int32_t)threadIdx.x / a.L, RL = kJoin / a.L;
        const int64_t q = (int64_t)blockIdx.y * a.L + ((int32_t)threadIdx.x - rl * a.L);
        const bool ok = rl < RL && q < a.CV;
        double acc[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
        if (ok) {
#pragma unroll 8
            for (int64_t r = run + rl; r <= last; r += RL) {
                const double* d = a.part + (r * 2 + (r == run ? 1 : 0)) * a.C + q * VEC;
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[j] += d[j];
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[j * kJoin + threadIdx.x] = acc[j];
        __syncthreads();
        if (ok && rl == 0) {
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                double t = 0.0;
                for (int32_t r = 0; r < RL; ++r) t += s[j * kJoin + r * a.L + (int32_t)threadIdx.x];
                v[j] = (float)(t * (double)a.scale);
            }
            store_vec<T, VEC>(gtab + (int64_t)k * a.C + q * VEC, v);
        }
        __syncthreads();
    }
}

struct EmbedLayout {
    int64_t R, RL, L, runs, tiles;
    bool wide;
    size_t key[2], val[2], hist, total, part, bytes;
};

// wide: 16-byte accesses
EmbedLayout embed_layout(const EmbedShape& e, bool wide)
{
    EmbedLayout w{};
    w.wide = wide;
    const int64_t cv = wide ? e.C / (16 / dtype_size(e.dtype)) : e.C;
    w.L = cv < kThreads ? cv : kThreads;
    w.RL = kThreads / w.L;
    // Positions of a group: enough groups to fill the chip (about 2^18 lanes), and 16
    // at least where they are many, so that hot ids leave fewer partial sums (50000
    // x 128: sum and join 14.2 us, with 8 positions 15.8 us)
    const int64_t R = cdiv64(e.N * cv, 1 << 18), least = e.N > 16384 ? 16 : kBatch;
    w.R = cdiv64(R < least ? least : R > 64 ? 64 : R, kBatch) * kBatch;
    w.runs = cdiv64(e.N, w.R * w.RL);
    w.tiles = cdiv64(e.N, kTile);
    size_t o = 0;
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o += align256((size_t)bytes);
        return at;
    };
    for (int k = 0; k < 2; ++k) {
        w.key[k] = take(4 * e.N);
        w.val[k] = take(4 * e.N);
    }
    w.hist = take(4 * kDigits * w.tiles);
    w.total = take(4 * kDigits);
    w.part = take((int64_t)sizeof(double) * 2 * w.runs * e.C);
    w.bytes = o > 0 ? o : 256;
    return w;
}

template <class T, int VEC>
hipError_t embed_fwd(const EmbedShape& e, const int32_t* ids, const void* table, void* out, hipStream_t s)
{
    const int64_t CV = e.C / VEC;
    const int32_t L = (int32_t)(CV < kThreads ? CV : kThreads), RL = kThreads / L;
    hipLaunchKernelGGL((k_embed_fwd<T, VEC>), dim3(grid_of(cdiv64(e.N, (int64_t)RL * kRows))), dim3(kThreads), 0, s,
                       e.N, (int32_t)e.V, CV, L, e.C, ids, (const T*)table, e.scale, (T*)out, e.ld);
    return hipGetLastError();
}

template <class T, int VEC>
hipError_t embed_sum(const EmbedShape& e, const EmbedLayout& w, const int32_t* key, const int32_t* val,
                     const void* grad, void* gtab, double* part, hipStream_t s)
{
    SumArgs a{};
    a.N = e.N;
    a.C = e.C;
    a.CV = e.C / VEC;
    a.runs = w.runs;
    a.ld = e.ld;
    a.V = (int32_t)e.V;
    a.L = (int32_t)w.L;
    a.R = (int32_t)w.R;
    a.RL = (int32_t)w.RL;
    a.scale = e.scale;
    a.key = key;
    a.val = val;
    a.part = part;
    const unsigned slices = (unsigned)cdiv64(a.CV, a.L);
    hipLaunchKernelGGL((k_embed_sum<T, VEC>), dim3(grid_of(w.runs), slices), dim3(kThreads), 0, s, a, (const T*)grad,
                       (T*)gtab);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || w.runs < 2) return err;
    hipLaunchKernelGGL((k_embed_join<T, VEC>), dim3(grid_of(w.runs - 1), slices), dim3(kJoin), 0, s, a, (T*)gtab);
    return hipGetLastError();
}

// The table's rows set to zero, by the blocks of a launch beside its other work.
Clear clear_of(const EmbedShape& e, void* gtab, int threads)
{
    const int64_t bytes = e.V * e.C * dtype_size(e.dtype);
    Clear c{};
    c.n16 = ((uintptr_t)gtab & 15u) == 0 ? bytes / 16 : 0;
    c.tail = (bytes - 16 * c.n16) / 2;
    c.p = (uint4*)gtab;
    c.t = (uint16_t*)((char*)gtab + 16 * c.n16);
    const int64_t blocks = cdiv64(c.n16 > c.tail ? c.n16 : c.tail, (int64_t)threads * 4);
    c.blocks = (uint32_t)(blocks < 4096 ? blocks : 4096);
    return c;
}

int bits_of(int64_t v)  // of 0 .. v
{
    int b = 0;
    while ((v >> b) != 0) ++b;
    return b;
}

}  // namespace

size_t embed_bwd_workspace_bytes(const EmbedShape& e)
{
    // of either form: which one runs depends on the arrays' alignment
    const size_t n = embed_layout(e, false).bytes;
    if (e.C * dtype_size(e.dtype) % 16 != 0) return n;
    const size_t m = embed_layout(e, true).bytes;
    return n > m ? n : m;
}

hipError_t launch_embed_fwd(const EmbedShape& e, const int32_t* ids, const void* table, void* out, hipStream_t s)
{
    if (e.N == 0) return hipSuccess;
    const int64_t es = dtype_size(e.dtype);
    const bool wide = e.C * es % 16 == 0 && aligned_rows(out, e.ld, es) && aligned_rows(table, e.C, es);
    if (e.dtype == kF32)
        return wide ? embed_fwd<float, kWide<float>>(e, ids, table, out, s) : embed_fwd<float, 1>(e, ids, table, out, s);
    return wide ? embed_fwd<bf16_t, kWide<bf16_t>>(e, ids, table, out, s) : embed_fwd<bf16_t, 1>(e, ids, table, out, s);
}

hipError_t launch_embed_bwd(const EmbedShape& e, const int32_t* ids, const void* grad, void* gtab, void* ws,
                            hipStream_t s)
{
    if (e.N == 0) {
        const Clear c = clear_of(e, gtab, kThreads);
        hipLaunchKernelGGL(k_clear, dim3(c.blocks), dim3(kThreads), 0, s, c);
        return hipGetLastError();
    }
    const int64_t es = dtype_size(e.dtype);
    const bool wide = e.C * es % 16 == 0 && aligned_rows(grad, e.ld, es) && aligned_rows(gtab, e.C, es);
    const EmbedLayout w = embed_layout(e, wide);
    char* base = (char*)ws;
    const int32_t *key, *val;
    const int key_bits = bits_of(e.V), row_bits = bits_of(e.N - 1);  // keys are 0 .. V
    if (e.N <= kOneKeys && key_bits + row_bits <= 32) {
        OneArgs a{};
        a.N = (int32_t)e.N;
        a.V = (int32_t)e.V;
        a.key_bits = key_bits;
        a.row_bits = row_bits;
        a.ids = ids;
        a.okey = (int32_t*)(base + w.key[0]);
        a.oval = (int32_t*)(base + w.val[0]);
        a.c = clear_of(e, gtab, kOneThreads);
        const dim3 grid(1 + a.c.blocks), thr(kOneThreads);
        switch (cdiv64(e.N, 4 * kOneThreads)) {  // the time goes with the keys of a thread
            case 1: hipLaunchKernelGGL(k_sort_one<4>, grid, thr, 0, s, a); break;
            case 2: hipLaunchKernelGGL(k_sort_one<8>, grid, thr, 0, s, a); break;
            case 3: hipLaunchKernelGGL(k_sort_one<12>, grid, thr, 0, s, a); break;
            case 4: hipLaunchKernelGGL(k_sort_one<16>, grid, thr, 0, s, a); break;
            case 5: hipLaunchKernelGGL(k_sort_one<20>, grid, thr, 0, s, a); break;
            default: hipLaunchKernelGGL(k_sort_one<kOnePer>, grid, thr, 0, s, a); break;
        }
        key = a.okey;
        val = a.oval;
    } else {
        SortArgs a{};
        a.N = e.N;
        a.V = (int32_t)e.V;
        a.tiles = (int32_t)w.tiles;
        a.hist = (int32_t*)(base + w.hist);
        a.total = (int32_t*)(base + w.total);
        int to = 0;
        for (int shift = 0; shift < key_bits; shift += kBits) {
            a.shift = shift;
            a.ids = shift == 0 ? ids : nullptr;
            a.key = (const int32_t*)(base + w.key[to ^ 1]);
            a.val = (const int32_t*)(base + w.val[to ^ 1]);
            a.okey = (int32_t*)(base + w.key[to]);
            a.oval = (int32_t*)(base + w.val[to]);
            a.c = shift == 0 ? clear_of(e, gtab, kThreads) : Clear{};
            hipLaunchKernelGGL(k_sort_hist, dim3((unsigned)w.tiles + a.c.blocks), dim3(kThreads), 0, s, a);
            if (w.tiles > kFewTiles) hipLaunchKernelGGL(k_sort_scan, dim3(kDigits), dim3(kThreads), 0, s, a);
            hipLaunchKernelGGL(k_sort_scatter, dim3((unsigned)w.tiles), dim3(kThreads), 0, s, a);
            to ^= 1;
        }
        key = (const int32_t*)(base + w.key[to ^ 1]);
        val = (const int32_t*)(base + w.val[to ^ 1]);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    double* part = (double*)(base + w.part);
    if (e.dtype == kF32)
        return wide ? embed_sum<float, kWide<float>>(e, w, key, val, grad, gtab, part, s)
                    : embed_sum<float, 1>(e, w, key, val, grad, gtab, part, s);
    return wide ? embed_sum<bf16_t, kWide<bf16_t>>(e, w, key, val, grad, gtab, part, s)
                : embed_sum<bf16_t, 1>(e, w, key, val, grad, gtab, part, s);
}

}  // namespace cgtp
