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

#include <type_traits>

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
// several rows are in flight behind their ids.  16385 rows x 1024 bf16 of 65536: 9.8 us
// (6.9 TB/s read and written); 10^6 rows x 128 fp32 of a table that L2 holds: 88 us
// (5.8 TB/s written, what a plain fill reaches is 6.8); 2000 x 128: 3.5 us, a launch.
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
__device__ __forceinline__ int32_t rank_in_wave(int32_t d, bool in, uint32_t (*mask)[2], int32_t* cnt)
{
    const int lane = threadIdx.x & 63;
    if (in)
        __hip_atomic_fetch_or(&mask[d][lane >> 5], 1u << (lane & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
    wave_fence();
    const unsigned long long same = in ? (unsigned long long)mask[d][1] << 32 | mask[d][0] : 0ull;
    const unsigned long long below = same & ((1ull << lane) - 1);
    const int32_t r = in ? cnt[d] + (int32_t)__popcll(below) : 0;
    wave_fence();
    if (in && below == 0) {
        cnt[d] += (int32_t)__popcll(same);
        mask[d][0] = mask[d][1] = 0u;
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
// the launch's other blocks clear the table.  One compute unit's LDS accesses bound it:
// 16385 ids of 65536, two passes, beside a table of 134 MB 28 us (the clearing alone takes
// 20.7 us, 6.5 TB/s).  Ranking every other key by votes on its bits gained 0.7 us, not
// worth a second way; 64-bit masks instead of two halves cost as much.
constexpr int kOneThreads = 1024, kOneWaves = kOneThreads / 64, kOnePer = 24;
constexpr int64_t kOneKeys = (int64_t)kOneThreads * kOnePer;

struct OneArgs {
    int32_t N, V, key_bits, row_bits;
    const int32_t* ids;
    int32_t *okey, *oval;
    Clear c;
};

template <int PER>
struct OneLds {
    // the exchanged words, and while ranks are formed the waves' masks
    static constexpr int kWords = kOneThreads * PER, kMasks = 2 * kOneWaves * kDigits;
    __attribute__((aligned(8))) uint32_t word[kWords > kMasks ? kWords : kMasks];
    int32_t cnt[kOneWaves][kDigits];
    int32_t s[kOneWaves];
};

// The words key << row_bits | position of N ids, sorted: in x.word by place (after a
// barrier), and this thread's in w.
template <int PER>
__device__ __forceinline__ void sort_one(const int32_t* __restrict__ ids, int32_t N, int32_t V, int32_t key_bits,
                                         int32_t row_bits, OneLds<PER>& x, uint32_t (&w)[PER])
{
    auto& word = x.word;
    auto& cnt = x.cnt;
    auto& s = x.s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t first = wave * 64 * PER + lane;  // a wave owns 64 PER keys in a row
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int32_t p = first + 64 * k;
        w[k] = (uint32_t)key_of(ids[p < N ? p : 0], V) << row_bits | (uint32_t)p;
    }
    for (int shift = 0; shift < key_bits; shift += kBits) {
        const int bits = key_bits - shift < kBits ? key_bits - shift : kBits;
        uint32_t(*mask)[2] = reinterpret_cast<uint32_t(*)[2]>(word) + wave * kDigits;
        if (shift > 0) __syncthreads();  // the words of the pass before are read
        for (int d = lane; d < kDigits; d += 64) {
            cnt[wave][d] = 0;
            mask[d][0] = mask[d][1] = 0u;
        }
        wave_fence();
        int32_t rank[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int32_t d = (int32_t)(w[k] >> (row_bits + shift)) & ((1 << bits) - 1);
            rank[k] = rank_in_wave(d, first + 64 * k < N, mask, cnt[wave]);
        }
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
            if (first + 64 * k < N)
                word[cnt[wave][(int32_t)(w[k] >> (row_bits + shift)) & ((1 << bits) - 1)] + rank[k]] = w[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (first + 64 * k < N) w[k] = word[first + 64 * k];
        // cnt is cleared by its own wave only, word written after two barriers
    }
}

template <int PER>
__global__ void __launch_bounds__(kOneThreads) k_sort_one(OneArgs a)
{
    __shared__ OneLds<PER> x;
    if (blockIdx.x > 0) {
        clear(a.c, blockIdx.x - 1);
        return;
    }
    uint32_t w[PER];
    sort_one<PER>(a.ids, a.N, a.V, a.key_bits, a.row_bits, x, w);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int32_t p = ((int)threadIdx.x >> 6) * 64 * PER + ((int)threadIdx.x & 63) + 64 * k;
        if (p < a.N) {
            a.okey[p] = (int32_t)(w[k] >> a.row_bits);
            a.oval[p] = (int32_t)(w[k] & ((1u << a.row_bits) - 1));
        }
    }
}

// -- more keys: tiles of kTile keys, a block each; per pass the tiles' counts, their
// sums over earlier tiles (by each scattering block where the tiles are few, else by a
// launch of their own), and the scatter.  Latency and launches: 50000 ids, one pass, 3.9 +
// 6.9 us; 10^6 ids 10.1 + 5.2 + 9.1 us.
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
    __shared__ __attribute__((aligned(8))) uint32_t mask[kWaves][kDigits][2];
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
        mask[wave][d][0] = mask[wave][d][1] = 0u;
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
// Bound by the gathered rows: 10^6 rows x 128 fp32 100 us (5.1 TB/s), 50000 x 128 7.5 us
// (3.4 TB/s), 16385 x 1024 bf16 13.7 us (2.4 TB/s, and the rows of some thousand ids written).
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

constexpr int kBatch = 8;    // rows in flight per lane
// Groups of a block, at most: a stretch adds its groups one by one (16385 x 8 in bf16:
// sort, sum and join 45 us, where 256 groups joined by one of them took 125 us).
constexpr int kGroups = 32;

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
            double v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = acc[j] * (double)a.scale;
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
        // The group in which a stretch begins adds what the groups after it hold.
        const int32_t head = on ? ids[0][rl] : -1;
        if (head >= 0) {
            auto flush = [&](int32_t id, const double (&acc)[VEC], bool from, bool to) {
                if (id < a.V && (from || to)) {
                    double* d = a.part + (run * 2 + (from ? 0 : 1)) * a.C + q * VEC;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) d[j] = acc[j];
                } else {
                    store(id, acc);
                }
            };
            const bool one = whole[rl];
            const bool begins = rl == 0 || (whole[rl - 1] ? ids[0][rl - 1] : ids[1][rl - 1]) != head;
            double acc[VEC];
            if (begins && !one) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[j] = ends[0][j][threadIdx.x];
                flush(head, acc, rl == 0 && head == before, false);
            }
            if (begins || !one) {  // the last stretch
                const int32_t id = one ? head : ids[1][rl];
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[j] = ends[one ? 0 : 1][j][threadIdx.x];
                int32_t g = rl + 1;
                bool goes = true;
                for (; goes && g < a.RL && ids[0][g] == id; ++g) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[j] += ends[0][j][g * a.L + lane];
                    goes = whole[g];
                }
                // it reaches the run's end if no group holds anything else
                flush(id, acc, one && rl == 0 && id == before,
                      goes && (g == a.RL || ids[0][g] < 0) && id == after);
            }
        }
        __syncthreads();
    }
}

// ---- few ids and a small table: the whole gradient in one launch --------------------------
// A small call is its launches: three of them take 13.7 us for 2000 x 128 of 10 ids, this
// 8.7 us (4096 x 128 of 4096: 20.6 and 18.3 us; a table of 4096 x 1024 no longer gains: 23.4
// and 25.5 us).  Every block sorts all ids for itself and sums LANES accesses of each row: 4,
// or 16 where fours would be more blocks than compute units (409 x 1778 fp32 12.8 -> 7.3 us;
// 4000 x 33, few blocks either way, 11.5 us with 4 and 16.5 with 16).  Its groups of LANES
// lanes take equal shares of the sorted positions; a group stores the stretches
// that lie inside its share, and a segmented sum over the groups (by shuffles in a wave,
// through LDS across waves) finishes those that reach over shares.
constexpr int kFewPer = 4;
constexpr int64_t kFewKeys = (int64_t)kOneThreads * kFewPer, kFewRows = 4096, kFewTable = 1 << 21;

struct FewArgs {
    int32_t N, V, key_bits, row_bits;
    int64_t C, CV, ld;
    float scale;
    const int32_t* ids;
};

template <class T, int VEC, int LANES>
__global__ void __launch_bounds__(kOneThreads) k_embed_few(FewArgs a, const T* __restrict__ grad, T* __restrict__ gtab)
{
    constexpr int kShares = kOneThreads / LANES;  // groups
    __shared__ OneLds<kFewPer> x;
    __shared__ double wsum[kOneWaves][LANES][VEC];  // of a wave's last stretch
    __shared__ bool wnew[kOneWaves];                    // it begins in that wave
    const int tid = threadIdx.x, wave = tid >> 6, l = tid % LANES, g = tid / LANES;
    const int64_t q = (int64_t)blockIdx.x * LANES + l;
    const bool on = q < a.CV;
    T* const col = gtab + q * VEC;
    if (on) {  // the sort's barriers put these stores before those of the sums
        float zero[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) zero[j] = 0.0f;
        for (int64_t v = g; v < a.V; v += kShares) store_vec<T, VEC>(col + v * a.C, zero);
    }
    uint32_t w[kFewPer];
    sort_one<kFewPer>(a.ids, a.N, a.V, a.key_bits, a.row_bits, x, w);
    __syncthreads();
    auto store = [&](int32_t id, const double (&sum)[VEC]) {
        if (!on || id >= a.V) return;
        double v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = sum[j] * (double)a.scale;
        store_vec<T, VEC>(col + (int64_t)id * a.C, v);
    };
    auto key = [&](int32_t p) { return (int32_t)(x.word[p] >> a.row_bits); };
    const int32_t R = (a.N + kShares - 1) / kShares;
    const int32_t p0 = g * R < a.N ? g * R : a.N, p1 = p0 + R < a.N ? p0 + R : a.N;
    const int32_t before = p0 > 0 ? key(p0 - 1) : -1, after = p1 < a.N ? key(p1) : -1;
    const T* const from = grad + (on ? q : 0) * VEC;
    double head[VEC], sum[VEC];  // of the first stretch and of the last
#pragma unroll
    for (int j = 0; j < VEC; ++j) head[j] = sum[j] = 0.0;
    int32_t first = -1, cur = -1;  // their ids
    bool whole = true;             // they are one
    if (p0 < p1) first = cur = key(p0);
    for (int32_t p = p0; p < p1; p += kBatch) {
        int32_t k[kBatch];
        Raw<T, VEC> v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t o = x.word[p + u < p1 ? p + u : p];
            k[u] = (int32_t)(o >> a.row_bits);
            v[u].load(from + (int64_t)(o & ((1u << a.row_bits) - 1)) * a.ld);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (p + u >= p1) continue;
            if (k[u] != cur) {
                if (!whole) store(cur, sum);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (whole) head[j] = sum[j];
                    sum[j] = 0.0;
                }
                whole = false;
                cur = k[u];
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] += (double)v[u][j];
        }
    }
    // sums of the last stretches from where they begin (`begun`), or from the wave's first group
    bool begun = p0 >= p1 || !whole || first != before;
#pragma unroll
    for (int d = LANES; d < 64; d *= 2) {
        const int b = __shfl_up((int)begun, d, 64);
        double t[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[j] = __shfl_up(sum[j], d, 64);
        if ((tid & 63) >= d && !begun) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] += t[j];
            begun = b != 0;
        }
    }
    if ((tid & 63) >= 64 - LANES) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) wsum[wave][l][j] = sum[j];
        if (l == 0) wnew[wave] = begun;
    }
    __syncthreads();
    double carry[VEC];  // of the stretch that enters this wave
#pragma unroll
    for (int j = 0; j < VEC; ++j) carry[j] = 0.0;
    for (int v = 0; v < wave; ++v) {
        const bool fresh = wnew[v];
#pragma unroll
        for (int j = 0; j < VEC; ++j) carry[j] = (fresh ? 0.0 : carry[j]) + wsum[v][l][j];
    }
    double enters[VEC];  // of the stretch that enters this group
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if (!begun) sum[j] += carry[j];
        enters[j] = __shfl_up(sum[j], LANES, 64);
        if ((tid & 63) < LANES) enters[j] = carry[j];
    }
    if (p0 >= p1) return;
    if (!whole) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) head[j] += first == before ? enters[j] : 0.0;
        store(first, head);
    }
    if (cur != after) store(cur, sum);
}

// Block (run, slice): if a stretch begins in this run and goes on after it, its
// partial sums from here to its end.  Latency: keys, one or two rounds of the search,
// partial sums, in turn (391 runs 6.5 us, 7815 runs 18.6 us, x 128 fp32).  Where a row is
// 256 accesses or more, each lane adds all of a hot id's runs by itself: 40000 x 1024 fp32 of
// six ids, 1000 runs, 50 us beside 27 us of sums.
constexpr int kJoin = 256;

template <class T, int VEC>
__global__ void __launch_bounds__(kJoin) k_embed_join(SumArgs a, T* __restrict__ gtab)
{
    __shared__ double s[kJoin * VEC];
    const int64_t rows = (int64_t)a.R * a.RL;
    for (int64_t run = blockIdx.x; run + 1 < a.runs; run += gridDim.x) {  // conditions are the same for the whole block
        const int64_t p0 = run * rows, p1 = p0 + rows;
        // the last run that begins with k: among the kJoin runs that follow (these
        // loads go with the others, ahead of the conditions), and where that is not
        // the end, by rounds that count probes spread over what is left
        int64_t last = run + 1, n = a.runs - last;
        const int32_t probe = a.key[(last + ((int64_t)threadIdx.x < n ? (int64_t)threadIdx.x : 0)) * rows];
        const int32_t k = a.key[p1 - 1], next = a.key[p1], head = a.key[p0], before = a.key[p0 > 0 ? p0 - 1 : 0];
        if (k >= a.V || next != k) continue;
        if (head == k && p0 > 0 && before == k) continue;
        const int begin = __syncthreads_count((int64_t)threadIdx.x < n && probe == k);
        last += begin - 1;
        n = begin == kJoin ? n - (kJoin - 1) : 1;
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
        for (int32_t m = RL; m > 1;) {  // by halves
            const int32_t up = (m + 1) / 2;
            if (ok && rl < m / 2) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[j * kJoin + threadIdx.x] += s[j * kJoin + up * a.L + threadIdx.x];
            }
            m = up;
            __syncthreads();
        }
        if (ok && rl == 0) {
            double v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = s[j * kJoin + threadIdx.x] * (double)a.scale;
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
    w.RL = kThreads / w.L < kGroups ? kThreads / w.L : kGroups;
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

int bits_of(int64_t v)  // of 0 .. v
{
    int b = 0;
    while ((v >> b) != 0) ++b;
    return b;
}

template <class T, int VEC>
hipError_t embed_few(const EmbedShape& e, const int32_t* ids, const void* grad, void* gtab, hipStream_t s)
{
    FewArgs a{};
    a.N = (int32_t)e.N;
    a.V = (int32_t)e.V;
    a.key_bits = bits_of(e.V);
    a.row_bits = bits_of(e.N - 1);
    a.C = e.C;
    a.CV = e.C / VEC;
    a.ld = e.ld;
    a.scale = e.scale;
    a.ids = ids;
    auto launch = [&](auto lanes) {
        constexpr int kLanes = decltype(lanes)::value;
        hipLaunchKernelGGL((k_embed_few<T, VEC, kLanes>), dim3((unsigned)cdiv64(a.CV, kLanes)), dim3(kOneThreads), 0, s,
                           a, (const T*)grad, (T*)gtab);
    };
    // blocks of few accesses while there are no more of them than compute units (256)
    if (a.CV <= 4 * 256) launch(std::integral_constant<int, 4>{});
    else launch(std::integral_constant<int, 16>{});
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
    const unsigned threads = (unsigned)(cdiv64(w.L * w.RL, 64) * 64);
    hipLaunchKernelGGL((k_embed_sum<T, VEC>), dim3(grid_of(w.runs), slices), dim3(threads), 0, s, a, (const T*)grad,
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
    if (e.N <= kFewKeys && e.V <= kFewRows && e.V * e.C <= kFewTable) {
        if (e.dtype == kF32)
            return wide ? embed_few<float, kWide<float>>(e, ids, grad, gtab, s) : embed_few<float, 1>(e, ids, grad, gtab, s);
        return wide ? embed_few<bf16_t, kWide<bf16_t>>(e, ids, grad, gtab, s) : embed_few<bf16_t, 1>(e, ids, grad, gtab, s);
    }
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
