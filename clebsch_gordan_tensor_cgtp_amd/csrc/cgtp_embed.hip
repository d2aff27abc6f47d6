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
            id[k] = n < N ? ids[n] : -1;
        }
        for (int64_t q = lane; q < CV; q += L) {
            float v[kRows][VEC];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (id[k] >= 0 && id[k] < V) {
                    load_vec<T, VEC>(v[k], table + (int64_t)id[k] * C + q * VEC);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) v[k][j] = 0.0f;
                }
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int64_t n = n0 + (int64_t)k * RL;
                if (n >= N) continue;
                if (id[k] >= 0 && id[k] < V)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) v[k][j] *= scale;
                store_vec<T, VEC>(out + n * ld + q * VEC, v[k]);
            }
        }
    }
}

// ---- stable radix sort of (id, row) pairs, eight bits at a time ----------------------
// Tiles of kTile consecutive keys, one block each; a wave owns kTile / 4
// consecutive keys of its tile.  Ids outside the table sort as the value V.
constexpr int kDigit = 256, kWaves = kThreads / 64, kPer = 8, kTile = kThreads * kPer;

struct SortArgs {
    int64_t N;
    int32_t V, shift, tiles;
    const int32_t* ids;          // first pass: keys from here, values are the positions
    const int32_t *key, *val;    // later passes
    int32_t *okey, *oval;
    int32_t *hist, *total;       // [256][tiles], [256]
};

__device__ __forceinline__ int32_t sort_key(const SortArgs& a, int64_t p)
{
    if (a.ids) {
        const int32_t v = a.ids[p];
        return v >= 0 && v < a.V ? v : a.V;
    }
    return a.key[p];
}

__global__ void __launch_bounds__(kThreads) k_sort_hist(SortArgs a)
{
    __shared__ int32_t h[kDigit];
    h[threadIdx.x] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kTile;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t p = t0 + k * kThreads + threadIdx.x;
        if (p < a.N) atomicAdd(&h[(sort_key(a, p) >> a.shift) & (kDigit - 1)], 1);
    }
    __syncthreads();
    a.hist[(int64_t)threadIdx.x * a.tiles + blockIdx.x] = h[threadIdx.x];
}

// exclusive sum over the block's threads of v; *all: the total.  s: [kWaves + 1]
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
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += s[w];
        sum += s[w];
    }
    __syncthreads();
    *all = sum;
    return before + x - v;
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
        const int32_t x = block_scan(v, s, &all);
        if (i < a.tiles) h[i] = base + x;
        base += all;
    }
    if (threadIdx.x == 0) a.total[blockIdx.x] = base;
}

__global__ void __launch_bounds__(kThreads) k_sort_scatter(SortArgs a)
{
    __shared__ int32_t cnt[kWaves][kDigit];  // keys of each digit met by each wave so far
    __shared__ int32_t s[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) cnt[w][tid] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * kTile + (int64_t)wave * (kTile / kWaves) + lane;
    int32_t key[kPer], rank[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t p = p0 + 64 * k;
        key[k] = p < a.N ? sort_key(a, p) : -1;
    }
    // rank of a key among its wave's earlier keys of the same digit: those of
    // earlier rounds (cnt) and those of lower lanes (equal-digit mask)
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const bool in = p0 + 64 * k < a.N;
        const int32_t d = (key[k] >> a.shift) & (kDigit - 1);
        uint64_t same = __ballot(in);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const uint64_t m = __ballot((d >> b) & 1);
            same &= ((d >> b) & 1) ? m : ~m;
        }
        const uint64_t below = same & ((1ull << lane) - 1);
        rank[k] = in ? cnt[wave][d] + (int32_t)__popcll(below) : 0;
        __builtin_amdgcn_wave_barrier();
        if (in && below == 0) cnt[wave][d] += (int32_t)__popcll(same);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // thread d: digit d's first place for this tile, then for each wave
    {
        int32_t all;
        const int32_t first = block_scan(a.total[tid], s, &all);
        int32_t at = first + a.hist[(int64_t)tid * a.tiles + blockIdx.x];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int32_t c = cnt[w][tid];
            cnt[w][tid] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t p = p0 + 64 * k;
        if (p >= a.N) continue;
        const int32_t d = (key[k] >> a.shift) & (kDigit - 1);
        const int64_t to = cnt[wave][d] + rank[k];
        a.okey[to] = key[k];
        a.oval[to] = a.ids ? (int32_t)p : a.val[p];
    }
}

// ---- sums over the sorted rows --------------------------------------------------------
// A run is R consecutive sorted positions.  A group of L lanes walks one run;
// a stretch of equal ids that lies inside the run is written to its table row,
// one that reaches over the run's ends goes to part[run][0] (it began before
// this run) or part[run][1] (it begins here and goes on).
struct SumArgs {
    int64_t N, C, CV, runs, ld;
    int32_t V, L, R;
    float scale;
    const int32_t *key, *val;  // sorted ids and their rows
    double* part;              // [runs][2][C]
};

constexpr int kBatch = 8;  // rows in flight per lane

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_sum(SumArgs a, const T* __restrict__ grad, T* __restrict__ gtab)
{
    const int32_t rl = (int32_t)threadIdx.x / a.L, RL = kThreads / a.L;
    const int64_t q = (int64_t)blockIdx.y * a.L + ((int32_t)threadIdx.x - rl * a.L);
    if (rl >= RL || q >= a.CV) return;
    for (int64_t run = (int64_t)blockIdx.x * RL + rl; run < a.runs; run += (int64_t)gridDim.x * RL) {
        const int64_t p0 = run * a.R, p1 = p0 + a.R < a.N ? p0 + a.R : a.N;
        const int32_t before = p0 > 0 ? a.key[p0 - 1] : -1, after = p1 < a.N ? a.key[p1] : -1;
        double acc[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
        int32_t cur = a.key[p0];
        bool first = true;  // the stretch began at p0
        auto flush = [&](bool last) {
            if (cur >= a.V) return;
            const bool from = first && cur == before, on = last && cur == after;
            if (from || on) {
                double* d = a.part + (run * 2 + (from ? 0 : 1)) * a.C + q * VEC;
#pragma unroll
                for (int j = 0; j < VEC; ++j) d[j] = acc[j];
            } else {
                float v[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] = (float)(acc[j] * (double)a.scale);
                store_vec<T, VEC>(gtab + (int64_t)cur * a.C + q * VEC, v);
            }
        };
        for (int64_t p = p0; p < p1; p += kBatch) {
            int32_t k[kBatch];
            float v[kBatch][VEC];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const bool in = p + u < p1;
                k[u] = in ? a.key[p + u] : a.V;
                if (in && k[u] < a.V) {
                    load_vec<T, VEC>(v[u], grad + (int64_t)a.val[p + u] * a.ld + q * VEC);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) v[u][j] = 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (p + u >= p1) continue;
                if (k[u] != cur) {
                    flush(false);
                    cur = k[u];
                    first = false;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[j] += (double)v[u][j];
            }
        }
        flush(true);
    }
}

// first position after `from` whose id differs from k (ids sorted, key[from] == k)
__device__ __forceinline__ int64_t stretch_end(const SumArgs& a, int64_t from, int32_t k)
{
    int64_t lo = from + 1, hi = a.N;
    while (lo < hi) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (a.key[mid] == k) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Block (run, slice): if a stretch begins in this run and goes on after it, its
// partial sums from here to its end.
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_embed_join(SumArgs a, T* __restrict__ gtab)
{
    __shared__ double s[kThreads * VEC];
    for (int64_t run = blockIdx.x; run + 1 < a.runs; run += gridDim.x) {  // conditions are the same for the whole block
        const int64_t p0 = run * a.R, p1 = p0 + a.R;
        const int32_t k = a.key[p1 - 1];
        if (k >= a.V || a.key[p1] != k) continue;
        if (a.key[p0] == k && p0 > 0 && a.key[p0 - 1] == k) continue;
        const int64_t last = (stretch_end(a, p1, k) - 1) / a.R;
        const int32_t rl = (int32_t)threadIdx.x / a.L, RL = kThreads / a.L;
        const int64_t q = (int64_t)blockIdx.y * a.L + ((int32_t)threadIdx.x - rl * a.L);
        const bool ok = rl < RL && q < a.CV;
        double acc[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = 0.0;
        if (ok) {
#pragma unroll 4
            for (int64_t r = run + rl; r <= last; r += RL) {
                const double* d = a.part + (r * 2 + (r == run ? 1 : 0)) * a.C + q * VEC;
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[j] += d[j];
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[threadIdx.x * VEC + j] = acc[j];
        __syncthreads();
        if (ok && rl == 0) {
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                double t = 0.0;
                for (int32_t r = 0; r < RL; ++r) t += s[(r * a.L + (int32_t)threadIdx.x) * VEC + j];
                v[j] = (float)(t * (double)a.scale);
            }
            store_vec<T, VEC>(gtab + (int64_t)k * a.C + q * VEC, v);
        }
        __syncthreads();
    }
}

// p[0 .. bytes) = 0; p aligned to 16 bytes or bytes counted one element at a time
__global__ void __launch_bounds__(kThreads) k_clear(int64_t n16, uint4* __restrict__ p, int64_t tail,
                                                    uint16_t* __restrict__ t)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
    for (int64_t k = i; k < n16; k += step) p[k] = uint4{0, 0, 0, 0};
    for (int64_t k = i; k < tail; k += step) t[k] = 0;
}

struct EmbedLayout {
    int64_t R, runs, tiles;
    size_t key[2], val[2], hist, total, part, bytes;
};

// Lanes per row of the wide form.
inline int64_t row_accesses(const EmbedShape& e, bool wide)
{
    return wide ? e.C / (16 / dtype_size(e.dtype)) : e.C;
}

EmbedLayout embed_layout(const EmbedShape& e)
{
    EmbedLayout w{};
    // Runs short enough to fill the chip (about 2^18 lanes), at least 16 rows
    // so that partial sums stay a small share of the traffic.
    const int64_t cv = row_accesses(e, e.C % (16 / dtype_size(e.dtype)) == 0);
    int64_t R = cdiv64(e.N * cv, 1 << 18);
    R = cdiv64(R < 16 ? 16 : R > 256 ? 256 : R, kBatch) * kBatch;
    w.R = R;
    w.runs = cdiv64(e.N, R);
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
    w.hist = take(4 * kDigit * w.tiles);
    w.total = take(4 * kDigit);
    w.part = take((int64_t)sizeof(double) * 2 * w.runs * e.C);
    w.bytes = o;
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
    a.L = (int32_t)(a.CV < kThreads ? a.CV : kThreads);
    a.R = (int32_t)w.R;
    a.scale = e.scale;
    a.key = key;
    a.val = val;
    a.part = part;
    const int32_t RL = kThreads / a.L;
    const unsigned slices = (unsigned)cdiv64(a.CV, a.L);
    hipLaunchKernelGGL((k_embed_sum<T, VEC>), dim3(grid_of(cdiv64(w.runs, RL)), slices), dim3(kThreads), 0, s, a,
                       (const T*)grad, (T*)gtab);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || w.runs < 2) return err;
    hipLaunchKernelGGL((k_embed_join<T, VEC>), dim3(grid_of(w.runs - 1), slices), dim3(kThreads), 0, s, a,
                       (T*)gtab);
    return hipGetLastError();
}

}  // namespace

size_t embed_bwd_workspace_bytes(const EmbedShape& e) { return embed_layout(e).bytes; }

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
    const int64_t es = dtype_size(e.dtype), bytes = e.V * e.C * es;
    hipError_t err = hipSuccess;
    {
        const bool a16 = ((uintptr_t)gtab & 15u) == 0;
        const int64_t n16 = a16 ? bytes / 16 : 0, tail = (bytes - 16 * n16) / 2;
        const int64_t blocks = cdiv64(n16 > tail ? n16 : tail, kThreads * 4);
        hipLaunchKernelGGL(k_clear, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(kThreads), 0, s, n16,
                           (uint4*)gtab, tail, (uint16_t*)((char*)gtab + 16 * n16));
        err = hipGetLastError();
        if (err != hipSuccess || e.N == 0) return err;
    }
    const EmbedLayout w = embed_layout(e);
    char* base = (char*)ws;
    int bits = 0;
    while ((e.V >> bits) != 0) ++bits;  // keys are 0 .. V
    SortArgs a{};
    a.N = e.N;
    a.V = (int32_t)e.V;
    a.tiles = (int32_t)w.tiles;
    a.hist = (int32_t*)(base + w.hist);
    a.total = (int32_t*)(base + w.total);
    int to = 0;
    for (int shift = 0; shift < bits; shift += 8) {
        a.shift = shift;
        a.ids = shift == 0 ? ids : nullptr;
        a.key = (const int32_t*)(base + w.key[to ^ 1]);
        a.val = (const int32_t*)(base + w.val[to ^ 1]);
        a.okey = (int32_t*)(base + w.key[to]);
        a.oval = (int32_t*)(base + w.val[to]);
        hipLaunchKernelGGL(k_sort_hist, dim3((unsigned)w.tiles), dim3(kThreads), 0, s, a);
        hipLaunchKernelGGL(k_sort_scan, dim3(kDigit), dim3(kThreads), 0, s, a);
        hipLaunchKernelGGL(k_sort_scatter, dim3((unsigned)w.tiles), dim3(kThreads), 0, s, a);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
        to ^= 1;
    }
    const int32_t* key = (const int32_t*)(base + w.key[to ^ 1]);
    const int32_t* val = (const int32_t*)(base + w.val[to ^ 1]);
    double* part = (double*)(base + w.part);
    const bool wide = e.C * es % 16 == 0 && aligned_rows(grad, e.ld, es) && aligned_rows(gtab, e.C, es);
    if (e.dtype == kF32)
        return wide ? embed_sum<float, kWide<float>>(e, w, key, val, grad, gtab, part, s)
                    : embed_sum<float, 1>(e, w, key, val, grad, gtab, part, s);
    return wide ? embed_sum<bf16_t, kWide<bf16_t>>(e, w, key, val, grad, gtab, part, s)
                : embed_sum<bf16_t, 1>(e, w, key, val, grad, gtab, part, s);
}

}  // namespace cgtp
