// cgtp_drop.h -- the dropout mask from a counter-based generator (device code).
//
// Whether element (n, c) of [N][C] rows is kept is a function of the seed, the
// offset, n and c alone, so a mask is formed again wherever it is needed and never
// stored.  Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011) at the counter (c / 8, n, offset low, offset high) and the
// key (seed low, seed high) gives 128 bits: eight fields of 16 bits, from the lowest,
// for the channels 8 (c / 8) .. + 7; an element is kept where its field is at least
// thr = 65536 p, rounded.  Sixteen bits to an element, and not 32, halve what is
// the kernels' largest cost beside memory: the generator's 20 wide products.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "cgtp_train_internal.h"

namespace cgtp {

struct Drawn {
    uint32_t w[4];
    // field j, 0 .. 7
    __device__ __forceinline__ uint32_t operator[](int j) const { return j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu; }
};

__device__ __forceinline__ Drawn philox(uint32_t block, uint32_t row, uint64_t offset, uint64_t seed)
{
    uint32_t a = block, b = row, c = (uint32_t)offset, d = (uint32_t)(offset >> 32);
    uint32_t k = (uint32_t)seed, l = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(q >> 32) ^ b ^ k;
        b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ d ^ l;
        d = (uint32_t)p;
        k += 0x9E3779B9u;
        l += 0xBB67AE85u;
    }
    return Drawn{{a, b, c, d}};
}

// the offset of a launch: the caller's and, where there is one, the device's step
__device__ __forceinline__ uint64_t drop_offset(const Drop& d)
{
    return d.offset + (d.step ? (uint64_t)*d.step : 0);
}

}  // namespace cgtp
