// cgtp_linear_wide.h -- launchers of the forms of the product beside the tiles of
// cgtp_linear.hip: planes (cgtp_linear_wide.hip), few rows (cgtp_linear_few.hip),
// rows that registers hold (cgtp_linear_rows.hip), narrow gradients (cgtp_linear_back.hip).
#pragma once

#include "cgtp_linear.h"

namespace cgtp {

struct WideArgs {
    GemmArgs g;              // shapes, tiles and parts (whole steps long), epilogue; rows, cols multiples of 8
    const uint16_t *P, *Q;   // planes of the rows' and the columns' operand, their rows on 16 bytes
    int64_t ldp, ldq;        // below 2^22
    int64_t planeP, planeQ;  // halves from one plane to the next
    int32_t side;            // of a tile: 256 or 128
};

// out [planes][rows][cols] of rows x (fp32: three planes), or of dz = mask x act'(Z) with its
// columns' sums to g.db_part [runs][cols] where g.db is set
struct PlaneArgs {
    GemmArgs g;      // Z, ldz, act, drop, db, db_part
    const void* x;
    int64_t ld, rows, cols;
    int64_t run;     // rows of a block
    uint16_t* out;   // or nullptr: the sums alone
};

hipError_t launch_linear_wide(int dtype, int kind, const WideArgs& w, hipStream_t s);
// y of few rows (A: x, B: W); vec: every array begins on 16 bytes and all rows are multiples of eight long
hipError_t launch_linear_few(int dtype, bool vec, const GemmArgs& a, hipStream_t s);
// y of rows of up to 128 inputs (A: x, B: W); vec as above
hipError_t launch_linear_rows(int dtype, bool vec, GemmArgs a, hipStream_t s);
// the gradients of up to 128 outputs in one pass (cgtp_linear_back.hip): tr slabs of W, kt x mt
// each, splits blocks to a slab
struct BackPlan {
    int kt, mt, rows;  // rows: of a chunk
    int64_t tr, splits;
};
BackPlan back_plan(int64_t n, int64_t k, int64_t m);
// A: x, B: g, rows: inputs, cols: outputs, depth: rows, want: dW; leaves parts of dW and db, and dx
hipError_t launch_linear_back(int dtype, bool vec, const GemmArgs& a, const BackPlan& p, const void* W, void* dx,
                              int64_t ldd, hipStream_t s);
// dx of up to 128 inputs, up to 64 for fp32 without Z alone (g: A, Z, rows, cols, depth and epilogue as for
// kDx; Q: planes of W)
hipError_t launch_linear_dx(int dtype, const WideArgs& w, hipStream_t s);
// parts of dW and db, fp32, up to 64 inputs, dz = g (A: x, B: g; tc: stretches of 128 outputs; run: rows
// of a part, a multiple of 64)
hipError_t launch_linear_dw(const GemmArgs& a, hipStream_t s);
hipError_t launch_linear_planes(int dtype, bool dz, const PlaneArgs& p, hipStream_t s);

}  // namespace cgtp
