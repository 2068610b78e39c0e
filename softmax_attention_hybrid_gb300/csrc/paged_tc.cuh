// What the tensor-core kernels of paged attention share (paged_tc.cu, paged_q8_tc.cu, paged_q8_rows.cu;
// paged_q8_simt.cu takes its addresses of shared memory).
#pragma once

#include "paged.h"
#include "tc_common.cuh"

namespace saf {
namespace paged_tc {

using namespace tc;

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A wait of a converged warp: every lane waits and the warp goes on, or gives up, together.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, kStatusTimeout));
}

// Whether keys [bx, bx + box) of the part hold one that some row sees.
__device__ __forceinline__ bool box_seen(const PagedRange& g, int bx, int box) {
    return bx < g.hi && (bx + box > g.lo || bx < g.sink);
}

// An item without keys: its rows' empty sums (out_row [rows]: the rows' places in o, -1: none), by `threads` threads.
__device__ __forceinline__ void write_empty(const PagedArgs& p, const PagedItem& it, int rows, const int* out_row,
                                            int threads) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int split = it.part ? p.chunks[0] + it.chunk : it.chunk;
    if (p.nsplit > 1) {
        for (int x = t; x < rows; x += threads)
            if (out_row[x] >= 0) p.ml[(size_t)out_row[x] * p.nsplit + split] = make_float2(-INFINITY, 0.f);
    } else {
        for (int x = warp; x < rows; x += threads / 32) {
            if (out_row[x] < 0) continue;
            const size_t at = (size_t)out_row[x];
            for (int c = 2 * lane; c < p.d; c += 64) *reinterpret_cast<uint32_t*>((__nv_bfloat16*)p.o + at * p.d + c) = 0u;
            if (lane == 0) p.lse[at] = -INFINITY;
        }
    }
}

}  // namespace paged_tc
}  // namespace saf
