// What the two kernels over 8-bit caches share (paged_q8_tc.cu, paged_q8_rows.cu).
#pragma once

#include "paged_tc.cuh"

namespace saf {
namespace paged_q8 {

using namespace paged_tc;

struct Q8Params {
    CUtensorMap tm_k, tm_v;
    PagedArgs a;
    int box;   // keys of a TMA box: the page's, at most a tile's
};

struct Work {
    PagedItem it;
    PagedRange g;
    int e0, e1;       // tiles
    int imin, imax;   // positions of the rows that see anything
    int off;          // position of the part's slot 0
    int there;        // rows of the block that are rows of the output
    int nf;           // rows of frozen heads: the block's last ones
    bool any_ord;     // an ordinary row is among them: K is loaded

    __device__ __forceinline__ int slot0(int j, int tile) const {   // first slot of the j-th tile, the newest first
        return paged_tile(g, e1 - 1 - j) * tile;
    }
    // place of its K and V in the order of loads
    __device__ __forceinline__ int k_load(int j) const { return j == 0 ? 0 : 2 * j - 1; }
    __device__ __forceinline__ int v_load(int j) const {
        if (!any_ord) return j;
        return j + 1 < e1 - e0 ? 2 * j + 2 : 2 * j + 1;
    }
};

__device__ __forceinline__ float pow2i(int e) {   // 2^e, -149 <= e <= 127
    return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}

// The loading warp. Lane l fetches box l of every tile, from its page, and the box's scales.
template <typename C, typename Shared>
__device__ __forceinline__ void load_warp(const Q8Params& P, const Work& w, uint8_t* sm, Shared& sh) {
    constexpr int kTile = C::tile;
    auto& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const PagedArgs& p = P.a;
    const int lane = threadIdx.x & 31;
    const int nbox = kTile / P.box, n = w.e1 - w.e0;
    const int in_page = (1 << p.page_log2) - 1;
    const uint32_t box_bytes = (uint32_t)P.box * (128u + 4u);
    // The pages of a batch of tiles are looked up together, lane l those of tile l / nbox, box
    // l mod nbox, a batch ahead of their use: a lookup for each tile would wait for the memory
    // in every one.
    const int batch = 32 / nbox;
    auto look = [&](int first) -> int {   // a page, -1: one that is not in the cache, -2: nothing to fetch
        const int j = first + lane / nbox;
        if (j >= n) return -2;
        const int bx = w.slot0(j, kTile) + (lane & (nbox - 1)) * P.box;
        return box_seen(w.g, bx, P.box) ? paged_page(p, w.it, bx) : -2;
    };
    int looked = look(0), ahead = look(batch);   // tiles [base, base + batch), and the batch behind
    int base = 0;
    if (lane == 0) {
        tma_prefetch_desc(&P.tm_k);
        tma_prefetch_desc(&P.tm_v);
    }
    auto page_of = [&](int j) -> int {   // my box's page of tile j (ascending), -1: nothing to fetch
        if (j == base + batch) {
            base = j;
            looked = ahead;
            ahead = look(base + batch);
        }
        const int pg = __shfl_sync(0xffffffffu, looked, ((j - base) * nbox + lane) & 31);
        if (lane >= nbox) return -1;
        if (pg == -1) {
            *(volatile int*)&sh.lost = 1;
            atomicOr(p.status, kStatusPage);
        }
        return pg;
    };
    int last = -1;   // the last load that was begun
    auto fetch = [&](int load, const CUtensorMap* map, const float* scales, int j, int pg) -> bool {
        const int s = load % C::slots;
        if (!wait_all(&bars.empty[s], ((load / C::slots) & 1) ^ 1u, abort, p.status)) return false;
        const uint32_t have = __ballot_sync(0xffffffffu, pg >= 0);
        if (lane == 0) mbar_expect_tx(&bars.full[s], __popc(have) * box_bytes);
        last = load;
        __syncwarp();
        if (pg >= 0) {
            const int in = (w.slot0(j, kTile) + lane * P.box) & in_page;
            const int z = pg * p.Hkv + w.it.hk;
            tma_load_3d(sm + C::ring + s * (kTile * 128) + lane * P.box * 128, map, &bars.full[s], 0, in, z);
            bulk_load(sm + C::scales + s * (kTile * 4) + lane * P.box * 4, scales + ((size_t)z << p.page_log2) + in,
                      (uint32_t)P.box * 4u, &bars.full[s]);
        }
        __syncwarp();
        return true;
    };
    int pg = page_of(0);
    bool ok = !w.any_ord || fetch(0, &P.tm_k, p.k_scale, 0, pg);
    for (int j = 0; j < n && ok; ++j) {
        const int next = j + 1 < n ? page_of(j + 1) : -1;
        if (w.any_ord && j + 1 < n) ok = fetch(w.k_load(j + 1), &P.tm_k, p.k_scale, j + 1, next);
        ok = ok && fetch(w.v_load(j), &P.tm_v, p.v_scale, j, pg);
        pg = next;
    }
    // no copy is on its way when the warp leaves (after a wait that ran out, nobody may have waited for the last ones)
    if (lane == 0)
        for (int load = last < C::slots ? 0 : last - C::slots + 1; load <= last; ++load)
            mbar_wait_bounded(&bars.full[load % C::slots], (load / C::slots) & 1, kWaitLimitNs);
    __syncwarp();
}

// What a launch passes on: the tensor maps of the caches, read in boxes of at most `tile` keys.
inline bool q8_params(Q8Params* P, const PagedArgs& a, int tile) {
    P->a = a;
    const int page = 1 << a.page_log2;
    P->box = page < tile ? page : tile;
    const uint64_t slices = (uint64_t)a.num_pages * a.Hkv;
    const void* k = a.k_cache ? a.k_cache : a.v_cache;   // (no K is loaded when every head is frozen)
    return make_tmap_u8_3d(&P->tm_k, k, a.d, page, slices, 128, P->box) &&
           make_tmap_u8_3d(&P->tm_v, a.v_cache, a.d, page, slices, 128, P->box);
}

}  // namespace paged_q8
}  // namespace saf
