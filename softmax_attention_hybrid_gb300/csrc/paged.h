// Shared declarations of the paged attention kernels (paged_tc.cu, paged_simt.cu; over
// 8-bit caches paged_q8_tc.cu, paged_q8_rows.cu, paged_q8_simt.cu), their host entry points and
// the joining kernel (paged_api.cu).
//
// One call answers T new tokens of each of B sequences. Query row (b, h, t), t below
// the sequence's number n of new tokens, stands at position i = P + ctx[b] + t (P: the
// length of the shared prefix, 0 without one) and sees the keys j <= i; an ordinary
// head with a window of w keys and s sinks sees those with i - j < w or j < s. The
// first P keys sit in the prefix's pages, which all sequences share; key P + x is slot x
// of the sequence's own pages.
//
// The keys are split over work items so that few rows still fill the GPU. Part 0 of a
// call is the prefix: an item takes a block of rows of one key/value head out of all
// sequences, so that each of the prefix's keys is read once per row block and not once
// per sequence. Part 1 is each sequence's own keys. An item writes its rows' unnormalised
// output, running maximum m and sum l (base 2), and join_kernel adds the items of a row:
//     O = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c,   M = max_c m_c.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "saf_internal.h"

namespace saf {

struct PagedArgs {
    const void* q;                 // [B, H, T, d]
    const void* k_cache;           // [num_pages, Hkv, page, d]
    const void* v_cache;
    const float* k_scale;          // 8-bit caches (codes of e4m3): a scale per row [num_pages, Hkv, page]; else NULL
    const float* v_scale;
    const int32_t* prefix_pages;   // [ceil(P / page)]
    const int32_t* page_table;     // [B, max_pages]
    const int32_t* ctx;            // [B]
    const int32_t* n_new;          // [B] or NULL: T each
    const float* a;                // [H, ld]
    const float* r;
    void* o;                       // [B, H, T, d]
    float* lse;                    // [B, H, T]
    float2* ml;                    // workspace: (m, l) of row, item: [B H T, nsplit]
    float* po;                     // workspace: unnormalised rows of items: [B H T, nsplit, d]
    uint32_t* status;
    int B, H, Hkv, G, T, d, ld;
    int max_pages, num_pages, page_log2;
    int P, max_len, window, sinks;
    int tile[2];                   // keys per tile of the kernel that runs: part 0, part 1
    int rows[2];                   // rows per block of the kernel that runs: part 0, part 1
    int nrb[2];                    // row blocks of part 0 and part 1
    int head_blocks[2];            // row blocks of each head, 0: blocks run on from head to head
    int chunks[2];                 // items along the keys: part 0, part 1
    int per_chunk[2];              // tiles of an item
    int nsplit;                    // chunks[0] + chunks[1]
    unsigned items0, items;        // items of part 0, of both parts
    float scale_log2;              // log2(e) / sqrt(d)
    HeadMask mask;
    uint8_t gheads[SAF_MAX_HEADS]; // query heads of key/value head hk at [hk G, hk G + G), ordinary first
    uint16_t gord[SAF_MAX_HEADS];  // ordinary query heads of key/value head hk (up to 256)
};

struct PagedItem {
    int part, hk, b, rb, chunk;    // b: the sequence of a part-1 item
};

// Items are numbered part 0 first (its items carry the most rows), and in a part the
// chunks of one (sequence, key/value head, row block) next to each other.
__device__ __forceinline__ PagedItem paged_item(const PagedArgs& p, unsigned idx) {
    PagedItem it;
    it.part = idx >= p.items0;
    if (it.part) idx -= p.items0;
    const unsigned C = (unsigned)p.chunks[it.part], nrb = (unsigned)p.nrb[it.part];
    unsigned u = idx / C;
    it.chunk = (int)(idx - u * C);
    const unsigned v = u / nrb;
    it.rb = (int)(u - v * nrb);
    it.b = (int)(v / (unsigned)p.Hkv);       // 0 in part 0
    it.hk = (int)(v - (unsigned)it.b * (unsigned)p.Hkv);
    return it;
}

// New tokens of sequence b, cut to [0, T] and to the room of max_len slots; a sequence
// whose ctx is negative has none.
__device__ __forceinline__ int paged_tokens(const PagedArgs& p, int b, int* ctx, bool* bad) {
    const int c = p.ctx[b];
    int n = p.n_new ? p.n_new[b] : p.T;
    *bad = c < 0 || n < 0 || n > p.T || (n > 0 && c > p.max_len - n);
    n = n < 0 ? 0 : n > p.T ? p.T : n;
    if (c < 0 || c >= p.max_len) n = 0;
    else if (n > p.max_len - c) n = p.max_len - c;
    *ctx = c;
    return n;
}

struct PagedRow {
    int h, b, t;
    int gi;       // member of the group
    int i;        // position, -1: the row is not there or sees nothing
    bool there;   // the row is one of the output's
    bool frozen;
};

// The rows of an item's block: rows first .. first + there - 1 of one (sequence,) key/value
// head's, in which the group's ordinary heads come first, and in a head the sequences (part 0)
// and tokens in order. Blocks run on from head to head, except where a head fills several:
// a block's positions then lie close together, and a window leaves it few keys.
struct PagedBlock {
    int first, there, per_head;
};
__device__ __forceinline__ PagedBlock paged_block(const PagedArgs& p, const PagedItem& it) {
    PagedBlock k;
    const int rows = p.rows[it.part], hb = p.head_blocks[it.part];
    k.per_head = it.part ? p.T : p.B * p.T;
    if (hb) {
        const int gi = it.rb / hb, at = (it.rb - gi * hb) * rows;
        k.first = gi * k.per_head + at;
        k.there = k.per_head - at < rows ? k.per_head - at : rows;
    } else {
        k.first = it.rb * rows;
        k.there = p.G * k.per_head - k.first < rows ? p.G * k.per_head - k.first : rows;
    }
    return k;
}

// Row x of the block, its position left out.
__device__ __forceinline__ PagedRow paged_place(const PagedArgs& p, const PagedItem& it, const PagedBlock& k, int x) {
    PagedRow w;
    w.there = x < k.there;
    w.h = w.b = w.t = w.gi = 0;
    w.i = -1;
    w.frozen = false;
    if (!w.there) return w;
    w.gi = (k.first + x) / k.per_head;
    const int rem = k.first + x - w.gi * k.per_head;
    w.b = it.part ? it.b : rem / p.T;
    w.t = it.part ? rem : rem - w.b * p.T;
    w.h = p.gheads[it.hk * p.G + w.gi];
    w.frozen = w.gi >= p.gord[it.hk];
    return w;
}

// Row x of the block.
__device__ __forceinline__ PagedRow paged_row(const PagedArgs& p, const PagedItem& it, const PagedBlock& k, int x) {
    PagedRow w = paged_place(p, it, k, x);
    if (!w.there) return w;
    int c;
    bool bad;
    const int n = paged_tokens(p, w.b, &c, &bad);
    if (w.t < n) w.i = p.P + c + w.t;
    return w;
}

// The keys of an item's part that its rows see, in slots x of the part (key j = x in part
// 0, j = P + x in part 1): x < hi and (x >= lo or x < sink). They lie in tiles
// [0, n_sink) and [t_lo, t_lo + n - n_sink).
struct PagedRange {
    int hi, lo, sink;
    int n_sink, t_lo, n;
};

// imin, imax: the smallest and largest position among the item's rows that see anything
// (imax = -1: none); full: a frozen head is among them, or there is no window.
__device__ __forceinline__ PagedRange paged_range(const PagedArgs& p, const PagedItem& it, int imin, int imax,
                                                  bool full) {
    PagedRange g;
    const int tile = p.tile[it.part];
    const int off = it.part ? p.P : 0;
    g.hi = imax < 0 ? 0 : it.part ? imax + 1 - off : (imax + 1 < p.P ? imax + 1 : p.P);
    g.lo = g.sink = g.n_sink = g.t_lo = 0;
    if (!full && g.hi > 0) {
        const int lo = imin - p.window + 1 - off;
        g.lo = lo > 0 ? lo : 0;
        const int sink = p.sinks - off;
        g.sink = sink < 0 ? 0 : sink < g.hi ? sink : g.hi;
    }
    const int t_hi = (g.hi + tile - 1) / tile;
    g.t_lo = g.lo < g.hi ? g.lo / tile : t_hi;
    g.n_sink = (g.sink + tile - 1) / tile;
    if (g.n_sink > g.t_lo) g.n_sink = g.t_lo;
    g.n = g.n_sink + t_hi - g.t_lo;
    return g;
}

__device__ __forceinline__ int paged_tile(const PagedRange& g, int e) { return e < g.n_sink ? e : g.t_lo + e - g.n_sink; }

// Page of slot x of the item's part; -1 where the table has none inside the cache.
__device__ __forceinline__ int paged_page(const PagedArgs& p, const PagedItem& it, int x) {
    const int at = x >> p.page_log2;
    const int pg = it.part ? p.page_table[(size_t)it.b * p.max_pages + at] : p.prefix_pages[at];
    return pg >= 0 && pg < p.num_pages ? pg : -1;
}

__device__ __forceinline__ size_t paged_out_row(const PagedArgs& p, const PagedRow& w) {
    return ((size_t)w.b * p.H + w.h) * p.T + w.t;
}

// paged_tc.cu: bf16, tensor cores; rows 32, 64 or 128 per block, and tiles of paged_tc_tile(d, rows)
// keys. paged_simt.cu: fp32, CUDA cores; rows kSimtRows, tiles kSimtTile.
__host__ __device__ constexpr int paged_tc_tile(int d, int rows) { return d == 64 && rows < 128 ? 128 : 64; }
cudaError_t launch_paged_tc(const PagedArgs& p, cudaStream_t s);
constexpr int kSimtRows = 8, kSimtTile = 32;
cudaError_t launch_paged_simt(const PagedArgs& p, cudaStream_t s);
// 8-bit caches, fp32 q and o, CUDA cores (paged_q8_simt.cu): blocks of 2, 4, 6 or 8 rows, tiles kQ8SimtTile.
constexpr int kQ8SimtTile = 128;
__host__ __device__ constexpr int paged_q8_simt_ctas(int d) { return d == 64 ? 4 : d == 96 ? 3 : 2; }   // of an SM
cudaError_t launch_paged_q8_simt(const PagedArgs& p, cudaStream_t s);
// 8-bit caches, bf16 q and o, tensor cores. paged_q8_tc.cu: blocks of 4, 8, 16, 24 or 32 rows, tiles kQ8Tile;
// paged_q8_rows.cu: blocks of 256 rows, tiles kQ8RowsTile. `items` of p's, the first ones.
constexpr int kQ8Tile = 128, kQ8RowsTile = 128, kQ8Rows = 256;
cudaError_t launch_paged_q8(const PagedArgs& p, int rows, unsigned items, cudaStream_t s);
cudaError_t launch_paged_q8_rows(const PagedArgs& p, unsigned items, cudaStream_t s);

}  // namespace saf
