// Paged attention on the 5th-generation tensor cores (bf16; see paged.h for the split).
//
// An item holds up to 128 query rows, the M = 128 rows of its MMAs, and walks its tiles of 64 or
// 128 keys: S = Q K^T, online softmax with one thread per row, O += P V. Keys and values come
// page by page through TMA, straight into the swizzled operand layout.
//
// Copies. A decoding step has far fewer rows than 128 (the query heads of a group times the new
// tokens), and one thread per row would leave most threads idle in the softmax, the longest
// part of a tile. With at most 64 (32) rows the tile therefore holds 2 (4) copies of each
// row, and copy c takes the tile's keys [c 64 / copies, ...) only, with zero weights for the
// others: the softmax of a row runs on 2 (4) threads, the MMAs cost the same, and the
// copies' (m, l, O) are added at the end like items.
//
// Warps (256 threads, two CTAs per SM): 0-3 rows, one thread per row of the tile (TMEM lane);
// 4 loads K and V (each of its lanes fetches one page of the tile); 5 owns tensor memory and
// issues S, 6 issues P V (two issuers, since a tile's waits, MMAs and commits take one about
// 1600 cycles at d = 64, longer than the softmax of a tile: a wait costs about 100, and a
// commit as much); 7 brings the frozen heads' a and r of the next tile into shared memory.
// Tensor memory (256 columns): S | P (bf16 pairs) | O. S has columns of its own so that the
// next tile's S runs under this one's softmax.
// Shared memory: Q, the frozen heads' patterns, and a ring of slots of one tile of K or V each,
// filled in the order in which the MMAs use them: K0, K1, V0, K2, V1, ... (V0, V1, ... where no
// row is ordinary).
//
// Tiles are 64 keys, and 128 at d = 64 with at most 64 rows: what a tile costs in waits and
// latencies is about the same for both, and 32 KB of K and V per tile pay for it where 16 KB
// do not. (128 rows at d = 64 keep 64: a thread cannot hold 128 scores.)
//
// Bound by memory in decoding: a tile of K and V is 32 KB at d = 128, 1400 cycles of an SM's share
// of the memory, against 512 cycles of MMAs.
#include <string.h>

#include <atomic>

#include "paged_tc.cuh"

namespace saf {
namespace {

using namespace paged_tc;

constexpr int kThreads = 256;
// Register split (setmaxnreg): warps 4-7 drop to kRegsOther, the row warps rise to kRegsRows, within
// the kRegsLaunch per thread that the launch hands out (checked on the host).
constexpr int kRegsLaunch = 128, kRegsRows = 184, kRegsOther = 72;
static_assert(kRegsRows + kRegsOther <= 2 * kRegsLaunch, "register split too large");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // lazy rescale: factor 256
constexpr int kPatFloats = 1792;   // room for the frozen heads' patterns of a tile (7 KB, two tiles)

struct TcParams {
    CUtensorMap tm_k, tm_v;
    PagedArgs a;
    int box;   // keys of a TMA box: min(page, 64)
};

// kD: head dimension as the tiles hold it (64, or 128 for 96 and 128: TMA fills the columns
// past the row's end with zeros). TK: keys of a tile.
template <int kD, int TK>
struct Smem {
    static constexpr int atom = TK * 128;               // TK keys x 64 columns
    static constexpr int tile = atom * (kD / 64);
    static constexpr int q_atom = 128 * 128;
    static constexpr int q = 0;
    static constexpr int ring = q + q_atom * (kD / 64);
    static constexpr int ring_bytes = kD == 64 ? 80 * 1024 : 64 * 1024;   // what two CTAs of an SM leave
    static constexpr int slots = ring_bytes / tile;
    static constexpr int pat = ring + ring_bytes;
    static constexpr int total = pat + 2 * kPatFloats * 4;
    // after the last MMA Q and the ring stage the output rows
    static constexpr int out_pitch = kD + 4;
    static_assert(128 * out_pitch * 4 <= pat, "output staging");
    // tensor-memory columns (S at 0)
    static constexpr uint32_t col_p = TK, col_o = TK == 64 ? 128 : 192;
    static_assert(col_p + TK / 2 <= col_o && col_o + kD <= 256, "tensor memory");
};
constexpr int kMaxSlots = 10;

struct Bars {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t s_full, s_empty, p_ready, o_done, pat_full[2], pat_empty[2], mma_idle[2];
};

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t* r) {
    if constexpr (N == 64) {
        tmem_ld32(addr, r);
        tmem_ld32(addr + 32, r + 32);
    } else if constexpr (N == 32) {
        tmem_ld32(addr, r);
    } else {
        tmem_ld16(addr, r);
    }
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t addr, const uint32_t* r) {
    if constexpr (N == 32) tmem_st32(addr, r);
    else if constexpr (N == 16) tmem_st16(addr, r);
    else tmem_st8(addr, r);
}

// What every thread of the CTA knows about its item.
struct Work {
    PagedItem it;
    PagedRange g;
    int e0, e1;       // tiles
    int imin, imax;   // positions of the rows that see anything
    int off;          // position of the part's slot 0
    int there;        // rows of the block that are rows of the output
    bool any_ord;     // an ordinary row is among them: K is loaded
    // the frozen heads of the block: group members f0 .. f0 + nf - 1, whose patterns the tile's
    // threads read from shared memory (staged) or from a and r themselves
    int f0, nf;
    bool staged;

    // place of tile e0 + j's K and V in the order of loads
    __device__ __forceinline__ int k_load(int j) const { return j == 0 ? 0 : 2 * j - 1; }
    __device__ __forceinline__ int v_load(int j) const {
        if (!any_ord) return j;
        return j + 1 < e1 - e0 ? 2 * j + 2 : 2 * j + 1;
    }
    // floats of one staged pattern: a of the tile's TK keys, and r of the distances imin - (last
    // key) .. imax - (first key), rounded up to whole 16 bytes
    __device__ __forceinline__ int pitch(int TK) const { return (2 * TK + (imax - imin) + 3) & ~3; }
};

// The loading warp. Lane l fetches box l of every tile, from its page.
template <int kD, int TK>
__device__ __forceinline__ void load_warp(const TcParams& P, const Work& w, uint8_t* sm, Bars& bars,
                                          volatile int* abort) {
    using S = Smem<kD, TK>;
    const PagedArgs& p = P.a;
    const int lane = threadIdx.x & 31;
    const int nbox = TK / P.box, n = w.e1 - w.e0;
    const int in_page = (1 << p.page_log2) - 1;
    const uint32_t box_bytes = (uint32_t)P.box * 128u * (kD / 64);
    // The pages of a batch of tiles are looked up together, lane l those of tile l / nbox, box
    // l mod nbox, a batch ahead of their use: a lookup for each tile would wait for the memory
    // in every one.
    const int batch = 32 / nbox;
    auto look = [&](int first) -> int {   // a page as the table has it, -1: nothing to fetch
        const int j = first + lane / nbox;
        if (j >= n) return -1;
        const int bx = paged_tile(w.g, w.e0 + j) * TK + (lane & (nbox - 1)) * P.box;
        if (!box_seen(w.g, bx, P.box)) return -1;
        const int at = bx >> p.page_log2;
        return __ldg(w.it.part ? p.page_table + (size_t)w.it.b * p.max_pages + at : p.prefix_pages + at);
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
        return lane < nbox && pg >= 0 && pg < p.num_pages ? pg : -1;
    };
    auto fetch = [&](int load, const CUtensorMap* map, int j, int pg) -> bool {
        const int s = load % S::slots;
        if (!wait_all(&bars.empty[s], ((load / S::slots) & 1) ^ 1u, abort, p.status)) return false;
        const uint32_t have = __ballot_sync(0xffffffffu, pg >= 0);
        if (lane == 0) mbar_expect_tx(&bars.full[s], __popc(have) * box_bytes);
        __syncwarp();
        if (pg >= 0) {
            const int bx = paged_tile(w.g, w.e0 + j) * TK + lane * P.box;
            uint8_t* dst = sm + S::ring + s * S::tile + lane * P.box * 128;
            const int z = pg * p.Hkv + w.it.hk;
#pragma unroll
            for (int c = 0; c < kD / 64; ++c) tma_load_3d(dst + c * S::atom, map, &bars.full[s], 64 * c, bx & in_page, z);
        }
        __syncwarp();
        return true;
    };
    int pg = page_of(0);
    bool ok = !w.any_ord || fetch(0, &P.tm_k, 0, pg);
    for (int j = 0; j < n && ok; ++j) {
        const int next = j + 1 < n ? page_of(j + 1) : -1;
        if (w.any_ord && j + 1 < n) ok = fetch(w.k_load(j + 1), &P.tm_k, j + 1, next);
        ok = ok && fetch(w.v_load(j), &P.tm_v, j, pg);
        pg = next;
    }
}

// The pattern warp: a and r of the block's frozen heads for every tile. A row at position i and
// key x need a[x] and r[i - x]; for all rows of a head and TK keys that is a run of r of
// imax - imin + TK entries, read here in whole lines, where a thread per row would read 64
// scattered entries of its own. (64 sequences after a 32K prefix, a frozen head of four: the
// rows' own reads took 2500 to 3500 cycles of a tile, traced.)
template <int kD, int TK>
__device__ __forceinline__ void pattern_warp(const TcParams& P, const Work& w, uint8_t* sm, Bars& bars,
                                             volatile int* abort) {
    using S = Smem<kD, TK>;
    const PagedArgs& p = P.a;
    const int lane = threadIdx.x & 31;
    const int band = w.imax - w.imin + TK, pitch = w.pitch(TK);
    const uint32_t pat = smem_u32(sm + S::pat);
    auto copy = [&](uint32_t dst, const float* src) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
    };
    const int n = w.e1 - w.e0;
    for (int j = 0; j <= n; ++j) {
        if (j < n) {   // tile j's copies are on their way while the rows work on tile j - 1
            const int b = j & 1, x0 = paged_tile(w.g, w.e0 + j) * TK;
            if (!wait_all(&bars.pat_empty[b], ((j >> 1) & 1) ^ 1u, abort, p.status)) break;
            for (int f = 0; f < w.nf; ++f) {
                const size_t h = p.gheads[w.it.hk * p.G + w.f0 + f];
                const float* a = p.a + h * p.ld;
                const float* r = p.r + h * p.ld;
                const uint32_t out = pat + 4u * (uint32_t)(b * kPatFloats + f * pitch);
                // (entries of keys past a row's own position are masked: any will do)
#pragma unroll
                for (int c = lane; c < TK; c += 32) copy(out + 4 * c, a + min(w.off + x0 + c, p.ld - 1));
                const int first = w.imin - w.off - x0 - (TK - 1);
#pragma unroll 4
                for (int c = lane; c < band; c += 32) copy(out + 4 * (TK + c), r + min(max(first + c, 0), p.ld - 1));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (j > 0) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");   // tile j - 1's
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.pat_full[(j - 1) & 1]);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The rows' part of an item: kCopies copies of 128 / kCopies rows; thread t holds row t mod
// (128 / kCopies) and the keys [kCols copy, ...) of every tile.
template <int kD, int TK, int kCopies>
__device__ __forceinline__ void row_warps(const TcParams& P, const Work& w, const PagedRow& row, bool lost,
                                          uint8_t* sm, Bars& bars, const int* out_row, float* sh_m, float* sh_l,
                                          uint32_t tmem, volatile int* abort) {
    using S = Smem<kD, TK>;
    const PagedArgs& p = P.a;
    constexpr int kCols = TK / kCopies, kRows = 128 / kCopies;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int c0 = (t / kRows) * kCols;   // my keys of a tile
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const int box_log2 = __ffs(P.box) - 1;
    const int i = row.i < 0 ? -1 : row.i - w.off;   // my last visible slot of the part
    const float sc = row.frozen ? kLog2e : p.scale_log2;
    const bool frozen = row.frozen && i >= 0;
    const bool any_frozen = __any_sync(0xffffffffu, frozen);
    const float* ra = p.a + (size_t)row.h * p.ld + w.off;
    const float* rr = p.r + (size_t)row.h * p.ld;
    // my staged pattern: a of my keys, and r of my keys from the far end on (entry k - c for key c)
    const float* pat_a = reinterpret_cast<const float*>(sm + S::pat) + (frozen ? row.gi - w.f0 : 0) * w.pitch(TK) + c0;
    const float* pat_r = pat_a + TK - 2 * c0 + (TK - 1) + (frozen ? row.i - w.imin : 0);
    float m = -INFINITY, l = 0.f;
    float m_raw = 0.f;   // the score that m is, before the factor sc
    bool ok = true;

    if (kCopies > 1) {   // the other copies' keys: weights that stay zero
        uint32_t z[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) z[c] = 0u;
#pragma unroll
        for (int c = 0; c < TK / 2; c += 32) tmem_st32(lane_base + S::col_p + c, z);
        tmem_st_wait();
    }
    int n = 0;
    for (int e = w.e0; e < w.e1; ++e, ++n) {
        const int x0 = paged_tile(w.g, e) * TK;
        uint32_t sv[kCols];
        if (w.any_ord) {
            if (!(ok = mbar_wait(&bars.s_full, n & 1, abort, p.status, kStatusTimeout))) break;
            tc_fence_after();
            tmem_ld_n<kCols>(lane_base + c0, sv);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.s_empty);
        }
        if (any_frozen) {   // the fixed pattern's logits (Eq. 3)
            if (w.staged) {
                const int b = n & 1;
                if (!(ok = mbar_wait(&bars.pat_full[b], (n >> 1) & 1, abort, p.status, kStatusTimeout))) break;
                if (frozen) {
                    const float* qa = pat_a + b * kPatFloats;
                    const float* qr = pat_r + b * kPatFloats;
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) {
                        const float4 a4 = *reinterpret_cast<const float4*>(qa + c);
                        sv[c] = __float_as_uint(a4.x + qr[-c]);
                        sv[c + 1] = __float_as_uint(a4.y + qr[-c - 1]);
                        sv[c + 2] = __float_as_uint(a4.z + qr[-c - 2]);
                        sv[c + 3] = __float_as_uint(a4.w + qr[-c - 3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.pat_empty[b]);
            } else if (frozen) {   // (keys past my own position are masked below)
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const int y = min(x0 + c0 + c, i);
                    sv[c] = __float_as_uint(__ldg(ra + y) + __ldg(rr + i - y));
                }
            }
        }
        uint32_t have = 0xffffffffu;   // boxes whose page is in the cache
        if (lost)
            for (int b = 0; b < TK / P.box; ++b) {
                const int bx = x0 + b * P.box;
                if (box_seen(w.g, bx, P.box) && paged_page(p, w.it, bx) < 0) have &= ~(1u << b);
            }
        // masks, in tiles that some row does not see whole
        if (lost || x0 + TK > w.g.hi || x0 + TK - 1 > w.imin - w.off ||
            (p.window > 0 && x0 <= w.imax - w.off - p.window)) {
            const int lo = row.frozen || p.window == 0 ? -1 : i - p.window;   // slots <= lo: sinks only
            const int sink = p.sinks - w.off, last = min(i, w.g.hi - 1);   // (a prefix ends before i)
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int x = x0 + c0 + c;
                const bool seen = x <= last && (x > lo || x < sink) && ((have >> ((c0 + c) >> box_log2)) & 1u);
                if (!seen) sv[c] = __float_as_uint(-INFINITY);
            }
        }
        float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
            ma = fmax3(ma, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            mb = fmax3(mb, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
        }
        const float most = fmaxf(ma, mb), m_new = fmaxf(m, most * sc);
        const bool need = m_new > m + kRescaleThreshold;
        const float f = need ? fast_exp2(m - m_new) : 1.f;
        if (need) {
            l *= f;
            m = m_new;
            m_raw = most;
        }
        const float ref = m == -INFINITY ? 0.f : m;   // a row that has seen no key yet: weights 2^-inf = 0
        const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-ref, -ref);
        // sc s - m leaves the rounding of m, which is no longer small beside scores past 2^20: it is taken off. (64
        // sequences after 32K tokens: 116 us, 113 without, 117 with the maximum taken off before the factor in such rows.)
        const float slip = fabsf(ref) > 1048576.f ? -fmaf(m_raw, sc, -ref) : 0.f;
        const float2 slip2 = make_float2(slip, slip);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        // The weights are rounded to bf16 for P V (both operands of an MMA have V's type): o is off by up
        // to 2^-8 of sum_j P_j |v_j|. l adds them unrounded, which lse and the joins of items need.
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
            const float2 y = ffma2(make_float2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sc2, nm2);
            const float2 x = fadd2(y, slip2);
            const float2 ex = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            if (c & 1) acc1 = fadd2(acc1, ex);
            else acc0 = fadd2(acc0, ex);
            pk[c] = pack_bf16(ex.x, ex.y);
        }
        l += (acc0.x + acc1.x) + (acc0.y + acc1.y);
        // values of slots that no row sees may be anything: zeros, for 0 * NaN is none
        if (lost || x0 + TK > w.g.hi || (x0 < w.g.lo && x0 + TK > w.g.sink)) {
            const int ld = w.v_load(n), s = ld % S::slots;
            if (!(ok = mbar_wait(&bars.full[s], (ld / S::slots) & 1, abort, p.status, kStatusTimeout))) break;
            const int kk = t & (TK - 1), x = x0 + kk;
            const bool seen = x < w.g.hi && (x >= w.g.lo || x < w.g.sink) && ((have >> (kk >> box_log2)) & 1u);
            if (!seen) {   // 128 / TK threads share a key's row of kD / 64 times 128 bytes
                constexpr int kShare = 128 / TK, kBytes = 2 * kD / kShare;
                const int part = TK == 128 ? 0 : t >> 6;
                uint8_t* vrow = sm + S::ring + s * S::tile + kk * 128 +
                                (kBytes == 128 ? part * S::atom : part * kBytes);
                static_assert(kBytes == 128 || (kBytes == 64 && kD == 64), "a share lies in one atom");
#pragma unroll
                for (int c = 0; c < kBytes / 16; ++c) *reinterpret_cast<uint4*>(vrow + 16 * c) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
        }
        if (n > 0) {   // P V of the previous tile is done: P is free, O is stable
            if (!(ok = mbar_wait(&bars.o_done, (n - 1) & 1, abort, p.status, kStatusTimeout))) break;
            tc_fence_after();
        }
        tmem_st_n<kCols / 2>(lane_base + S::col_p + c0 / 2, pk);
        if (n > 0 && __any_sync(0xffffffffu, need)) {
            uint32_t ov[32];
#pragma unroll
            for (int q = 0; q < kD; q += 32) {
                tmem_ld32(lane_base + S::col_o + q, ov);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * f);
                tmem_st32(lane_base + S::col_o + q, ov);
            }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_ready);
    }
    // the last P V is done: nothing reads shared memory any more (a lane whose wait ran out
    // leaves its warp's loop alone; the warp meets again here)
    __syncwarp();
    ok = __all_sync(0xffffffffu, ok) && mbar_wait_warp(&bars.o_done, (n - 1) & 1, abort, p.status, kStatusTimeout);
    tc_fence_after();
    if (row.i < 0) {
        m = -INFINITY;
        l = 0.f;
    }
    // copies of a row: a common maximum, then the sums
    float* out = reinterpret_cast<float*>(sm);
    sh_m[t] = m;
    sh_l[t] = l;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const int r = t & (kRows - 1);
    float M = m;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) M = fmaxf(M, sh_m[c * kRows + r]);
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - M);
    if (ok) {
        uint32_t ov[32];
#pragma unroll
        for (int q = 0; q < kD; q += 32) {
            tmem_ld32(lane_base + S::col_o + q, ov);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; c += 4)
                *reinterpret_cast<float4*>(out + t * S::out_pitch + q + c) =
                    make_float4(__uint_as_float(ov[c]) * f, __uint_as_float(ov[c + 1]) * f,
                                __uint_as_float(ov[c + 2]) * f, __uint_as_float(ov[c + 3]) * f);
        }
    }
    float L = 0.f;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
        const float mc = sh_m[c * kRows + r];
        L += sh_l[c * kRows + r] * (mc == -INFINITY ? 0.f : fast_exp2(mc - M));   // (a NaN sum stays one)
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    sh_m[t] = M;
    sh_l[t] = L;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (!ok) return;
    // kLanes lanes per row, 16 bytes of its output each
    constexpr int kLanes = kD / 4;
    const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
    const int col = 4 * (t & (kLanes - 1));
#pragma unroll 4
    for (int x = t / kLanes; x < w.there; x += 128 / kLanes) {
        const size_t at = (size_t)out_row[x];
        const float l_row = sh_l[x], m_row = sh_m[x];
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (l_row != 0.f)
#pragma unroll
            for (int k = 0; k < kCopies; ++k) {
                const float4 z = *reinterpret_cast<const float4*>(out + (k * kRows + x) * S::out_pitch + col);
                y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
            }
        if (p.nsplit > 1) {
            if (col < p.d) *reinterpret_cast<float4*>(p.po + (at * p.nsplit + split) * p.d + col) = y;
            if (col == 0) p.ml[at * p.nsplit + split] = make_float2(m_row, l_row);
        } else {
            const float inv = l_row != 0.f ? 1.f / l_row : 0.f;
            if (col < p.d)
                *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o + at * p.d + col) =
                    make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
            if (col == 0) p.lse[at] = l_row != 0.f ? (m_row + log2f(l_row)) * kLn2 : -INFINITY;
        }
    }
}

struct Shared {
    Bars bars;
    uint32_t tmem_base;
    int abort_flag, imin, imax, kinds, frozen_warps, lost;
    int out_row[128];
    float m[128], l[128];
};

// Every warp but the loading one: Q, tensor memory and the check of the pages are done.
__device__ __forceinline__ void set_up_done() {
    tc_fence_before();
    asm volatile("bar.sync 2, 224;" ::: "memory");
    tc_fence_after();
}

// Warps 0-3 of an item with keys.
template <int kD, int TK, int kCopies>
__device__ __forceinline__ void run_rows(const TcParams& P, const Work& w, const PagedRow& row, uint8_t* sm, Shared& sh) {
    using S = Smem<kD, TK>;
    const PagedArgs& p = P.a;
    const int t = threadIdx.x;
    // Q, one row per thread (zeros for frozen rows and those without a token)
    if (w.any_ord) {
        const bool have = row.i >= 0 && !row.frozen;
        const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.q + paged_out_row(p, row) * p.d);
        uint4 x[kD / 8];
#pragma unroll
        for (int c = 0; c < kD / 8; ++c) x[c] = have && 8 * c < p.d ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < kD / 8; ++c)
            *reinterpret_cast<uint4*>(sm + S::q + (c >> 3) * S::q_atom + sw128_offset(t, 16 * (c & 7))) = x[c];
        fence_proxy_async_smem();
    }
    if (t == 0 && sh.frozen_warps > 0) {
        mbar_init(&sh.bars.pat_empty[0], sh.frozen_warps);
        mbar_init(&sh.bars.pat_empty[1], sh.frozen_warps);
        fence_mbar_init();
    }
    set_up_done();
    const bool lost = sh.lost != 0;
    if (lost && t == 0) atomicOr(p.status, kStatusPage);
    row_warps<kD, TK, kCopies>(P, w, row, lost, sm, sh.bars, sh.out_row, sh.m, sh.l, sh.tmem_base, &sh.abort_flag);
}

// Warps 4-7 of an item with keys.
template <int kD, int TK>
__device__ __forceinline__ void run_others(const TcParams& P, const Work& w, uint8_t* sm, Shared& sh) {
    using S = Smem<kD, TK>;
    const PagedArgs& p = P.a;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    volatile int* abort = &sh.abort_flag;
    if (warp == 4) {   // K and V need nothing but the range of keys: on their way under the rest of the set-up
        load_warp<kD, TK>(P, w, sm, sh.bars, abort);
        return;
    }
    if (warp == 5) {
        tmem_alloc(&sh.tmem_base, 256);
        tmem_relinquish();
    }
    // pages that the item needs and the table does not have
    {
        const int nbox = TK / P.box, end = (w.e1 - w.e0) * nbox;
        bool lost = false;
        for (int b = t - 160; b < end; b += 96) {
            const int bx = paged_tile(w.g, w.e0 + b / nbox) * TK + (b & (nbox - 1)) * P.box;
            if (box_seen(w.g, bx, P.box) && paged_page(p, w.it, bx) < 0) lost = true;
        }
        if (lost) sh.lost = 1;
    }
    set_up_done();
    const uint32_t tmem = sh.tmem_base;
    const int n = w.e1 - w.e0;
    const uint32_t ring = smem_u32(sm + S::ring);
    Bars& bars = sh.bars;
    if (warp == 5) {
        // S of tile j, when K is there and the rows have read S of tile j - 1
        const uint32_t id_s = idesc_bf16(128, TK, 0, 0);
        const uint64_t d_q = sdesc_sw128(smem_u32(sm + S::q), 16, 1024);   // K-major, as K
        const uint64_t d_ring = sdesc_sw128(ring, 16, 1024);
        for (int j = 0; j < n && w.any_ord; ++j) {
            const int ld = w.k_load(j), s = ld % S::slots;
            if (!wait_all(&bars.full[s], (ld / S::slots) & 1, abort, p.status)) break;
            if (j > 0 && !wait_all(&bars.s_empty, (j - 1) & 1, abort, p.status)) break;
            tc_fence_after();
            const uint64_t d_k = sdesc_advance(d_ring, s * S::tile);
#pragma unroll
            for (int k = 0; k < kD / 16; ++k)
                mma_ss_warp(tmem, sdesc_advance(d_q, (k >> 2) * S::q_atom + (k & 3) * 32),
                            sdesc_advance(d_k, (k >> 2) * S::atom + (k & 3) * 32), id_s, k > 0);
            mma_commit_warp(&bars.s_full);
            mma_commit_warp(&bars.empty[s]);
        }
    } else if (warp == 6) {
        // O += P V of tile j, when V and the rows' weights are there
        const uint32_t id_o = idesc_bf16(128, kD, 0, 1);
        const uint64_t d_ring = sdesc_sw128(ring, S::atom, 1024);   // MN-major
        for (int j = 0; j < n; ++j) {
            const int ld = w.v_load(j), s = ld % S::slots;
            if (!wait_all(&bars.full[s], (ld / S::slots) & 1, abort, p.status)) break;
            if (!wait_all(&bars.p_ready, j & 1, abort, p.status)) break;
            tc_fence_after();
            const uint64_t d_v = sdesc_advance(d_ring, s * S::tile);
#pragma unroll
            for (int k = 0; k < TK / 16; ++k)
                mma_ts_warp(tmem + S::col_o, tmem + S::col_p + 8 * k, sdesc_advance(d_v, k * 2048), id_o,
                            (j > 0 || k > 0) ? 1u : 0u);
            mma_commit_warp(&bars.o_done);
            mma_commit_warp(&bars.empty[s]);
        }
    } else if (sh.frozen_warps > 0 && w.staged) {
        pattern_warp<kD, TK>(P, w, sm, bars, abort);
    }
    if (warp == 5 || warp == 6) {   // every MMA issued here is done before tensor memory is freed
        mma_commit_warp(&bars.mma_idle[warp - 5]);
        if (lane == 0) mbar_wait_bounded(&bars.mma_idle[warp - 5], 0, kWaitLimitNs);
        __syncwarp();
    }
}

template <int kD>
__global__ void __launch_bounds__(kThreads, 2) paged_tc_kernel(const __grid_constant__ TcParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Shared sh;
    const PagedArgs& p = P.a;
    grid_dep_wait();
    grid_dep_launch();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    Work w;
    w.it = paged_item(p, blockIdx.x);
    const int rows = p.rows[w.it.part];
    const PagedBlock block = paged_block(p, w.it);
    if (t == 0) {
        sh.abort_flag = 0;
        sh.imin = 0x7fffffff;
        sh.imax = -1;
        sh.kinds = sh.frozen_warps = sh.lost = 0;
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&sh.bars.full[i], 1);
            mbar_init(&sh.bars.empty[i], 1);
        }
        mbar_init(&sh.bars.s_full, 1);
        mbar_init(&sh.bars.s_empty, 4);
        mbar_init(&sh.bars.p_ready, 4);
        mbar_init(&sh.bars.o_done, 1);
        mbar_init(&sh.bars.pat_full[0], 1);
        mbar_init(&sh.bars.pat_full[1], 1);
        mbar_init(&sh.bars.mma_idle[0], 1);
        mbar_init(&sh.bars.mma_idle[1], 1);
        fence_mbar_init();
    }
    PagedRow row;
    if (t < 128) {
        row = paged_row(p, w.it, block, t & (rows - 1));
        sh.out_row[t] = row.there ? (int)paged_out_row(p, row) : -1;
    }
    __syncthreads();
    if (t < 128) {
        int lo = row.i >= 0 ? row.i : 0x7fffffff, hi = row.i;
        const int kinds = row.i < 0 ? 0 : row.frozen ? 2 : 1;
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        const int k = __reduce_or_sync(0xffffffffu, (unsigned)kinds);
        if (lane == 0) {
            atomicMin(&sh.imin, lo);
            atomicMax(&sh.imax, hi);
            atomicOr(&sh.kinds, k);
            if (k & 2) atomicAdd(&sh.frozen_warps, 1);
        }
    } else if (t == 128 && w.it.part == 1 && w.it.chunk == 0 && w.it.rb == 0 && w.it.hk == 0) {
        int c;   // each sequence's counts are checked once
        bool bad;
        paged_tokens(p, w.it.b, &c, &bad);
        if (bad) atomicOr(p.status, kStatusPage);
    }
    __syncthreads();
    w.imin = sh.imin;
    w.imax = sh.imax;
    w.any_ord = (sh.kinds & 1) != 0;
    w.off = w.it.part ? p.P : 0;
    w.there = block.there;
    w.g = paged_range(p, w.it, w.imin, w.imax, (sh.kinds & 2) != 0 || p.window == 0);
    const int per = p.per_chunk[w.it.part];
    w.e0 = min(w.it.chunk * per, w.g.n);
    w.e1 = min(w.e0 + per, w.g.n);
    if (w.e0 >= w.e1) {   // no keys: nothing but the rows' empty sums
        write_empty(p, w.it, w.there, sh.out_row, kThreads);
        return;
    }
    // the block's frozen heads: of its members of the group those from gord on
    w.f0 = max(block.first / block.per_head, (int)p.gord[w.it.hk]);
    w.nf = (block.first + w.there - 1) / block.per_head - w.f0 + 1;
    const int tile = p.tile[w.it.part];
    w.staged = (long long)w.nf * ((long long)w.imax - w.imin + 2 * tile + 3) <= kPatFloats;

    // one setmaxnreg for each warpgroup
    if (warp < 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
        switch (rows) {
            case 32: run_rows<kD, paged_tc_tile(kD, 32), 4>(P, w, row, sm, sh); break;
            case 64: run_rows<kD, paged_tc_tile(kD, 64), 2>(P, w, row, sm, sh); break;
            default: run_rows<kD, paged_tc_tile(kD, 128), 1>(P, w, row, sm, sh); break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (rows < 128) run_others<kD, paged_tc_tile(kD, 32)>(P, w, sm, sh);
        else run_others<kD, paged_tc_tile(kD, 128)>(P, w, sm, sh);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(sh.tmem_base, 256);
    }
}

template <int kD>
cudaError_t launch_d(const TcParams& P, cudaStream_t s) {
    const int smem = Smem<kD, 64>::total + 1024;
    static_assert(Smem<kD, 64>::total == Smem<kD, paged_tc_tile(kD, 32)>::total, "one layout for all tiles");
    static_assert(Smem<kD, 64>::slots <= kMaxSlots, "barriers of the ring");
    cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // A build that launches with fewer registers could never hand the row warps theirs (a
    // property of the compiled kernel, looked up once).
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, paged_tc_kernel<kD>);
        if (e != cudaSuccess) return e;
        regs.store(fa.numRegs);
    }
    if (kRegsRows + kRegsOther > 2 * regs.load()) return cudaErrorInvalidConfiguration;
    return launch_ex(paged_tc_kernel<kD>, dim3(P.a.items), dim3(kThreads), (size_t)smem, s, true, 1, P);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedArgs& a, cudaStream_t s) {
    TcParams P;
    P.a = a;
    const int page = 1 << a.page_log2;
    P.box = page < 64 ? page : 64;
    const uint64_t slices = (uint64_t)a.num_pages * a.Hkv;
    const void* k = a.k_cache ? a.k_cache : a.v_cache;   // (no K is loaded when every head is frozen)
    if (!make_tmap_bf16_3d(&P.tm_k, k, a.d, page, slices, 64, P.box) ||
        !make_tmap_bf16_3d(&P.tm_v, a.v_cache, a.d, page, slices, 64, P.box))
        return cudaErrorInvalidValue;
    return a.d == 64 ? launch_d<64>(P, s) : launch_d<128>(P, s);
}

}  // namespace saf
