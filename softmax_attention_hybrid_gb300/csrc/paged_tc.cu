// Paged attention on the 5th-generation tensor cores (bf16; see paged.h for the split).
//
// An item holds up to 128 query rows, the M = 128 rows of its MMAs, and walks its tiles of 64
// keys: S = Q K^T, online softmax with one thread per row, O += P V. Keys and values come
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
// issues S, 6 issues P V; 7 idles. Two issuers, since a tile's waits, MMAs and commits take
// one about 1600 cycles at d = 64 (traced; a wait costs about 100 and a commit as much),
// longer than the softmax of a tile.
// Tensor memory (256 columns): S [0, 64) fp32 | P [64, 96) bf16 pairs | O [128, 128 + d).
// S has columns of its own so that the next tile's S runs under this one's softmax.
// Shared memory: Q, and a ring of slots of one tile of K or V each, filled in the order in
// which the MMAs use them: K0, K1, V0, K2, V1, ... (V0, V1, ... where no row is ordinary).
//
// Bound by memory in decoding: a tile of K and V is 32 KB at d = 128, 1400 cycles of an SM's share
// of the memory, against 512 cycles of MMAs.
#include <string.h>

#include "paged.h"
#include "tc_common.cuh"

namespace saf {
namespace {

using namespace tc;

constexpr int kThreads = 256;
// Register split (setmaxnreg): warps 4-7 drop to kRegsOther, the row warps rise to kRegsRows, within
// the kRegsLaunch per thread that the launch hands out (checked on the host).
constexpr int kRegsLaunch = 128, kRegsRows = 184, kRegsOther = 72;
static_assert(kRegsRows + kRegsOther <= 2 * kRegsLaunch, "register split too large");
constexpr int TK = kTcTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // lazy rescale: factor 256
constexpr uint32_t kColP = 64, kColO = 128;

struct TcParams {
    CUtensorMap tm_k, tm_v;
    PagedArgs a;
    int box;   // rows of a TMA box: min(page, 64)
};

// kD: head dimension as the tiles hold it (64, or 128 for 96 and 128: TMA fills the columns
// past the row's end with zeros)
template <int kD>
struct Smem {
    static constexpr int atom = TK * 128;               // 64 keys x 64 columns
    static constexpr int tile = atom * (kD / 64);
    static constexpr int q_atom = 128 * 128;
    static constexpr int q = 0;
    static constexpr int ring = q + q_atom * (kD / 64);
    static constexpr int slots = kD == 64 ? 10 : 4;     // 80 KB, 64 KB: what two CTAs of an SM leave
    static constexpr int total = ring + slots * tile;
    // after the last MMA the whole region stages the output rows
    static constexpr int out_pitch = kD + 4;
    static_assert(128 * out_pitch * 4 <= total, "output staging");
};

template <int kD>
struct Bars {
    uint64_t full[Smem<kD>::slots], empty[Smem<kD>::slots];
    uint64_t s_full, s_empty, p_ready, o_done, mma_idle[2];
};

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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
    bool any_ord;     // an ordinary row is among them: K is loaded
    bool lost;        // a page that is needed is not in the cache

    // place of tile e0 + j's K and V in the order of loads
    __device__ __forceinline__ int k_load(int j) const { return j == 0 ? 0 : 2 * j - 1; }
    __device__ __forceinline__ int v_load(int j) const {
        if (!any_ord) return j;
        return j + 1 < e1 - e0 ? 2 * j + 2 : 2 * j + 1;
    }
};

// A wait of a converged warp: every lane waits and the warp goes on, or gives up, together.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, kStatusTimeout));
}

// Whether keys [bx, bx + box) of the part hold one that some row sees.
__device__ __forceinline__ bool box_seen(const PagedRange& g, int bx, int box) {
    return bx < g.hi && (bx + box > g.lo || bx < g.sink);
}

// The loading warp. Lane l fetches box l of every tile, from its page.
template <int kD>
__device__ __forceinline__ void load_warp(const TcParams& P, const Work& w, uint8_t* sm, Bars<kD>& bars,
                                          volatile int* abort) {
    using S = Smem<kD>;
    const PagedArgs& p = P.a;
    const int lane = threadIdx.x & 31;
    const int nbox = TK / P.box, n = w.e1 - w.e0;
    const int in_page = (1 << p.page_log2) - 1;
    const uint32_t box_bytes = (uint32_t)P.box * 128u * (kD / 64);
    if (lane == 0) {
        tma_prefetch_desc(&P.tm_k);
        tma_prefetch_desc(&P.tm_v);
    }
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

// kN consecutive values p[0 .. kN), of which p - 3 .. p + kN + 3 may be read, through aligned
// 16-byte loads (a quarter of the requests; neighbouring threads read far apart).
template <int kN>
__device__ __forceinline__ void load_run(const float* p, float* v) {
    const int m = (int)((uintptr_t)p >> 2) & 3;
    const float4* a = reinterpret_cast<const float4*>(p - m);
    float u[kN + 4];
#pragma unroll
    for (int c = 0; c < kN / 4 + 1; ++c) {
        const float4 x = __ldg(a + c);
        u[4 * c] = x.x;
        u[4 * c + 1] = x.y;
        u[4 * c + 2] = x.z;
        u[4 * c + 3] = x.w;
    }
#pragma unroll
    for (int c = 0; c < kN + 3; ++c) u[c] = (m & 1) ? u[c + 1] : u[c];
#pragma unroll
    for (int c = 0; c < kN; ++c) v[c] = (m & 2) ? u[c + 2] : u[c];
}

// The rows' part of an item: kCopies copies of 128 / kCopies rows; thread t holds row t mod
// (128 / kCopies) and the keys [kCols copy, ...) of every tile.
template <int kD, int kCopies>
__device__ __forceinline__ void row_warps(const TcParams& P, const Work& w, const PagedRow& row, uint8_t* sm,
                                          Bars<kD>& bars, const int* out_row, uint32_t tmem, volatile int* abort) {
    using S = Smem<kD>;
    const PagedArgs& p = P.a;
    constexpr int kCols = TK / kCopies, kRows = 128 / kCopies;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int c0 = (t / kRows) * kCols;   // my keys of a tile
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const int box_log2 = __ffs(P.box) - 1;
    const int i = row.i < 0 ? -1 : row.i - w.off;   // my last visible slot of the part
    const float sc = row.frozen ? 1.f : p.scale_log2;
    const bool frozen = row.frozen && i >= 0;
    const float* ra = p.a + (size_t)row.h * p.ld + w.off;
    const float* rr = p.r + (size_t)row.h * p.ld;
    float m = -INFINITY, l = 0.f;
    bool ok = true;

    if (kCopies > 1) {   // the other copies' keys: weights that stay zero
        uint32_t z[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) z[c] = 0u;
        tmem_st32(lane_base + kColP, z);
        tmem_st_wait();
    }
    int n = 0;
    for (int e = w.e0; e < w.e1; ++e, ++n) {
        const int x0 = paged_tile(w.g, e) * TK;
        float lg[kCols];   // a frozen row's logits (Eq. 3), loaded while S is computed
        if (frozen) {
            const int x = x0 + c0, back = i - x - (kCols - 1);   // r[back ..] backwards
            if (back >= 3 && i - x + 4 < p.ld) {
                load_run<kCols>(rr + back, lg);
#pragma unroll
                for (int c = 0; c < kCols / 2; ++c) {
                    const float y = lg[c];
                    lg[c] = lg[kCols - 1 - c];
                    lg[kCols - 1 - c] = y;
                }
#pragma unroll
                for (int c = 0; c < kCols; ++c) lg[c] += __ldg(ra + x + c);
            } else {   // slots past my own position are masked below
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const int y = min(x + c, i);
                    lg[c] = ra[y] + rr[i - y];
                }
            }
        }
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
        if (frozen)
#pragma unroll
            for (int c = 0; c < kCols; ++c) sv[c] = __float_as_uint(lg[c] * kLog2e);
        uint32_t have = 0xffffffffu;   // boxes whose page is in the cache
        if (w.lost)
            for (int b = 0; b < TK / P.box; ++b) {
                const int bx = x0 + b * P.box;
                if (box_seen(w.g, bx, P.box) && paged_page(p, w.it, bx) < 0) have &= ~(1u << b);
            }
        // masks, in tiles that some row does not see whole
        if (w.lost || x0 + TK > w.g.hi || x0 + TK - 1 > w.imin - w.off ||
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
        const float m_new = fmaxf(m, fmaxf(ma, mb) * sc);
        const bool need = m_new > m + kRescaleThreshold;
        const float f = need ? fast_exp2(m - m_new) : 1.f;
        if (need) {
            l *= f;
            m = m_new;
        }
        const float ref = m == -INFINITY ? 0.f : m;   // a row that has seen no key yet: weights 2^-inf = 0
        const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-ref, -ref);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
            const float2 x = ffma2(make_float2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sc2, nm2);
            const float2 ex = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            if (c & 1) acc1 = fadd2(acc1, ex);
            else acc0 = fadd2(acc0, ex);
            pk[c] = pack_bf16(ex.x, ex.y);
        }
        l += (acc0.x + acc1.x) + (acc0.y + acc1.y);
        // values of slots that no row sees may be anything: zeros, for 0 * NaN is none
        if (w.lost || x0 + TK > w.g.hi || (x0 < w.g.lo && x0 + TK > w.g.sink)) {
            const int ld = w.v_load(n), s = ld % S::slots;
            if (!(ok = mbar_wait(&bars.full[s], (ld / S::slots) & 1, abort, p.status, kStatusTimeout))) break;
            const int kk = t & 63, x = x0 + kk;
            const bool seen = x < w.g.hi && (x >= w.g.lo || x < w.g.sink) && ((have >> (kk >> box_log2)) & 1u);
            if (!seen) {
                constexpr int kHalf = kD == 128 ? 8 : 4;   // two threads per key
                uint8_t* vrow = sm + S::ring + s * S::tile + kk * 128 + (t >> 6) * (kD == 128 ? S::atom : 64);
#pragma unroll
                for (int c = 0; c < kHalf; ++c) *reinterpret_cast<uint4*>(vrow + 16 * c) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
        }
        if (n > 0) {   // P V of the previous tile is done: P is free, O is stable
            if (!(ok = mbar_wait(&bars.o_done, (n - 1) & 1, abort, p.status, kStatusTimeout))) break;
            tc_fence_after();
        }
        tmem_st_n<kCols / 2>(lane_base + kColP + c0 / 2, pk);
        if (n > 0 && __any_sync(0xffffffffu, need)) {
            uint32_t ov[32];
#pragma unroll
            for (int q = 0; q < kD; q += 32) {
                tmem_ld32(lane_base + kColO + q, ov);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * f);
                tmem_st32(lane_base + kColO + q, ov);
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
    __shared__ float sh_m[128], sh_l[128];
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
            tmem_ld32(lane_base + kColO + q, ov);
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
        if (mc != -INFINITY) L += sh_l[c * kRows + r] * fast_exp2(mc - M);
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    sh_m[t] = M;
    sh_l[t] = L;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (!ok) return;
    // a warp per row: whole rows to memory
    const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
    for (int x = warp; x < kRows; x += 4) {
        if (out_row[x] < 0) break;   // rows that are there come first
        const size_t at = (size_t)out_row[x];
        const float l_row = sh_l[x], m_row = sh_m[x];
        const float inv = p.nsplit > 1 ? 1.f : l_row > 0.f ? 1.f / l_row : 0.f;
        for (int c = 2 * lane; c < p.d; c += 64) {
            float2 y = make_float2(0.f, 0.f);
            if (l_row > 0.f)
#pragma unroll
                for (int k = 0; k < kCopies; ++k)
                    y = fadd2(y, *reinterpret_cast<const float2*>(out + (k * kRows + x) * S::out_pitch + c));
            if (p.nsplit > 1)
                *reinterpret_cast<float2*>(p.po + (at * p.nsplit + split) * p.d + c) = y;
            else
                *reinterpret_cast<uint32_t*>((__nv_bfloat16*)p.o + at * p.d + c) = pack_bf16(y.x * inv, y.y * inv);
        }
        if (lane == 0) {
            if (p.nsplit > 1) p.ml[at * p.nsplit + split] = make_float2(m_row, l_row);
            else p.lse[at] = l_row > 0.f ? (m_row + log2f(l_row)) * kLn2 : -INFINITY;
        }
    }
}

template <int kD>
__global__ void __launch_bounds__(kThreads, 2) paged_tc_kernel(const __grid_constant__ TcParams P) {
    using S = Smem<kD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Bars<kD> bars;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag, sh_imin, sh_imax, sh_kinds, out_row[128];
    const PagedArgs& p = P.a;
    grid_dep_wait();
    grid_dep_launch();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    Work w;
    w.it = paged_item(p, blockIdx.x);
    const int rows = p.rows[w.it.part];
    if (t == 0) {
        abort_flag = 0;
        sh_imin = 0x7fffffff;
        sh_imax = -1;
        sh_kinds = 0;
        for (int i = 0; i < S::slots; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.s_empty, 4);
        mbar_init(&bars.p_ready, 4);
        mbar_init(&bars.o_done, 1);
        mbar_init(&bars.mma_idle[0], 1);
        mbar_init(&bars.mma_idle[1], 1);
        fence_mbar_init();
    }
    __syncthreads();
    PagedRow row;
    if (t < 128) {
        row = paged_row(p, w.it, w.it.rb * rows + (t & (rows - 1)));
        out_row[t] = row.there ? (int)paged_out_row(p, row) : -1;
        int lo = row.i >= 0 ? row.i : 0x7fffffff, hi = row.i;
        const int kinds = row.i < 0 ? 0 : row.frozen ? 2 : 1;
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        const int k = __reduce_or_sync(0xffffffffu, (unsigned)kinds);
        if (lane == 0) {
            atomicMin(&sh_imin, lo);
            atomicMax(&sh_imax, hi);
            atomicOr(&sh_kinds, k);
        }
    } else if (t == 128 && w.it.part == 1 && w.it.chunk == 0 && w.it.rb == 0 && w.it.hk == 0) {
        int c;   // each sequence's counts are checked once
        bool bad;
        paged_tokens(p, w.it.b, &c, &bad);
        if (bad) atomicOr(p.status, kStatusPage);
    }
    __syncthreads();
    w.imin = sh_imin;
    w.imax = sh_imax;
    w.any_ord = (sh_kinds & 1) != 0;
    w.off = w.it.part ? p.P : 0;
    w.g = paged_range(p, w.it, w.imin, w.imax, (sh_kinds & 2) != 0 || p.window == 0);
    const int per = p.per_chunk[w.it.part];
    w.e0 = min(w.it.chunk * per, w.g.n);
    w.e1 = min(w.e0 + per, w.g.n);
    if (w.e0 >= w.e1) {   // no keys: nothing but the rows' empty sums
        const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
        for (int x = warp; x < rows; x += kThreads / 32) {
            if (out_row[x] < 0) break;
            const size_t at = (size_t)out_row[x];
            if (p.nsplit > 1) {
                if (lane == 0) p.ml[at * p.nsplit + split] = make_float2(-INFINITY, 0.f);
            } else {
                for (int c = 2 * lane; c < p.d; c += 64) *reinterpret_cast<uint32_t*>((__nv_bfloat16*)p.o + at * p.d + c) = 0u;
                if (lane == 0) p.lse[at] = -INFINITY;
            }
        }
        return;
    }
    if (warp == 5) {
        tmem_alloc(&tmem_base_sh, 256);
        tmem_relinquish();
    }
    // Q, one row per thread (zeros for frozen rows and those without a token)
    if (t < 128 && w.any_ord) {
        const bool have = row.i >= 0 && !row.frozen;
        const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.q + paged_out_row(p, row) * p.d);
#pragma unroll
        for (int c = 0; c < kD / 8; ++c) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (have && 8 * c < p.d) x = __ldg(src + c);
            *reinterpret_cast<uint4*>(sm + S::q + (c >> 3) * S::q_atom + sw128_offset(t, 16 * (c & 7))) = x;
        }
        fence_proxy_async_smem();
    }
    // pages that the item needs and the table does not have
    bool lost = false;
    {
        const int nbox = TK / P.box;
        for (int b = t; b < (w.e1 - w.e0) * nbox; b += kThreads) {
            const int bx = paged_tile(w.g, w.e0 + b / nbox) * TK + (b % nbox) * P.box;
            if (box_seen(w.g, bx, P.box) && paged_page(p, w.it, bx) < 0) lost = true;
        }
    }
    tc_fence_before();
    w.lost = __syncthreads_or(lost) != 0;
    tc_fence_after();
    if (w.lost && t == 0) atomicOr(p.status, kStatusPage);
    const uint32_t tmem = tmem_base_sh;
    volatile int* abort = &abort_flag;

    const int n = w.e1 - w.e0;
    const uint32_t ring = smem_u32(sm + S::ring);
    if (warp < 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
        switch (rows) {
            case 32: row_warps<kD, 4>(P, w, row, sm, bars, out_row, tmem, abort); break;
            case 64: row_warps<kD, 2>(P, w, row, sm, bars, out_row, tmem, abort); break;
            default: row_warps<kD, 1>(P, w, row, sm, bars, out_row, tmem, abort); break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 4) {
            load_warp<kD>(P, w, sm, bars, abort);
        } else if (warp == 5) {
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
                    mma_ts_warp(tmem + kColO, tmem + kColP + 8 * k, sdesc_advance(d_v, k * 2048), id_o,
                                (j > 0 || k > 0) ? 1u : 0u);
                mma_commit_warp(&bars.o_done);
                mma_commit_warp(&bars.empty[s]);
            }
        }
        if (warp == 5 || warp == 6) {   // every MMA issued here is done before tensor memory is freed
            mma_commit_warp(&bars.mma_idle[warp - 5]);
            if (lane == 0) mbar_wait_bounded(&bars.mma_idle[warp - 5], 0, kWaitLimitNs);
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int kD>
cudaError_t launch_d(const TcParams& P, cudaStream_t s) {
    const int smem = Smem<kD>::total + 1024;
    cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // a build that launches with fewer registers could never hand the row warps theirs
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, paged_tc_kernel<kD>);
    if (e != cudaSuccess) return e;
    if (kRegsRows + kRegsOther > 2 * fa.numRegs) return cudaErrorInvalidConfiguration;
    return launch_ex(paged_tc_kernel<kD>, dim3((unsigned)P.a.items), dim3(kThreads), (size_t)smem, s, true, 1, P);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedArgs& a, cudaStream_t s) {
    TcParams P;
    P.a = a;
    const int page = 1 << a.page_log2;
    P.box = page < TK ? page : TK;
    const uint64_t slices = (uint64_t)a.num_pages * a.Hkv;
    const void* k = a.k_cache ? a.k_cache : a.v_cache;   // (no K is loaded when every head is frozen)
    if (!make_tmap_bf16_3d(&P.tm_k, k, a.d, page, slices, 64, P.box) ||
        !make_tmap_bf16_3d(&P.tm_v, a.v_cache, a.d, page, slices, 64, P.box))
        return cudaErrorInvalidValue;
    return a.d == 64 ? launch_d<64>(P, s) : launch_d<128>(P, s);
}

}  // namespace saf
