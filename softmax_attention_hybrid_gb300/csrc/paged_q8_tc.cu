// Paged attention over 8-bit caches on the tensor cores (bf16 q and o; see paged.h for the split).
//
// Few rows meet many keys in a decoding step, so the keys take the M = 128 lanes of the MMAs
// and the rows (R = 4, 8, 16, 24 or 32 of a block) the columns:
//     S^T [128 keys, rows] = K q^T,      O^T [d, rows] += V^T P^T,
// with K and V as they lie in the cache: codes of e4m3 (kind::f8f6f4), never unpacked. A thread of
// the softmax holds one key of the tile, with that key's two scales, for all rows.
//
// The other operand is e4m3 too, as a sum of terms in columns of their own, which are added in
// fp32 when they are read:
//   q, scaled by a power of two so that the row's largest lies in (224, 448]: hi = e4m3(q),
//     lo = e4m3(16 (q - hi)), S = S_hi + S_lo / 16. Off by 2^-14 near zero, 2^-21 of the largest, else exact
//     (bf16 has 8 bits, each term 4).
//   w = P s_v 2^(4 - E) <= 256 with P s_v <= 2^E the row's products so far: hi = e4m3(w), mid = e4m3(16 (w - hi)),
//     lo = e4m3(256 (w - hi - mid / 16)). Off by 2^-12 of itself (bf16: 2^-8), or 2^-18 near zero, 2^-21 of the
//     row's largest. E is the row's own: with the largest scale in its place, a key with a large value would take
//     bits from rows that do not see it, or give it no weight.
// Sums are fp32 in tensor memory. The scale of a key multiplies its scores, that of its value the weight.
//
// The running maxima m of the scores and E of log2(P s_v), one each per row, are those of all 128 keys: a tile whose
// scores stay below m + 4 and whose products stay below 2^(E + 4) leaves them (one barrier with an OR); else
// they are found anew, and O and l are scaled. Tiles are walked from the newest key to the oldest: the
// patterns of frozen heads, and most ordinary rows, look nearby first, so that the maximum is found early.
//
// 32 sequences of 4K to 16K tokens, 32 heads over 8 of 128 (a quarter frozen): 120 us, 5.9 TB/s, 87% of a plain copy's rate.
// 64 sequences with a window of 1024: 42 us (512 items of 10 tiles on 456 places, and what an item costs beside its
// tiles: counts, page, first load, softmax and product one after the other, 7 us). Five tokens each of 16 sequences, 20
// rows: 72 us with two warpgroups in the softmax (some 7 more with one); a tile takes a CTA about 2700 cycles alone, two on
// an SM 4200 (issue slots 49%), and SMs with two of the longest items run the longest. (With one unit for all rows of a
// warpgroup, the largest value scale, these took 119, 41 and 71 us, and rows beside large values came out wrong.)
//
// Warps (256 threads, two CTAs per SM, three with 4 rows; 384 threads from 16 rows on): a warpgroup of the softmax, from 16 rows
// on two with half of the rows each; then a warp that loads K, V and their scales (each of its lanes fetches one page of the
// tile), one that owns tensor memory and issues S, one that issues P V. (The last completes the
// warpgroup: from 16 rows on the softmax takes registers over from it, since what it spills costs the latency of the L2
// each time in the little L1 that is left.)
// Shared memory: q's terms (K-major, 128-byte swizzle), P's terms of two tiles (MN-major: the 16 bytes of
// a key's columns next to each other), and a ring of tiles of 128 keys with their scales, filled in the order in
// which the MMAs use them: K0, K1, V0, K2, V1, ... (V0, V1, ... where no row is ordinary). Rows of d < 128
// codes are filled up with zeros by TMA.
#include <string.h>

#include <atomic>

#include "paged_q8.cuh"

namespace saf {
namespace {

using namespace paged_q8;

// Register split (setmaxnreg) from 16 rows on, within the kRegsLaunch per thread that the launch hands out (checked on the host).
constexpr int kRegsLaunch = 80, kRegsRows = 96, kRegsOther = 48;
static_assert(2 * kRegsRows + kRegsOther <= 3 * kRegsLaunch, "register split too large");
constexpr int kTile = kQ8Tile;            // keys of a tile
constexpr int kTileBytes = kTile * 128;
constexpr int kScaleBytes = kTile * 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 4.0f;            // scores may pass the maximum by this much (base 2)
// A row that has seen no key yet: below every finite score (those of patterns are at least -2.3e38 log2(e)).
constexpr float kNoMax = -3.4e38f;
constexpr int kAhead = 8;                 // frozen rows whose patterns are loaded a tile ahead
constexpr int kWeightExp = 4;              // 8 - kSlack: a weight times its value's scale at the maximum is 2^4
// Bounds of E: 2^(4 - E) is a float, and no product of a weight below 2^4 and a finite scale is 2^128 or more.
constexpr int kLeastExp = -123, kMostExp = 128;

template <int R>
struct Cfg {
    static constexpr int groups = R > 8 ? 2 : 1;      // warpgroups of the softmax,
    static constexpr int rows = R / groups;           // and the rows of each
    static constexpr int threads = 128 * groups + 128;
    static constexpr int ns = R == 4 ? 16 : 2 * R;    // columns of S: a group's hi, lo, the next one's (of an MMA at least 16)
    // columns of O, and bytes of a key's weights: a group's hi, mid, lo, the next one's, in 16-byte blocks
    static constexpr int pb = groups == 1 ? (3 * R + 15) / 16 * 16 : (3 * rows + 7) / 8 * 8;
    static constexpr int np = groups * pb;
    static constexpr int blocks = np / 16;
    static constexpr int tile = kTile;
    static constexpr int ctas = R == 4 ? 3 : 2;       // of an SM
    static constexpr int slots = R == 4 ? 4 : R == 8 ? 6 : R == 16 ? 5 : 4;
    static constexpr int ring = 0;
    static constexpr int q = ring + slots * kTileBytes;
    static constexpr int p = q + ns * 128;
    static constexpr int p_bytes = blocks * kTile * 16;
    static constexpr int scales = p + 2 * p_bytes;
    static constexpr bool split = groups == 2;
    static constexpr int total = scales + slots * kScaleBytes;
    static_assert(total + 4 * 1024 <= (ctas == 3 ? 76 : 114) * 1024, "CTAs of an SM");
    static constexpr uint32_t col_o = 2 * ns;         // S of two tiles, then O
    static constexpr uint32_t cols = R <= 8 ? 64 : R == 16 ? 128 : 256;
    static_assert(col_o + np <= cols, "tensor memory");
    static_assert(p % 128 == 0 && q % 1024 == 0, "operand alignment");
};
constexpr int kMaxSlots = 6;

struct Bars {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t s_full[2], s_empty[2], p_ready[2], o_done[2], mma_idle[2];
};

template <int R>
struct Shared {
    Bars bars;
    uint32_t tmem_base;
    int abort_flag;
    int lost;                      // a page that the item needs is not in the cache (set before its tile is there)
    // rows of the block: ordinary ones from the front, frozen ones from the back
    alignas(16) float scale[R];    // what a score times its key's scale is multiplied by: log2(e) / sqrt(d), and q's factor back
    alignas(16) float nm[R];       // running maxima, negated
    alignas(16) float nlim[R];     // E, negated
    alignas(16) float gain[R];     // 2^(4 - E)
    alignas(16) float fall[R];     // 2^(old maximum - new one)
    alignas(16) float fall_o[R];   // the same of O, whose unit is 2^(m + E - 4)
    float most[R];                 // log2 of the largest product of a weight and its value's scale
    int out_row[R], pos[R];        // place in o (-1: none), last visible slot of the part (-1: none)
    const float* a[R];             // frozen rows: a and r at the part's slot 0 and at the row's distance from it
    const float* r[R];
    float part[4 * Cfg<R>::groups][Cfg<R>::rows];   // the warps' maxima, and sums
};

// OR over the 128 threads of a warpgroup of the softmax, who all wait for each other.
__device__ __forceinline__ bool rows_any(bool x, int group) {
    uint32_t y;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(y)
        : "r"((uint32_t)x), "r"(1 + 2 * group)
        : "memory");
    return y != 0;
}
__device__ __forceinline__ void rows_sync(int group) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + 2 * group) : "memory");
}

__device__ __forceinline__ float log2_of(float x) {   // to 2^-22, or a step of it
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Largest of a warp's values (NaN left out), by integers that have the order of the floats.
__device__ __forceinline__ float warp_max(float x) {
    int k = x == x ? __float_as_int(x) : (int)0xff800000;
    k ^= (k >> 31) & 0x7fffffff;
    k = __reduce_max_sync(0xffffffffu, k);
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// Rows of q on their way, a warp's every fourth or eighth (in: the rows' places in o).
template <int R>
__device__ __forceinline__ void get_q(const Q8Params& P, const Work& w, int place, uint2* x) {
    const PagedArgs& p = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < Cfg<R>::rows / 4; ++k) {
        const int r = 4 * Cfg<R>::groups * k + warp, at = __shfl_sync(0xffffffffu, place, r);
        x[k] = make_uint2(0, 0);
        if (r < w.there - w.nf && 4 * lane < p.d)
            x[k] = __ldg(reinterpret_cast<const uint2*>((const __nv_bfloat16*)p.q + (size_t)at * p.d) + lane);
    }
}

// q's terms of the block's ordinary rows, and the rows' factors.
template <int R>
__device__ __forceinline__ void put_q(const Q8Params& P, const Work& w, uint8_t* sm, Shared<R>& sh, const uint2* q) {
    const PagedArgs& p = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool mine = 4 * lane < p.d;
#pragma unroll
    for (int k = 0; k < Cfg<R>::rows / 4; ++k) {
        const int r = 4 * Cfg<R>::groups * k + warp, place = r + r / Cfg<R>::rows * Cfg<R>::rows;   // of its hi in S
        if (r >= w.there - w.nf || sh.pos[r] < 0) continue;   // (uniform)
        const uint2 x = q[k];
        const float v[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                            __uint_as_float(x.y & 0xffff0000u)};
        // the row's largest magnitude as bits: above 0x7f7fffff it holds an infinity or a NaN
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) top = max(top, __float_as_uint(v[c]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        // 448 = 1.75 x 2^8
        int e = 8 - ((int)(top >> 23) - 127) - ((top & 0x7fffffu) > 0x600000u);
        e = top >= 0x7f800000u ? 0 : e < -120 ? -120 : e > 120 ? 120 : e;
        const float f = pow2i(e);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float y0 = v[2 * c] * f, y1 = v[2 * c + 1] * f;
            hi[c] = pack_e4m3(y0, y1);
            const float2 z = unpack_e4m3(hi[c]);
            lo[c] = pack_e4m3(16.f * (y0 - z.x), 16.f * (y1 - z.y));
        }
        uint32_t word[2] = {hi[0] | hi[1] << 16, lo[0] | lo[1] << 16};
        if (top >= 0x7f800000u) word[0] = word[1] = 0x7f7f7f7fu;   // (saturation would hide an infinity)
        if (mine) {
            *reinterpret_cast<uint32_t*>(sm + Cfg<R>::q + sw128_offset(place, 4 * lane)) = word[0];
            *reinterpret_cast<uint32_t*>(sm + Cfg<R>::q + sw128_offset(place + Cfg<R>::rows, 4 * lane)) = word[1];
        }
        if (lane == 0) sh.scale[r] = p.scale_log2 * pow2i(-e);
    }
}

// Every warp but the loading one: q's terms and tensor memory are there.
template <int R>
__device__ __forceinline__ void set_up_done() {
    tc_fence_before();
    asm volatile("bar.sync 2, %0;" ::"n"(128 * Cfg<R>::groups + 64) : "memory");
    tc_fence_after();
}

// hi + lo / 16 of N rows
template <int N>
__device__ __forceinline__ void read_s(uint32_t addr, float* s) {
    uint32_t x[2 * N];
    if constexpr (N == 4) tmem_ld8(addr, x);
    else if constexpr (N == 16) tmem_ld32(addr, x);
    else tmem_ld16(addr, x);
    if constexpr (N == 12) tmem_ld8(addr + 16, x + 16);
    tmem_ld_wait();
#pragma unroll
    for (int r = 0; r < N; ++r) s[r] = fmaf(__uint_as_float(x[N + r]), 0.0625f, __uint_as_float(x[r]));
}

// N columns of tensor memory, 8 or 16 at a time.
template <int N>
__device__ __forceinline__ void read_columns(uint32_t addr, uint32_t* x) {
    if constexpr (N == 16) tmem_ld16(addr, x);
    else tmem_ld8(addr, x);
}
template <int N>
__device__ __forceinline__ void write_columns(uint32_t addr, const uint32_t* x) {
    if constexpr (N == 16) tmem_st16(addr, x);
    else tmem_st8(addr, x);
}

// Warps 0-3, and 4-7 from 16 rows on: a warpgroup holds R / groups of the rows. Thread t of it holds key t of every
// tile. Loops over rows have no branches: rows behind
// the last one have columns of their own that nobody reads.
template <int R>
__device__ __forceinline__ void row_warps(const Q8Params& P, const Work& w, const uint2* q, uint8_t* sm, Shared<R>& sh) {
    using C = Cfg<R>;
    constexpr int N = C::rows;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const int g = C::groups == 1 ? 0 : (int)(threadIdx.x >> 7), r0 = g * N;   // my group and its first row
    const int t = threadIdx.x & 127, warp = t >> 5, lane = t & 31;
    const int nf = C::groups == 1 ? w.nf : g ? min(w.nf, N) : max(w.nf - N, 0), tiles = w.e1 - w.e0;
    const float* scale_q = sh.scale + r0;
    const float* nm = sh.nm + r0;
    const float* nlim = sh.nlim + r0;
    const float* gain = sh.gain + r0;
    const int* pos = sh.pos + r0;
    const float* const* pa = sh.a + r0;
    const float* const* ra_ = sh.r + r0;
    float(*part)[N] = sh.part + 4 * g;
    const int my_box = t / P.box * P.box;
    float l[N];
#pragma unroll
    for (int r = 0; r < N; ++r) l[r] = 0.f;
    bool ok = true;

    // The fixed patterns' entries (Eq. 3) of my key, a tile ahead: neighbouring keys, neighbouring entries. Frozen
    // rows stand at the end, the first of them last, so that registers hold them; four at a time, for a branch for each
    // row costs as much as its entries (keys past the row's own position are masked below, and what is loaded for
    // a place without a frozen row is not used).
    constexpr int kA = N < kAhead ? N : kAhead;
    float fa[kA], fr[kA];
    auto ahead = [&](int j) {
        const int x = w.slot0(j, kTile) + t;
#pragma unroll
        for (int k0 = 0; k0 < kA; k0 += 4)
            if (k0 < nf) {
#pragma unroll
                for (int k = k0; k < k0 + 4; ++k) {
                    const int y = max(min(x, pos[N - 1 - k]), 0);
                    fa[k] = __ldg(pa[N - 1 - k] + y);
                    fr[k] = __ldg(ra_[N - 1 - k] - y);
                }
            }
    };
    if (nf > 0) ahead(0);
    if (w.any_ord) {
        put_q<R>(P, w, sm, sh, q);
        fence_proxy_async_smem();
    }
    set_up_done<R>();
    const uint32_t tmem = sh.tmem_base + ((uint32_t)(warp * 32) << 16);

    constexpr int kStep = C::pb % 16 ? 8 : 16;   // columns of O at a time
    int n = 0;
    for (; n < tiles; ++n) {
        const int x0 = w.slot0(n, kTile), x = x0 + t, buf = n & 1;
        float s[N];
        if (w.any_ord) {
            const int ld = w.k_load(n), slot = ld % C::slots;
            ok = mbar_wait(&bars.s_full[buf], (n >> 1) & 1, abort, p.status, kStatusTimeout) && ok;
            ok = mbar_wait(&bars.full[slot], (ld / C::slots) & 1, abort, p.status, kStatusTimeout) && ok;
            __syncwarp();
            tc_fence_after();
            const float ks = reinterpret_cast<const float*>(sm + C::scales + slot * kScaleBytes)[t];
            read_s<N>(tmem + buf * C::ns + g * 2 * N, s);
            tc_fence_before();
            // Every lane's scale must be in its register before the slot is given back, and nothing here waits for that
            // otherwise: reads of shared memory that other blocks' writes hold up (masked tiles) then found the next load's
            // scales. So the arrival takes a value from them (the comparison always holds).
            const bool read = __reduce_or_sync(0xffffffffu, __float_as_uint(ks) & 0x7fffffffu) != 0xffffffffu;
            if (lane == 0 && read) {
                mbar_arrive(&bars.s_empty[buf]);
                mbar_arrive(&bars.empty[slot]);
            }
#pragma unroll
            for (int r = 0; r < N; r += 4) {
                const float4 q = *reinterpret_cast<const float4*>(&scale_q[r]);
                s[r] *= ks * q.x;
                s[r + 1] *= ks * q.y;
                s[r + 2] *= ks * q.z;
                s[r + 3] *= ks * q.w;
            }
        } else {
#pragma unroll
            for (int r = 0; r < N; ++r) s[r] = -INFINITY;
        }
        if (nf > 0) {
#pragma unroll
            for (int k0 = 0; k0 < N; k0 += 4)
                if (k0 < nf) {
#pragma unroll
                    for (int k = k0; k < k0 + 4; ++k) {
                        const int r = N - 1 - k;
                        float y;
                        if (k < kA) {
                            y = fa[k < kA ? k : 0] + fr[k < kA ? k : 0];
                        } else {
                            const int z = max(min(x, pos[r]), 0);
                            y = __ldg(pa[r] + z) + __ldg(ra_[r] - z);
                        }
                        s[r] = k < nf ? y * kLog2e : s[r];
                    }
                }
            if (n + 1 < tiles) ahead(n + 1);
        }
        const int ldv = w.v_load(n), vslot = ldv % C::slots;
        ok = mbar_wait(&bars.full[vslot], (ldv / C::slots) & 1, abort, p.status, kStatusTimeout) && ok;
        float vs = reinterpret_cast<const float*>(sm + C::scales + vslot * kScaleBytes)[t];
        const bool lost = *(volatile int*)&sh.lost != 0;
        // masks, in tiles that some row does not see whole
        if (lost || x0 + kTile > w.g.hi || x0 + kTile - 1 > w.imin - w.off ||
            (p.window > 0 && x0 <= w.imax - w.off - p.window)) {
            const bool have = !(lost && box_seen(w.g, x0 + my_box, P.box) && paged_page(p, w.it, x0 + my_box) < 0);
            const bool any = have && x < w.g.hi && (x >= w.g.lo || x < w.g.sink);
            const int sink = p.sinks - w.off;
#pragma unroll
            for (int r = 0; r < N; ++r) {
                const int i = pos[r];
                const int lo = r >= N - nf || p.window == 0 ? -1 : i - p.window;   // slots <= lo: sinks only
                if (!(any && x <= i && (x > lo || x < sink))) s[r] = -INFINITY;
            }
            if (!any) {   // codes and scales of slots that no row sees may be anything: zeros, for 0 * NaN is none
                vs = 0.f;
            }
            if (!any && g == 0) {
                uint4* row = reinterpret_cast<uint4*>(sm + C::ring + vslot * kTileBytes + t * 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
            }
        }
        // (an infinite scale stands for rows of NaN; as a term of e4m3 the weight would saturate)
        if (!(vs <= 3.402823466e38f)) vs = __int_as_float(0x7fffffff);
        // by how much a score passes its row's maximum, or its product with the value's scale the limit (a NaN does not)
        float past = 0.f;
        const float lv = log2_of(vs);
#pragma unroll
        for (int r = 0; r < N; r += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&nm[r]), e = *reinterpret_cast<const float4*>(&nlim[r]);
            const float2 d0 = fadd2(make_float2(s[r], s[r + 1]), make_float2(m.x, m.y));
            const float2 d1 = fadd2(make_float2(s[r + 2], s[r + 3]), make_float2(m.z, m.w));
            const float2 u0 = fadd2(d0, fadd2(make_float2(lv, lv), make_float2(e.x, e.y)));
            const float2 u1 = fadd2(d1, fadd2(make_float2(lv, lv), make_float2(e.z, e.w)));
            past = fmax3(past, d0.x, d0.y);
            past = fmax3(past, d1.x, d1.y);
            past = fmax3(past, u0.x, u0.y);
            past = fmax3(past, u1.x, u1.y);
        }
        if (rows_any(past > kSlack || !ok, g)) {
            if (rows_any(!ok, g)) break;   // every thread leaves here
#pragma unroll
            for (int r = 0; r < N; ++r) {
                const float mx = warp_max(s[r]);
                if (lane == 0) part[warp][r] = mx;
            }
            rows_sync(g);
            float rise = 0.f;   // of my row's maximum
            if (t < N) {
                const float old = -nm[t];
                const float now = fmaxf(fmaxf(fmaxf(part[0][t], part[1][t]), fmaxf(part[2][t], part[3][t])), old);
                rise = now > old ? now - old : 0.f;
                sh.nm[r0 + t] = -now;
                sh.fall[r0 + t] = fast_exp2(-rise);
            }
            rows_sync(g);
            // (after the maximum was taken off: beside a large score the scale's part would be rounded away)
#pragma unroll
            for (int r = 0; r < N; ++r) {
                const float mx = warp_max((s[r] + nm[r]) + lv);
                if (lane == 0) part[warp][r] = mx;
            }
            rows_sync(g);
            if (t < N) {
                const float most = fmaxf(fmaxf(fmaxf(part[0][t], part[1][t]), fmaxf(part[2][t], part[3][t])),
                                         sh.most[r0 + t] - rise);
                const float e = fminf(fmaxf(ceilf(most), (float)kLeastExp), (float)kMostExp);
                // 2^(E - rise - new E), whole powers apart from the rest: the sum of both would round the rest
                const float whole = rintf(rise), n2 = -nlim[t] - whole - e;
                sh.fall_o[r0 + t] = n2 < -149.f ? 0.f : exp2f(whole - rise) * pow2i((int)n2);
                sh.most[r0 + t] = most;
                sh.nlim[r0 + t] = -e;
                sh.gain[r0 + t] = pow2i(kWeightExp - (int)e);
            }
            rows_sync(g);
#pragma unroll
            for (int r = 0; r < N; ++r) l[r] *= sh.fall[r0 + r];
            if (n > 0) {   // P V of the previous tile is done: O is stable
                ok = mbar_wait(&bars.o_done[buf ^ 1], ((n - 1) >> 1) & 1, abort, p.status, kStatusTimeout) && ok;
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < C::pb; c += kStep) {
                    uint32_t o[kStep];
                    read_columns<kStep>(tmem + C::col_o + g * C::pb + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < kStep; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) * sh.fall_o[r0 + (c + k) % N]);
                    write_columns<kStep>(tmem + C::col_o + g * C::pb + c, o);
                }
                tmem_st_wait();
                tc_fence_before();
            }
        }
        if (n > 1)   // P V of the tile before the previous one is done: its weights' buffer is free
            ok = mbar_wait(&bars.o_done[buf], ((n - 2) >> 1) & 1, abort, p.status, kStatusTimeout) && ok;
        uint8_t* mine = sm + C::p + buf * C::p_bytes + t * 16;
        uint32_t word[C::pb / 4];   // bytes: columns of the terms, hi, mid, lo
        word[C::pb / 4 - 1] = word[C::pb / 4 - 2] = 0u;   // (what the terms leave)
#pragma unroll
        for (int r = 0; r < N; r += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&nm[r]), e = *reinterpret_cast<const float4*>(&gain[r]);
            const float2 d[2] = {fadd2(make_float2(s[r], s[r + 1]), make_float2(m.x, m.y)),
                                 fadd2(make_float2(s[r + 2], s[r + 3]), make_float2(m.z, m.w))};
            const float2 up[2] = {make_float2(e.x, e.y), make_float2(e.z, e.w)};
            uint32_t h[2], md[2], lo[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float2 pr = make_float2(fast_exp2(d[c].x), fast_exp2(d[c].y));
                l[r + 2 * c] += pr.x;
                l[r + 2 * c + 1] += pr.y;
                // (the gain last: a weight of 0 times a large scale stays 0, for any gain)
                const float2 w2 = fmul2(fmul2(pr, make_float2(vs, vs)), up[c]);
                const float y0 = w2.x, y1 = w2.y;
                h[c] = pack_e4m3(y0, y1);
                float2 z = unpack_e4m3(h[c]);
                const float a0 = 16.f * (y0 - z.x), a1 = 16.f * (y1 - z.y);
                md[c] = pack_e4m3(a0, a1);
                z = unpack_e4m3(md[c]);
                lo[c] = pack_e4m3(16.f * (a0 - z.x), 16.f * (a1 - z.y));
            }
            word[r / 4] = h[0] | h[1] << 16;
            word[N / 4 + r / 4] = md[0] | md[1] << 16;
            word[N / 2 + r / 4] = lo[0] | lo[1] << 16;
        }
        if constexpr (C::pb % 16 == 0) {
#pragma unroll
            for (int b = 0; b < C::pb / 16; ++b)
                *reinterpret_cast<uint4*>(mine + (g * (C::pb / 16) + b) * kTile * 16) =
                    make_uint4(word[4 * b], word[4 * b + 1], word[4 * b + 2], word[4 * b + 3]);
        } else {   // the groups share a block
            const int skip = 2 * g;   // words of mine in it: the last two of group 0, the first two of group 1
            *reinterpret_cast<uint2*>(mine + C::pb / 16 * kTile * 16 + 8 * g) =
                g ? make_uint2(word[0], word[1]) : make_uint2(word[C::pb / 4 - 2], word[C::pb / 4 - 1]);
#pragma unroll
            for (int b = 0; b < C::pb / 16; ++b)
                *reinterpret_cast<uint4*>(mine + (g * (C::pb / 16 + 1) + b) * kTile * 16) =
                    skip ? make_uint4(word[4 * b + 2], word[4 * b + 3], word[4 * b + 4], word[4 * b + 5])
                         : make_uint4(word[4 * b], word[4 * b + 1], word[4 * b + 2], word[4 * b + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bars.p_ready[buf]);
            mbar_arrive(&bars.empty[vslot]);
        }
    }
    // (a lane whose wait ran out has left with all the others, or does so below)
    if (n > 0) ok = mbar_wait(&bars.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort, p.status, kStatusTimeout) && ok;
    __syncwarp();
    tc_fence_after();
#pragma unroll
    for (int r = 0; r < N; ++r) {
        float x = l[r];
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) part[warp][r] = x;
    }
    if (rows_any(!ok, g)) return;
    // O of element t of a row: the terms' sums
    const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
    uint32_t y[C::pb];
#pragma unroll
    for (int c = 0; c < C::pb; c += kStep) read_columns<kStep>(tmem + C::col_o + g * C::pb + c, y + c);
    tmem_ld_wait();
#pragma unroll
    for (int r = 0; r < N; ++r) {
        if (sh.out_row[r0 + r] < 0) continue;
        const float o = fmaf(fmaf(__uint_as_float(y[2 * N + r]), 0.0625f, __uint_as_float(y[N + r])), 0.0625f,
                             __uint_as_float(y[r])) * pow2i(-(int)nlim[r] - kWeightExp);
        const size_t at = (size_t)sh.out_row[r0 + r];
        const bool sees = pos[r] >= 0;
        const float lr = sees ? (part[0][r] + part[1][r]) + (part[2][r] + part[3][r]) : 0.f;
        const float mr = lr != 0.f ? -nm[r] : -INFINITY;
        if (p.nsplit > 1) {
            if (t < p.d) p.po[(at * p.nsplit + split) * p.d + t] = lr != 0.f ? o : 0.f;
            if (t == 0) p.ml[at * p.nsplit + split] = make_float2(mr, lr);
        } else {
            if (t < p.d) ((__nv_bfloat16*)p.o)[at * p.d + t] = __float2bfloat16_rn(lr != 0.f ? o / lr : 0.f);
            if (t == 0) p.lse[at] = lr != 0.f ? (mr + log2f(lr)) * kLn2 : -INFINITY;
        }
    }
}

// The first warp behind the loading one issues S, the second P V.
template <int R>
__device__ __forceinline__ void issue_warps(const Q8Params& P, const Work& w, uint8_t* sm, Shared<R>& sh) {
    using C = Cfg<R>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const int role = (int)(threadIdx.x >> 5) - 4 * C::groups - 1, lane = threadIdx.x & 31, n = w.e1 - w.e0;
    if (role == 0) {
        tmem_alloc(&sh.tmem_base, C::cols);
        tmem_relinquish();
    }
    set_up_done<R>();
    const uint32_t tmem = sh.tmem_base;
    const uint32_t ring = smem_u32(sm + C::ring);
    if (role == 0) {
        // S of tile j, when K is there and the rows have read S of tile j - 2
        constexpr uint32_t id_s = idesc_e4m3(128, C::ns, 0, 0);
        const uint64_t d_q = sdesc_sw128(smem_u32(sm + C::q), 16, 1024);   // K-major, as K
        const uint64_t d_ring = sdesc_sw128(ring, 16, 1024);
        const int steps = p.d / 32;
        for (int j = 0; j < n && w.any_ord; ++j) {
            const int ld = w.k_load(j), s = ld % C::slots;
            if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) break;
            if (j > 1 && !wait_all(&bars.s_empty[j & 1], ((j - 2) >> 1) & 1, abort, p.status)) break;
            tc_fence_after();
            const uint64_t d_k = sdesc_advance(d_ring, s * kTileBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < steps)
                    mma_ss_e4m3_warp(tmem + (j & 1) * C::ns, sdesc_advance(d_k, 32 * k), sdesc_advance(d_q, 32 * k),
                                 id_s, k > 0);
            mma_commit_warp(&bars.s_full[j & 1]);
            mma_commit_warp(&bars.empty[s]);
        }
    } else {
        // O^T += V^T P^T of tile j, when V and the weights are there
        constexpr uint32_t id_o = idesc_e4m3(128, C::np, 1, 1);
        const uint64_t d_ring = sdesc_sw128(ring, 16384, 1024);                        // MN-major
        const uint64_t d_p = sdesc_none(smem_u32(sm + C::p), 128, kTile * 16);
        for (int j = 0; j < n; ++j) {
            const int ld = w.v_load(j), s = ld % C::slots;
            if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) break;
            if (!wait_all(&bars.p_ready[j & 1], (j >> 1) & 1, abort, p.status)) break;
            tc_fence_after();
            const uint64_t d_v = sdesc_advance(d_ring, s * kTileBytes);
            const uint64_t d_w = sdesc_advance(d_p, (j & 1) * C::p_bytes);
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
                mma_ss_e4m3_warp(tmem + C::col_o, sdesc_advance(d_v, 4096 * k), sdesc_advance(d_w, 512 * k), id_o,
                                 (j > 0 || k > 0) ? 1u : 0u);
            mma_commit_warp(&bars.o_done[j & 1]);
            mma_commit_warp(&bars.empty[s]);
        }
    }
    // every MMA issued here is done before tensor memory is freed
    mma_commit_warp(&bars.mma_idle[role]);
    if (lane == 0) mbar_wait_bounded(&bars.mma_idle[role], 0, kWaitLimitNs);
    __syncwarp();
}

template <int R>
__global__ void __launch_bounds__(Cfg<R>::threads, Cfg<R>::ctas) paged_q8_kernel(const __grid_constant__ Q8Params P) {
    using C = Cfg<R>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Shared<R> sh;
    const PagedArgs& p = P.a;
    constexpr int kRowWarps = 4 * C::groups;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if (t == 0) {
        sh.abort_flag = sh.lost = 0;
        for (int i = 0; i < C::slots; ++i) {
            mbar_init(&sh.bars.full[i], 1);
            mbar_init(&sh.bars.empty[i], 1 + kRowWarps);   // the MMAs, and the warps that read the scales
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.bars.s_full[i], 1);
            mbar_init(&sh.bars.s_empty[i], kRowWarps);
            mbar_init(&sh.bars.p_ready[i], kRowWarps);
            mbar_init(&sh.bars.o_done[i], 1);
            mbar_init(&sh.bars.mma_idle[i], 1);
        }
        fence_mbar_init();
    }
    Work w;
    w.it = paged_item(p, blockIdx.x);
    w.off = w.it.part ? p.P : 0;
    const PagedBlock block = paged_block(p, w.it);
    w.there = block.there;
    // every warp finds the rows for itself, a lane each: nobody waits for another's loads
    const PagedRow row = paged_place(p, w.it, block, lane);
    const int place = row.there ? (int)paged_out_row(p, row) : -1;
    const uint32_t kind = __ballot_sync(0xffffffffu, row.there && row.frozen);
    w.nf = __popc(kind);   // (they are the block's last rows)
    const int slot = lane < w.there - w.nf ? lane : R - 1 - (lane - (w.there - w.nf));   // the row's place here
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    uint2 q[C::rows / 4];
    if (warp < kRowWarps) get_q<R>(P, w, place, q);
    int i = -1;
    if (row.there) {
        int c;
        bool bad;
        const int n = paged_tokens(p, row.b, &c, &bad);
        if (row.t < n) i = p.P + c + row.t;
        // each sequence's counts are checked once
        if (bad && t == 0 && w.it.part == 1 && w.it.chunk == 0 && w.it.rb == 0 && w.it.hk == 0)
            atomicOr(p.status, kStatusPage);
    }
    w.imin = __reduce_min_sync(0xffffffffu, i >= 0 ? i : 0x7fffffff);
    w.imax = __reduce_max_sync(0xffffffffu, i);
    w.any_ord = __ballot_sync(0xffffffffu, i >= 0 && !row.frozen) != 0;
    const bool any_frozen = __ballot_sync(0xffffffffu, i >= 0 && row.frozen) != 0;
    w.g = paged_range(p, w.it, w.imin, w.imax, any_frozen || p.window == 0);
    const int per = p.per_chunk[w.it.part];
    w.e0 = min(w.it.chunk * per, w.g.n);
    w.e1 = min(w.e0 + per, w.g.n);
    if (warp == 0 && lane < R) {
        sh.out_row[slot] = place;
        sh.pos[slot] = i < 0 ? -1 : i - w.off;
        // (rows that see nothing, whose columns of S may hold anything: no score passes their maximum)
        sh.nm[slot] = i < 0 ? -INFINITY : -kNoMax;
        sh.nlim[slot] = (float)-kLeastExp;
        sh.gain[slot] = pow2i(kWeightExp - kLeastExp);
        sh.most[slot] = -INFINITY;
        sh.scale[slot] = 0.f;
        sh.a[slot] = p.a + (size_t)row.h * p.ld + w.off;
        sh.r[slot] = p.r + (size_t)row.h * p.ld + (i < 0 ? 0 : i - w.off);
    }
    if (w.e0 >= w.e1) {   // no keys: nothing but the rows' empty sums
        __syncthreads();
        write_empty(p, w.it, R, sh.out_row, C::threads);
        return;
    }
    // (one setmaxnreg for each warpgroup)
    if (warp < kRowWarps) {
        if constexpr (C::split) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
        asm volatile("barrier.cta.sync 4, %0;" ::"n"(32 * kRowWarps) : "memory");   // the rows' places
        row_warps<R>(P, w, q, sm, sh);
    } else {
        if constexpr (C::split) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kRowWarps) load_warp<C>(P, w, sm, sh);
        else if (warp < kRowWarps + 3) issue_warps<R>(P, w, sm, sh);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kRowWarps + 1) {
        tc_fence_after();
        tmem_dealloc(sh.tmem_base, C::cols);
    }
}

template <int R>
cudaError_t launch_r(const Q8Params& P, unsigned items, cudaStream_t s) {
    constexpr int smem = Cfg<R>::total + 1024;
    static_assert(Cfg<R>::slots <= kMaxSlots, "barriers of the ring");
    const cudaError_t e =
        cudaFuncSetAttribute(paged_q8_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if constexpr (Cfg<R>::split) {
        // A build that launches with fewer registers could never hand the softmax theirs (a property of the
        // compiled kernel, looked up once).
        static std::atomic<int> regs{0};
        if (regs.load() == 0) {
            cudaFuncAttributes fa;
            const cudaError_t f = cudaFuncGetAttributes(&fa, paged_q8_kernel<R>);
            if (f != cudaSuccess) return f;
            regs.store(fa.numRegs);
        }
        if (2 * kRegsRows + kRegsOther > 3 * regs.load()) return cudaErrorInvalidConfiguration;
    }
    return launch_ex(paged_q8_kernel<R>, dim3(items), dim3(Cfg<R>::threads), (size_t)smem, s, true, 1, P);
}

}  // namespace

cudaError_t launch_paged_q8(const PagedArgs& a, int rows, unsigned items, cudaStream_t s) {
    Q8Params P;
    if (!q8_params(&P, a, kTile)) return cudaErrorInvalidValue;
    switch (rows) {
        case 4: return launch_r<4>(P, items, s);
        case 8: return launch_r<8>(P, items, s);
        case 16: return launch_r<16>(P, items, s);
        case 24: return launch_r<24>(P, items, s);
        default: return launch_r<32>(P, items, s);
    }
}

}  // namespace saf
