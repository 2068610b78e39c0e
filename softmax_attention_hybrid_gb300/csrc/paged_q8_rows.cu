// Paged attention over 8-bit caches for blocks of many rows (bf16 q and o): chunks of prompts, and
// a prefix that a batch shares. See paged.h for the split, paged_q8_tc.cu for few rows.
//
// Up to 256 rows of one key/value head, in two groups of M = 128 (a thread per row), meet tiles of
// 128 keys:
//   S = q K^T with K's codes as they lie in the cache (kind::f8f6f4): q, scaled by a power of two so that
//     its largest lies in (224, 448], as hi = e4m3(q) and lo = e4m3(q - hi), two products into one sum.
//     What they leave is at most 2^-10, 2^-17 of the row's largest.
//   O += P V in fp16 (kind::f16). Four warps turn a tile of V into code s_v 2^(7 - V) <= 57344, once for all
//     rows, with s_v <= 2^V the tile's scales (the scale and the product are rounded: 2^-11); the weight is
//     P 2^(7 + V - E) in fp16, at most 2^15, with E the row's own bound of log2(P s_v) so far (off by 2^-12, or 2^-23
//     of the row's largest). A tile whose scales lie further apart than 2^8 gives each key its own V, which its weights
//     then take up one by one: with one V for all, keys with large values, seen or not, took the others' bits.
// The key's scale multiplies the scores. Sums are fp32 in tensor memory, l adds the weights unrounded.
//
// A group's S and P share their columns of tensor memory, so that its S, softmax and P V follow one
// another; the two groups do so in turn. The softmax goes over the tile twice, 32 keys at a time: scaled
// and masked scores back to tensor memory with their maximum, then the weights.
//
// 512 tokens of each of four prompts after up to 8K, 32 heads over 8 of 128, a quarter frozen: 302 us, 472 TFLOP/s (25% of
// a large matrix product's rate; tensor pipe 28% active, issue slots 43%). A tile takes a group about 3 us, the chain of
// S, two passes of the softmax over tensor memory, and P V, with the other group's in between. 64 sequences
// after 32K, all heads of a group in a block: 71 us for the prefix (one read of it takes 10). (289 us for the
// chunk with the largest value scale so far as the unit of all values, which lost the others' bits.)
// Other forms of the same work, in us, beside 290 at that time: tiles of 64 keys with the loops unrolled 369 (the loop leaves the instruction cache)
// and rolled 401, two CTAs of 128 rows 412, two threads to a row 365.
//
// Warps (512 threads, one CTA per SM): 0-7 rows, 8-11 unpack V and hand out the scales, 12 loads K, V and
// scales, 13 and 14 issue a group's MMAs each (13 owns tensor memory), 15 brings the frozen heads' a and r
// of the next tile into shared memory.
// Tensor memory, per group: S, then P (fp16 pairs) in its place | O.
// Shared memory: q's terms, a ring of tiles of K or V in the order in which they are used (K0, K1, V0,
// K2, V1, ...; V0, V1, ... where no row is ordinary), two tiles of V in fp16, the patterns.
#include <string.h>

#include <atomic>

#include "paged_q8.cuh"
#include "pattern_run.h"

namespace saf {
namespace {

using namespace paged_q8;

constexpr int kThreads = 512;
constexpr int kMostOrdered = 256;   // sequences of a batch that are put in order
// Register split (setmaxnreg), within the kRegsLaunch per thread that the launch hands out (checked on the host).
constexpr int kRegsLaunch = 128, kRegsRows = 168, kRegsOther = 80;
static_assert(kRegsRows + kRegsOther <= 2 * kRegsLaunch, "register split too large");
constexpr int TK = kQ8RowsTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // lazy rescale: factor 256
constexpr int kWeightExp = 7;               // a weight of the maximum is 2^7; values of the largest scale are 2^7 codes
constexpr int kEvenRange = 8;               // scales of a tile that share one V: within 2^8
constexpr int kNoExp = -1000;               // no scale but zeros
constexpr int kLeastV = -110, kMostV = 128; // 2^(7 - V) is a float
constexpr int kLeastExp = -112, kMostExp = 130;   // of E: 2^(E - 14) is a float
constexpr int kLeastShift = -60;        // weights of a tile whose values are nothing beside the row's: for the sums' sake
constexpr int kPatFloats = 2560;            // room for the frozen heads' patterns of a tile

// kD: columns of O as the tiles hold them (64, or 128 for 96 and 128).
template <int kD>
struct Cfg {
    static constexpr int tile = TK;
    static constexpr int slots = 4;
    static constexpr int q = 0;                                   // group g, term t at 16384 (2 g + t)
    static constexpr int ring = q + 4 * 128 * 128;
    static constexpr int v16_atom = TK * 128;                     // TK keys x 64 columns
    static constexpr int v16_tile = v16_atom * (kD / 64);
    static constexpr int v16 = ring + slots * TK * 128;
    static constexpr int scales = v16 + 2 * v16_tile;
    static constexpr int pat = scales + slots * TK * 4;
    static constexpr int total = pat + 2 * kPatFloats * 4;
    // tensor-memory columns of a group (S at 0)
    static constexpr uint32_t group = 256, col_o = TK;
    static_assert(col_o + kD <= group, "tensor memory");
};

struct Bars {
    uint64_t full[4], empty[4];
    uint64_t s_full[2], p_ready[2], o_done[2];               // of a group
    uint64_t sc_ready[2], v_ready[2], v_free[2];             // of the tile's parity
    uint64_t pat_full[2], pat_empty[2], mma_idle[2];
    uint64_t first;                                          // group 0 has read its first scores
};

struct Shared {
    Bars bars;
    uint32_t tmem_base;
    int abort_flag, imin, imax, kinds, frozen_warps, lost;
    alignas(16) float ks[2][TK];   // scales of a tile's keys
    alignas(16) float ve[2][TK];   // of an uneven tile: a key's V less the tile's
    int vexp[2], even[2];          // V; whether all keys share it
    int out_row[256], q_row[256];  // the rows' places in o, and in q where they are ordinary; -1: none
    float q_scale[256];            // what a score times its key's scale is multiplied by
    alignas(16) int length[kMostOrdered];
    int sequence;
};

struct RowsWork : Work {
    int groups;       // 1 or 2
    // the frozen heads of the block: group members fz0 .. fz0 + heads - 1, whose patterns the tile's
    // threads read from shared memory (staged) or from a and r themselves
    int fz0, heads;
    bool staged;
    // floats of one staged pattern: a of the tile's keys, and r of the distances imin - (last key) ..
    // imax - (first key), in whole 16-byte lines
    __device__ __forceinline__ int pitch() const { return (2 * TK + (imax - imin) + 9) & ~3; }
    // how far into a line the run of r begins (tiles are a multiple of a line apart)
    __device__ __forceinline__ int shift(const PagedArgs& p, size_t h) const {
        return (int)((((uintptr_t)(p.r + h * p.ld) >> 2) + (uintptr_t)(imin - off - (TK - 1))) & 3);
    }
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two codes of e4m3 (the low 16 bits) as fp16 pairs: exact.
__device__ __forceinline__ uint32_t codes_f16(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}

__device__ __forceinline__ void copy4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// The entries of a run that its lines leave: below them, behind them, or all of it where there is none. (Not inline: the
// chunk of 512 tokens, which has none, takes 305 us with it and 302 without.)
__device__ __noinline__ void copy_ends(float* to, const float* r, int first, int end, int lo, int hi) {
    const int lane = threadIdx.x & 31, c = lane < 8 ? lo + lane : max(end, lo) + lane - 8;
    if (lane < 16 && c <= hi && (lane < 8 ? c < first || first >= end : first < end)) copy4(to + c, r + c);
}

// The pattern warp: a and r of the block's frozen heads for every tile. A row at position i and
// key x need a[x] and r[i - x]; for all rows of a head and TK keys that is a run of r of imax - imin + TK
// entries, copied as whole 16-byte lines (so that an entry lies as far into a line as in r; at most three entries
// of other rows come with it), and one by one where a line is not inside the array. The copies arrive on their
// barrier by themselves.
template <int kD>
__device__ __forceinline__ void pattern_warp(const Q8Params& P, const RowsWork& w, uint8_t* sm, Shared& sh) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    const int lane = threadIdx.x & 31;
    const int pitch = w.pitch();
    const int n = w.e1 - w.e0;
    for (int j = 0; j < n; ++j) {
        const int b = j & 1, x0 = w.slot0(j, TK);
        if (!wait_all(&bars.pat_empty[b], ((j >> 1) & 1) ^ 1u, &sh.abort_flag, p.status)) break;
        float* out = reinterpret_cast<float*>(sm + C::pat) + b * kPatFloats;
        const int r0 = w.imin - w.off - x0 - (TK - 1), r1 = w.imax - w.off - x0;   // (entries of keys past
        const int lo = max(r0, 0), hi = min(r1, p.ld - 1);                         // a row's position are masked)
        uint32_t bytes = 0;
        for (int f = 0; f < w.heads; ++f) {
            const size_t h = p.gheads[w.it.hk * p.G + w.fz0 + f];
            const float* a = p.a + h * p.ld + w.off + x0;
            const float* r = p.r + h * p.ld;
            const int keys = min(TK, p.ld - w.off - x0);
            for (int c = lane; c < keys; c += 32) copy4(out + f * pitch + c, a + c);
            if (hi >= lo) {
                float* to = out + f * pitch + TK + w.shift(p, h) - r0;
                const PatternRun run = pattern_run((uintptr_t)r, (long long)h * p.ld, (long long)(p.H - (int)h) * p.ld, lo, hi);
                const uint32_t line_bytes = run.first < run.end ? 4u * (uint32_t)(run.end - run.first) : 0u;
                if (lane == 0 && line_bytes) bulk_load(to + run.first, r + run.first, line_bytes, &bars.pat_full[b]);
                bytes += line_bytes;
                if (run.first > lo || run.end <= hi) copy_ends(to, r, run.first, run.end, lo, hi);
            }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars.pat_full[b])) : "memory");
        if (lane == 0) mbar_expect_tx(&bars.pat_full[b], bytes);
        __syncwarp();
    }
    // no copy is on its way when the warp leaves
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0)
        for (int j = n < 2 ? 0 : n - 2; j < n; ++j) mbar_wait_bounded(&bars.pat_full[j & 1], (j >> 1) & 1, kWaitLimitNs);
    __syncwarp();
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Warps 8-11: the scales of a tile, then its values as fp16.
template <int kD>
__device__ __forceinline__ void unpack_warps(const Q8Params& P, const RowsWork& w, uint8_t* sm, Shared& sh) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int n = w.e1 - w.e0;
    for (int j = 0; j < n; ++j) {
        const int buf = j & 1, x0 = w.slot0(j, TK);
        // P V of tile j - 2 is done: its scales are read, its values free
        if (!wait_all(&bars.v_free[buf], ((j >> 1) & 1) ^ 1u, abort, p.status)) break;
        if (w.any_ord) {
            const int ld = w.k_load(j), s = ld % C::slots;
            if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) break;
            const float* ks = reinterpret_cast<const float*>(sm + C::scales + s * TK * 4);
            if (warp == 0) *reinterpret_cast<float4*>(&sh.ks[buf][4 * lane]) = *reinterpret_cast<const float4*>(&ks[4 * lane]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.empty[s]);
        }
        const int ld = w.v_load(j), s = ld % C::slots;
        if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) break;
        const float* vs = reinterpret_cast<const float*>(sm + C::scales + s * TK * 4);
        // codes and scales of slots that no row sees may be anything: zeros, for 0 * NaN is none
        const bool lost = *(volatile int*)&sh.lost != 0;
        const bool cut = lost || x0 + TK > w.g.hi || (x0 < w.g.lo && x0 + TK > w.g.sink);
        float v[TK / 32];        // of keys lane, lane + 32, ...
        uint32_t seen[TK / 32];
        float top = 0.f;
        uint32_t low = 0x7f800000u;   // smallest scale of a key that some row sees
#pragma unroll
        for (int k = 0; k < TK / 32; ++k) {
            v[k] = vs[32 * k + lane];
            seen[k] = 0xffffffffu;
            if (cut) {
                const int x = x0 + 32 * k + lane, bx = x0 + (32 * k + lane) / P.box * P.box;
                const bool a = x < w.g.hi && (x >= w.g.lo || x < w.g.sink) && !(lost && paged_page(p, w.it, bx) < 0);
                seen[k] = __ballot_sync(0xffffffffu, a);
                if (!a) v[k] = 0.f;
            }
            top = fmaxf(top, v[k]);
            if ((seen[k] >> lane) & 1u) low = min(low, __float_as_uint(v[k]));
        }
        // (scales are not negative: their bits have their order)
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        low = __reduce_min_sync(0xffffffffu, low);
        auto exponent = [](float x) {   // x < 2^exponent
            const int e = (int)((__float_as_uint(x) >> 23) & 255u) - 126;
            return e < kLeastV ? kLeastV : e > kMostV ? kMostV : e;
        };
        const int vexp = exponent(top);
        const bool even = top == 0.f || exponent(__uint_as_float(low)) >= vexp - kEvenRange;
        if (warp == 0) {   // (each lane has used what it read of the ring before the warp meets and its slot is given back)
            if (!even)   // (a value of scale zero has no part in what is the row's largest)
#pragma unroll
                for (int k = 0; k < TK / 32; ++k)
                    sh.ve[buf][32 * k + lane] = v[k] == 0.f ? (float)kNoExp : (float)(exponent(v[k]) - vexp);
            __syncwarp();
            if (lane == 0) {
                sh.vexp[buf] = top > 0.f ? vexp : kNoExp;
                sh.even[buf] = even;
                mbar_arrive(&bars.sc_ready[buf]);   // (behind the other lanes' scales)
            }
            __syncwarp();
        }
        // A warp takes a quarter of the keys; lane: 16 codes of a key.
        const uint8_t* src = sm + C::ring + s * TK * 128;
        uint8_t* dst = sm + C::v16 + buf * C::v16_tile;
        constexpr int kChunks = kD / 16;            // of 16 codes in a row
        constexpr int kKeys = 32 / kChunks;         // keys at a time
        const int c = lane % kChunks;
        static_assert(TK == 128, "a warp takes the keys whose scales lie in v[warp]");
        float mine = warp == 0 ? v[0] : warp == 1 ? v[1] : warp == 2 ? v[2] : v[3];
        mine *= pow2i(kWeightExp - (even ? vexp : exponent(mine)));
        const uint32_t here = warp == 0 ? seen[0] : warp == 1 ? seen[1] : warp == 2 ? seen[2] : seen[3];
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += kKeys) {
            const int in = k0 + lane / kChunks, key = 32 * warp + in;
            uint4 x = *reinterpret_cast<const uint4*>(src + sw128_offset(key, 16 * c));
            const float sv = __shfl_sync(0xffffffffu, mine, in);
            const uint32_t s2 = pack_f16(sv, sv);
            if (!((here >> in) & 1u)) x = make_uint4(0, 0, 0, 0);
            const uint4 a = make_uint4(hmul2(codes_f16(x.x), s2), hmul2(codes_f16(x.x >> 16), s2),
                                       hmul2(codes_f16(x.y), s2), hmul2(codes_f16(x.y >> 16), s2));
            const uint4 b = make_uint4(hmul2(codes_f16(x.z), s2), hmul2(codes_f16(x.z >> 16), s2),
                                       hmul2(codes_f16(x.w), s2), hmul2(codes_f16(x.w >> 16), s2));
            // 32 bytes of a row of 64 columns; lanes of the second atom write theirs in the other order, to other banks
            uint8_t* row = dst + (c >> 2) * C::v16_atom;
            const uint32_t o0 = sw128_offset(key, 32 * (c & 3)), o1 = sw128_offset(key, 32 * (c & 3) + 16);
            const bool flip = (c >> 2) != 0;
            *reinterpret_cast<uint4*>(row + (flip ? o1 : o0)) = flip ? b : a;
            *reinterpret_cast<uint4*>(row + (flip ? o0 : o1)) = flip ? a : b;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bars.v_ready[buf]);
            mbar_arrive(&bars.empty[s]);
            if (warp < w.groups) mbar_arrive(&bars.empty[s]);   // (a slot's barrier counts the groups' MMAs on K too)
        }
    }
}

// Keys [first, first + 32) of which those below `end` are set.
__device__ __forceinline__ uint32_t below(int end, int first) {
    const int n = end - first;
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// An uneven tile's scores s become (s - m) sc + the key's V less the tile's. Returns the largest of them, and the sum of
// the weights without the V's, times 2^kWeightExp. (Not inline: as a part of the loop it costs the chunk of 512 tokens
// 318 us in place of 301, without a single uneven tile.)
__device__ __noinline__ float2 uneven_scores(uint32_t tmem, float ref, float sc, const float* ve) {
    float cand = -INFINITY, l = 0.f;
    uint32_t sv[8];
#pragma unroll 1
    for (int c0 = 0; c0 < TK; c0 += 8) {
        tmem_ld8(tmem + c0, sv);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float z = (__uint_as_float(sv[c]) - ref) * sc, y = z + ve[c0 + c];
            l += fast_exp2(z + kWeightExp);
            cand = fmaxf(cand, y);
            sv[c] = __float_as_uint(y);
        }
        tmem_st8(tmem + c0, sv);
    }
    tmem_st_wait();
    return make_float2(cand, l);
}

// Warps 0-7 of a group that has rows: thread = row.
template <int kD>
__device__ __forceinline__ void row_warps(const Q8Params& P, const RowsWork& w, const PagedRow& row, uint8_t* sm,
                                          Shared& sh) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const int t = threadIdx.x, g = t >> 7, warp = (t >> 5) & 3, lane = t & 31;
    const uint32_t tmem = sh.tmem_base + g * C::group + ((uint32_t)(warp * 32) << 16);
    const int i = row.i < 0 ? -1 : row.i - w.off;   // my last visible slot of the part
    const bool frozen = row.frozen && i >= 0;
    const float sc = row.frozen ? kLog2e : sh.q_scale[t];
    const bool any_frozen = __any_sync(0xffffffffu, frozen), any_scaled = __any_sync(0xffffffffu, i >= 0 && !row.frozen);
    const float* ra = p.a + (size_t)row.h * p.ld + w.off;
    const float* rr = p.r + (size_t)row.h * p.ld;
    // my staged pattern: a of the tile's keys, and r from the far end on (entry k - c for key c)
    const float* pat_a = reinterpret_cast<const float*>(sm + C::pat) + (frozen ? row.gi - w.fz0 : 0) * w.pitch();
    const float* pat_r = pat_a + TK + (TK - 1) + (frozen ? row.i - w.imin + w.shift(p, row.h) : 0);
    float m = -INFINITY, l = 0.f;   // (m: before the factor sc; l: times 2^kWeightExp)
    int lim = kLeastExp;            // E
    float largest = -INFINITY;      // log2 of the largest product of a weight and its value's scale
    bool ok = true;

    const int tiles = w.e1 - w.e0;
    int n = 0;
    for (; n < tiles; ++n) {
        const int x0 = w.slot0(n, TK), buf = n & 1;
        if (!(ok = wait_all(&bars.sc_ready[buf], (n >> 1) & 1, abort, p.status))) break;
        if (any_frozen && w.staged && !(ok = wait_all(&bars.pat_full[buf], (n >> 1) & 1, abort, p.status))) break;
        // S is there; and P V of the previous tile, after which it was issued, is done: O is stable
        if (w.any_ord) ok = wait_all(&bars.s_full[g], n & 1, abort, p.status);
        else if (n > 0) ok = wait_all(&bars.o_done[g], (n - 1) & 1, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const bool lost = *(volatile int*)&sh.lost != 0;
        // masks, in tiles that some row does not see whole
        const bool cut = lost || x0 + TK > w.g.hi || x0 + TK - 1 > w.imin - w.off ||
                         (p.window > 0 && x0 <= w.imax - w.off - p.window);
        float ma = -INFINITY, mb = -INFINITY;
        uint32_t sv[32];
#pragma unroll 1
        for (int c0 = 0; c0 < TK; c0 += 32) {
            if (any_scaled) {
                tmem_ld32(tmem + c0, sv);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float4 ks = *reinterpret_cast<const float4*>(&sh.ks[buf][c0 + c]);
                    const float2 a = fmul2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), make_float2(ks.x, ks.y));
                    const float2 b = fmul2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), make_float2(ks.z, ks.w));
                    sv[c] = __float_as_uint(a.x);
                    sv[c + 1] = __float_as_uint(a.y);
                    sv[c + 2] = __float_as_uint(b.x);
                    sv[c + 3] = __float_as_uint(b.y);
                }
            } else {   // (rows without a token: anything finite)
#pragma unroll
                for (int c = 0; c < 32; ++c) sv[c] = 0u;
            }
            if (any_frozen) {   // the fixed pattern's logits (Eq. 3)
                if (w.staged) {
                    const float* qa = pat_a + buf * kPatFloats + c0;
                    const float* qr = pat_r + buf * kPatFloats - c0;
                    if (frozen) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 a4 = *reinterpret_cast<const float4*>(qa + c);
                            sv[c] = __float_as_uint(a4.x + qr[-c]);
                            sv[c + 1] = __float_as_uint(a4.y + qr[-c - 1]);
                            sv[c + 2] = __float_as_uint(a4.z + qr[-c - 2]);
                            sv[c + 3] = __float_as_uint(a4.w + qr[-c - 3]);
                        }
                    }
                } else if (frozen) {   // (keys past my own position are masked below)
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const int y = min(x0 + c0 + c, i);
                        sv[c] = __float_as_uint(__ldg(ra + y) + __ldg(rr + i - y));
                    }
                }
            }
            if (cut) {
                const int first = x0 + c0, last = min(i, w.g.hi - 1);   // (a prefix ends before i)
                uint32_t vis = below(last + 1, first);
                if (!row.frozen && p.window > 0) vis &= ~below(i - p.window + 1, first) | below(p.sinks - w.off, first);
                if (lost)
                    for (int bx = first & ~(P.box - 1); bx < first + 32; bx += P.box)
                        if (box_seen(w.g, bx, P.box) && paged_page(p, w.it, bx) < 0)
                            vis &= ~(below(bx + P.box, first) & ~below(bx, first));
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (!((vis >> c) & 1u)) sv[c] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
                ma = fmax3(ma, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
                mb = fmax3(mb, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
            }
            tmem_st32(tmem + c0, sv);
        }
        if (any_frozen && w.staged) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.pat_empty[buf]);
        }
        // (a score that the factor makes -infinity is none)
        const float most = fmaxf(ma, mb), m_new = most * sc > -INFINITY ? fmaxf(m, most) : m;
        float rise = 0.f;   // of the maximum, in powers of two
        if ((m_new - m) * sc > kRescaleThreshold) {
            rise = (m_new - m) * sc;
            l *= fast_exp2(-rise);
            m = m_new;
        }
        const float ref = m == -INFINITY ? 0.f : m;   // a row that has seen no key yet: weights 2^-inf = 0
        const int vexp = sh.vexp[buf];   // (the same for every row)
        const bool even = sh.even[buf] != 0;
        tmem_st_wait();
        if (n == 0 && t == 0) mbar_arrive(&bars.first);
        // The largest product of a weight and its value's scale, as a power of two: in an even tile at most its
        // largest weight with its V.
        float cand = (most - ref) * sc, uneven_l = 0.f;
        if (!even) {
            const float2 x = uneven_scores(tmem, ref, sc, sh.ve[buf]);
            cand = x.x;
            uneven_l = x.y;
        }
        cand = vexp == kNoExp ? -INFINITY : cand + (float)vexp;
        float f = 1.f;   // of O, whose unit is 2^(m + E - 14)
        const bool need = rise > 0.f || cand > (float)lim + kRescaleThreshold;
        if (need) {
            largest = fmaxf(largest - rise, cand);
            const int e = (int)fminf(fmaxf(ceilf(largest), (float)kLeastExp), (float)kMostExp);
            // whole powers apart from the rest: the sum of both would round the rest
            const float whole = rintf(rise), n2 = (float)(lim - e) - whole;
            f = n2 < -149.f ? 0.f : exp2f(whole - rise) * pow2i((int)n2);
            lim = e;
        }
        if (n > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
            for (int q = 0; q < kD; q += 32) {
                tmem_ld32(tmem + C::col_o + q, sv);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; ++c) sv[c] = __float_as_uint(__uint_as_float(sv[c]) * f);
                tmem_st32(tmem + C::col_o + q, sv);
            }
        }
        // The maximum is taken off before the factor: sc s - sc m in one step would leave the rounding of sc m,
        // which is no longer small beside scores of 2^24 and more.
        const float take = even ? -ref : 0.f, times = even ? sc : 1.f;
        // from a weight to its product with the tile's V; the weights of the sum are those of the product, in other units
        const int up = vexp == kNoExp ? 0 : max(vexp - lim, kLeastShift);
        const float2 sc2 = make_float2(times, times), nm2 = make_float2(take, take);
        const float2 up2 = make_float2((float)(up + kWeightExp), (float)(up + kWeightExp));
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c0 = 0; c0 < TK; c0 += 32) {
            tmem_ld32(tmem + c0, sv);
            tmem_ld_wait();
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float2 y = fadd2(make_float2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), nm2);
                const float2 x = ffma2(y, sc2, up2);
                const float2 ex = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                if (c & 1) acc1 = fadd2(acc1, ex);
                else acc0 = fadd2(acc0, ex);
                pk[c] = pack_f16(ex.x, ex.y);
            }
            tmem_st16(tmem + c0 / 2, pk);   // (in the place of scores that are read)
        }
        // (2^-up, and 0 below what a float holds)
        l += even ? ((acc0.x + acc1.x) + (acc0.y + acc1.y)) * __int_as_float(max(127 - up, 0) << 23) : uneven_l;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_ready[g]);
    }
    ok = ok && mbar_wait_warp(&bars.o_done[g], (n - 1) & 1, abort, p.status, kStatusTimeout);
    tc_fence_after();
    if (!ok) return;
    // my row
    l *= pow2i(-kWeightExp);
    const bool sees = row.i >= 0 && l != 0.f;   // (a NaN sum is one)
    m *= sc;
    const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
    const float back = pow2i(lim - 2 * kWeightExp);
    const float mul = p.nsplit > 1 ? back : back * (1.f / l);
    // 32 columns of the warp's rows at a time through its part of the group's q, which is no longer read, so that
    // whole lines are written: 8 lanes to a row
    float* stage = reinterpret_cast<float*>(sm + C::q + (t >> 5) * 8192);
    const int sub = lane >> 3, c4 = lane & 7;
#pragma unroll 1
    for (int q = 0; q < p.d; q += 32) {
        uint32_t ov[32];
        tmem_ld32(tmem + C::col_o + q, ov);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 8; ++c)   // (16-byte chunks, turned by the row)
            *reinterpret_cast<float4*>(stage + lane * 32 + 4 * (c ^ (lane & 7))) =
                sees ? make_float4(__uint_as_float(ov[4 * c]) * mul, __uint_as_float(ov[4 * c + 1]) * mul,
                                   __uint_as_float(ov[4 * c + 2]) * mul, __uint_as_float(ov[4 * c + 3]) * mul)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const int at = sh.out_row[(t & ~31) + k + sub];
            const float4 y = *reinterpret_cast<const float4*>(stage + (k + sub) * 32 + 4 * (c4 ^ ((k + sub) & 7)));
            if (at < 0) continue;
            if (p.nsplit > 1)
                *reinterpret_cast<float4*>(p.po + ((size_t)at * p.nsplit + split) * p.d + q + 4 * c4) = y;
            else
                *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o + (size_t)at * p.d + q + 4 * c4) =
                    make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        }
        __syncwarp();
    }
    if (!row.there) return;
    const size_t at = (size_t)sh.out_row[t];
    if (p.nsplit > 1) p.ml[at * p.nsplit + split] = sees ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
    else p.lse[at] = sees ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Warps 13 and 14: a group's MMAs. S of tile j + 1 takes the place of P of tile j, so it waits for its P V.
template <int kD>
__device__ __forceinline__ void issue_warp(const Q8Params& P, const RowsWork& w, int g, uint8_t* sm, Shared& sh) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    constexpr uint32_t id_s = idesc_e4m3(128, TK, 0, 0), id_o = idesc_f16(128, kD, 0, 1);
    const uint64_t d_q = sdesc_sw128(smem_u32(sm + C::q) + g * 2 * 16384, 16, 1024);   // K-major, as K
    const uint64_t d_ring = sdesc_sw128(smem_u32(sm + C::ring), 16, 1024);
    const uint64_t d_v16 = sdesc_sw128(smem_u32(sm + C::v16), C::v16_atom, 1024);      // MN-major
    const uint32_t tmem = sh.tmem_base + g * C::group;
    const int n = w.e1 - w.e0;
    auto scores = [&](int j) -> bool {
        const int ld = w.k_load(j), s = ld % C::slots;
        if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) return false;
        if (j > 0 && !wait_all(&bars.o_done[g], (j - 1) & 1, abort, p.status)) return false;
        tc_fence_after();
        const uint64_t d_k = sdesc_advance(d_ring, s * TK * 128);
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {   // hi, then lo
            const int term = k / (kD / 32), at = k % (kD / 32);
            mma_ss_e4m3_warp(tmem, sdesc_advance(d_q, term * 16384 + 32 * at), sdesc_advance(d_k, 32 * at), id_s, k > 0);
        }
        mma_commit_warp(&bars.s_full[g]);
        mma_commit_warp(&bars.empty[s]);
        return true;
    };
    // The second group begins half a tile later: in step, both would wait for their MMAs at the same time.
    if (g == 1) wait_all(&bars.first, 0, abort, p.status);
    bool ok = !w.any_ord || scores(0);
    for (int j = 0; j < n && ok; ++j) {
        if (!wait_all(&bars.v_ready[j & 1], (j >> 1) & 1, abort, p.status)) break;
        if (!wait_all(&bars.p_ready[g], j & 1, abort, p.status)) break;
        tc_fence_after();
        const uint64_t d_v = sdesc_advance(d_v16, (j & 1) * C::v16_tile);
#pragma unroll
        for (int k = 0; k < TK / 16; ++k)
            mma_ts_warp(tmem + C::col_o, tmem + 8 * k, sdesc_advance(d_v, k * 2048), id_o, (j > 0 || k > 0) ? 1u : 0u);
        mma_commit_warp(&bars.o_done[g]);
        mma_commit_warp(&bars.v_free[j & 1]);
        if (w.any_ord && j + 1 < n) ok = scores(j + 1);
    }
    // every MMA issued here is done before tensor memory is freed
    mma_commit_warp(&bars.mma_idle[g]);
    if ((threadIdx.x & 31) == 0) mbar_wait_bounded(&bars.mma_idle[g], 0, kWaitLimitNs);
    __syncwarp();
}

// Every warp but the loading one: q's terms and tensor memory are there.
__device__ __forceinline__ void set_up_done() {
    tc_fence_before();
    asm volatile("bar.sync 2, 480;" ::: "memory");
    tc_fence_after();
}

// Rows of q: 16 lanes of 8 elements to a row, a warp's 32 rows in four batches, of which the first is on its way
// before anything about the sequences is known.
struct RowsOfQ {
    uint4 x[4];
    __device__ __forceinline__ static int row(int batch, int k) {
        return 32 * (int)(threadIdx.x >> 5) + 8 * batch + 2 * k + (int)((threadIdx.x >> 4) & 1);
    }
    __device__ __forceinline__ void get(const PagedArgs& p, const Shared& sh, int batch) {
        const int c = threadIdx.x & 15;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = sh.q_row[row(batch, k)];
            x[k] = at >= 0 && 8 * c < p.d
                       ? __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.q + (size_t)at * p.d) + c)
                       : make_uint4(0, 0, 0, 0);
        }
    }
    // the rows' terms and factors
    template <typename C, int kCols>
    __device__ __forceinline__ void put(const PagedArgs& p, uint8_t* sm, Shared& sh, int batch) const {
        const int c = threadIdx.x & 15;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            // the row's largest magnitude as bits: above 0x7f7f it holds an infinity or a NaN
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __vmaxu2(top, v[e] & 0x7fff7fffu);
#pragma unroll
            for (int o = 8; o; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = max(top & 0xffffu, top >> 16);
            const bool bad = top >= 0x7f80u;
            // 448 = 1.75 x 2^8
            int e = 8 - ((int)(top >> 7) - 127) - ((top & 0x7fu) > 0x60u);
            e = bad ? 0 : e < -120 ? -120 : e > 120 ? 120 : e;
            const float f = pow2i(e);
            uint32_t h[4], l[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float y0 = __uint_as_float(v[b] << 16) * f, y1 = __uint_as_float(v[b] & 0xffff0000u) * f;
                h[b] = pack_e4m3(y0, y1);
                const float2 z = unpack_e4m3(h[b]);
                l[b] = pack_e4m3(y0 - z.x, y1 - z.y);
            }
            uint2 hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16), lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
            if (bad) hi = lo = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);   // (saturation would hide an infinity)
            const int r = row(batch, k);
            uint8_t* q = sm + C::q + (r >> 7) * 2 * 16384;
            if (8 * c < kCols) {   // (zeros behind the row's end, as TMA leaves behind K's)
                *reinterpret_cast<uint2*>(q + sw128_offset(r & 127, 8 * c)) = hi;
                *reinterpret_cast<uint2*>(q + 16384 + sw128_offset(r & 127, 8 * c)) = lo;
            }
            if (c == 0) sh.q_scale[r] = p.scale_log2 * pow2i(-e);
        }
    }
};

// Items are as long as their sequences, a few to an SM: the longest sequences begin, so that the last items to
// run are the shortest. (512 tokens of four prompts, one item to a block of rows: 342 us in the batch's order.)
__device__ __forceinline__ void longest_first(const PagedArgs& p, PagedItem* it, Shared& sh) {
    const int t = threadIdx.x;
    if (t < kMostOrdered) {
        int c = 0, n = 0;
        bool bad;
        if (t < p.B) n = paged_tokens(p, t, &c, &bad);
        sh.length[t] = t >= p.B ? -1 : n > 0 ? c + n : 0;
    }
    __syncthreads();
    if (t < p.B) {
        const int mine = sh.length[t];
        int before = 0;   // sequences that begin earlier
        for (int u = 0; u < p.B; u += 4) {
            const int4 x = *reinterpret_cast<const int4*>(&sh.length[u]);
            before += (x.x > mine || (x.x == mine && u < t)) + (x.y > mine || (x.y == mine && u + 1 < t)) +
                      (x.z > mine || (x.z == mine && u + 2 < t)) + (x.w > mine || (x.w == mine && u + 3 < t));
        }
        if (before == it->b) sh.sequence = t;
    }
    __syncthreads();
    it->b = sh.sequence;
}

template <int kD>
__global__ void __launch_bounds__(kThreads, 1) paged_q8_rows_kernel(const __grid_constant__ Q8Params P) {
    using C = Cfg<kD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Shared sh;
    const PagedArgs& p = P.a;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    Bars& bars = sh.bars;
    RowsWork w;
    w.it = paged_item(p, blockIdx.x);
    const PagedBlock block = paged_block(p, w.it);
    w.there = block.there;
    w.groups = block.there > 128 ? 2 : 1;
    if (warp == 0) {
        if (lane == 0) {
            sh.abort_flag = 0;
            sh.imin = 0x7fffffff;
            sh.imax = -1;
            sh.kinds = sh.frozen_warps = sh.lost = 0;
        }
        if (lane == 31) mbar_init(&bars.first, 1);
        if (lane < C::slots) {
            mbar_init(&bars.full[lane], 1);
            mbar_init(&bars.empty[lane], 4 + w.groups);   // K: the groups' MMAs and the four warps that read its scales
        } else if (lane < C::slots + 2) {
            const int i = lane - C::slots;
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_ready[i], 4);
            mbar_init(&bars.o_done[i], 1);
            mbar_init(&bars.sc_ready[i], 1);
            mbar_init(&bars.v_ready[i], 4);
            mbar_init(&bars.v_free[i], w.groups);
            mbar_init(&bars.pat_full[i], 33);   // the pattern warp's lanes, and its count of bytes
            mbar_init(&bars.mma_idle[i], 1);
        }
        fence_mbar_init();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    if (w.it.part && p.B > 1 && p.B <= kMostOrdered) longest_first(p, &w.it, sh);
    PagedRow row;
    if (t < 256) {
        row = paged_place(p, w.it, block, t);
        sh.out_row[t] = row.there ? (int)paged_out_row(p, row) : -1;
        sh.q_row[t] = row.there && !row.frozen ? sh.out_row[t] : -1;
    }
    __syncthreads();
    RowsOfQ q;
    if (t < 256) {
        if (p.q) q.get(p, sh, 0);
        if (row.there) {
            int c;
            bool bad;
            const int n = paged_tokens(p, row.b, &c, &bad);
            if (row.t < n) row.i = p.P + c + row.t;
        }
        int lo = row.i >= 0 ? row.i : 0x7fffffff, hi = row.i;
        const int kinds = row.i < 0 ? 0 : row.frozen ? 2 : 1;
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        const int k = __reduce_or_sync(0xffffffffu, (unsigned)kinds);
        if (lane == 0 && k) {
            atomicMin(&sh.imin, lo);
            atomicMax(&sh.imax, hi);
            atomicOr(&sh.kinds, k);
            if (k & 2) atomicAdd(&sh.frozen_warps, 1);
        }
    } else if (t == 256 && w.it.part == 1 && w.it.chunk == 0 && w.it.rb == 0 && w.it.hk == 0) {
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
    w.g = paged_range(p, w.it, w.imin, w.imax, (sh.kinds & 2) != 0 || p.window == 0);
    const int per = p.per_chunk[w.it.part];
    w.e0 = min(w.it.chunk * per, w.g.n);
    w.e1 = min(w.e0 + per, w.g.n);
    if (w.e0 >= w.e1) {   // no keys: nothing but the rows' empty sums
        if (t < 256 && row.there) {
            const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
            const size_t at = (size_t)sh.out_row[t];
            if (p.nsplit > 1) {
                p.ml[at * p.nsplit + split] = make_float2(-INFINITY, 0.f);
            } else {
                for (int c = 0; c < p.d; c += 8) *reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + at * p.d + c) = make_uint4(0, 0, 0, 0);
                p.lse[at] = -INFINITY;
            }
        }
        return;
    }
    // the block's frozen heads: of its members of the group those from gord on
    w.fz0 = max(block.first / block.per_head, (int)p.gord[w.it.hk]);
    w.heads = (block.first + w.there - 1) / block.per_head - w.fz0 + 1;
    w.staged = (long long)w.heads * ((long long)w.imax - w.imin + 2 * TK + 9) <= kPatFloats;

    // one setmaxnreg for each warpgroup
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
        if (w.any_ord) {
            RowsOfQ next;
#pragma unroll 1
            for (int batch = 0; batch < 4; batch += 2) {
                next.get(p, sh, batch + 1);
                q.put<C, kD>(p, sm, sh, batch);
                if (batch == 0) q.get(p, sh, 2);
                next.put<C, kD>(p, sm, sh, batch + 1);
            }
            fence_proxy_async_smem();
        }
        if (t == 0 && sh.frozen_warps > 0) {
            mbar_init(&bars.pat_empty[0], sh.frozen_warps);
            mbar_init(&bars.pat_empty[1], sh.frozen_warps);
            fence_mbar_init();
        }
        set_up_done();
        if ((t >> 7) < w.groups) row_warps<kD>(P, w, row, sm, sh);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        set_up_done();
        unpack_warps<kD>(P, w, sm, sh);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 12) {   // K and V need nothing but the range of keys
            load_warp<C>(P, w, sm, sh);
        } else {
            if (warp == 13) {
                tmem_alloc(&sh.tmem_base, 512);
                tmem_relinquish();
            }
            set_up_done();
            if (warp < 15) {
                if (warp - 13 < w.groups) issue_warp<kD>(P, w, warp - 13, sm, sh);
            } else if (sh.frozen_warps > 0 && w.staged) {
                pattern_warp<kD>(P, w, sm, sh);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(sh.tmem_base, 512);
    }
}

template <int kD>
cudaError_t launch_d(const Q8Params& P, unsigned items, cudaStream_t s) {
    constexpr int smem = Cfg<kD>::total + 1024;
    cudaError_t e = cudaFuncSetAttribute(paged_q8_rows_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // A build that launches with fewer registers could never hand the row warps theirs (a
    // property of the compiled kernel, looked up once).
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, paged_q8_rows_kernel<kD>);
        if (e != cudaSuccess) return e;
        regs.store(fa.numRegs);
    }
    if (kRegsRows + kRegsOther > 2 * regs.load()) return cudaErrorInvalidConfiguration;
    return launch_ex(paged_q8_rows_kernel<kD>, dim3(items), dim3(kThreads), (size_t)smem, s, true, 1, P);
}

}  // namespace

cudaError_t launch_paged_q8_rows(const PagedArgs& a, unsigned items, cudaStream_t s) {
    Q8Params P;
    if (!q8_params(&P, a, TK)) return cudaErrorInvalidValue;
    return a.d == 64 ? launch_d<64>(P, items, s) : launch_d<128>(P, items, s);
}

}  // namespace saf
