// Paged attention over 8-bit caches for blocks of many rows (bf16 q and o): chunks of prompts, and
// a prefix that a batch shares. See paged.h for the split, paged_q8_tc.cu for few rows.
//
// Up to 256 rows of one key/value head, in two groups of M = 128 (a thread per row), meet tiles of
// 64 keys:
//   S = q K^T with K's codes as they lie in the cache (kind::f8f6f4): q, scaled by a power of two so that
//     its largest lies in (224, 448], as hi = e4m3(q) and lo = e4m3(q - hi), two products into one sum.
//     What they leave is at most 2^-10, 2^-17 of the row's largest.
//   O += P V in fp16 (kind::f16): a code of e4m3 is an fp16 number, exactly; four warps unpack the tile of V
//     once for all rows. The weight takes its value's scale, P_j s_v[j] 2^(7 - V) <= 2^15 with s_v <= 2^V
//     the scales so far, and is rounded to fp16: off by 2^-11, or by 2^-32 of a weight at the maximum.
// The key's scale multiplies the scores. Sums are fp32 in tensor memory, l adds the weights unrounded.
//
// Bound by exponentials: 256 x 64 of a tile take 1024 cycles of an SM, its MMAs 512. (256 rows to
// a CTA because 128 would read each tile twice as often from L2: 32 bytes a cycle and SM.)
//
// Warps (512 threads, one CTA per SM): 0-7 rows, 8-11 unpack V and hand out the scales, 12 loads K, V and
// scales, 13 owns tensor memory and issues S, 14 issues P V, 15 brings the frozen heads' a and r
// of the next tile into shared memory.
// Tensor memory, per group: S (64 columns) | P (32, fp16 pairs) | O.
// Shared memory: q's terms, a ring of tiles of K or V in the order in which they are used (K0, K1, V0,
// K2, V1, ...; V0, V1, ... where no row is ordinary), two tiles of V in fp16, the patterns.
#include <string.h>

#include <atomic>

#include "paged_q8.cuh"

namespace saf {
namespace {

using namespace paged_q8;

constexpr int kThreads = 512;
// Register split (setmaxnreg), within the kRegsLaunch per thread that the launch hands out (checked on the host).
constexpr int kRegsLaunch = 128, kRegsRows = 168, kRegsOther = 80;
static_assert(kRegsRows + kRegsOther <= 2 * kRegsLaunch, "register split too large");
constexpr int TK = kQ8RowsTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // lazy rescale: factor 256
constexpr int kWeightExp = 7;               // a weight of the maximum is 2^7, before the value's scale
constexpr int kPatFloats = 2048;            // room for the frozen heads' patterns of a tile

// kD: columns of O as the tiles hold them (64, or 128 for 96 and 128).
template <int kD>
struct Cfg {
    static constexpr int tile = TK;
    static constexpr int slots = 8;
    static constexpr int q = 0;                                   // group g, term t at 16384 (2 g + t)
    static constexpr int ring = q + 4 * 128 * 128;
    static constexpr int v16_atom = TK * 128;                     // TK keys x 64 columns
    static constexpr int v16_tile = v16_atom * (kD / 64);
    static constexpr int v16 = ring + slots * TK * 128;
    static constexpr int scales = v16 + 2 * v16_tile;
    static constexpr int pat = scales + slots * TK * 4;
    static constexpr int total = pat + 2 * kPatFloats * 4;
    // tensor-memory columns of a group (S at 0)
    static constexpr uint32_t group = 256, col_p = TK, col_o = 128;
    static_assert(col_p + TK / 2 <= col_o && col_o + kD <= group, "tensor memory");
};

struct Bars {
    uint64_t full[8], empty[8];
    uint64_t s_full[2], s_empty[2], p_ready[2], o_done[2];   // of a group
    uint64_t sc_ready[2], v_ready[2], v_free[2];             // of the tile's parity
    uint64_t pat_full[2], pat_empty[2], mma_idle[2];
};

struct Shared {
    Bars bars;
    uint32_t tmem_base;
    int abort_flag, imin, imax, kinds, frozen_warps, lost;
    alignas(16) float ks[2][TK];   // scales of a tile's keys
    alignas(16) float vs[2][TK];   // of its values, times 2^(7 - V); 0 where no row sees the key
    int vexp[2];                   // V
};

struct RowsWork : Work {
    int groups;       // 1 or 2
    // the frozen heads of the block: group members fz0 .. fz0 + nf - 1, whose patterns the tile's
    // threads read from shared memory (staged) or from a and r themselves
    int fz0, nf;
    bool staged;
    // floats of one staged pattern: a of the tile's keys, and r of the distances imin - (last key) ..
    // imax - (first key), rounded up to whole 16 bytes
    __device__ __forceinline__ int pitch() const { return (2 * TK + (imax - imin) + 3) & ~3; }
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

// The pattern warp: a and r of the block's frozen heads for every tile. A row at position i and
// key x need a[x] and r[i - x]; for all rows of a head and TK keys that is a run of r of
// imax - imin + TK entries, read here in whole lines.
template <int kD>
__device__ __forceinline__ void pattern_warp(const Q8Params& P, const RowsWork& w, uint8_t* sm, Shared& sh) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const int lane = threadIdx.x & 31;
    const int band = w.imax - w.imin + TK, pitch = w.pitch();
    const uint32_t pat = smem_u32(sm + C::pat);
    auto copy = [&](uint32_t dst, const float* src) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
    };
    const int n = w.e1 - w.e0;
    for (int j = 0; j <= n; ++j) {
        if (j < n) {   // tile j's copies are on their way while the rows work on tile j - 1
            const int b = j & 1, x0 = w.slot0(j, TK);
            if (!wait_all(&bars.pat_empty[b], ((j >> 1) & 1) ^ 1u, abort, p.status)) break;
            for (int f = 0; f < w.nf; ++f) {
                const size_t h = p.gheads[w.it.hk * p.G + w.fz0 + f];
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

// Warps 8-11: the scales of a tile, then its values as fp16.
template <int kD>
__device__ __forceinline__ void unpack_warps(const Q8Params& P, const RowsWork& w, uint8_t* sm, Shared& sh) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int n = w.e1 - w.e0;
    float vtop = 0.f;   // 2^V, 0: no value seen yet
    int vexp = 0;
    for (int j = 0; j < n; ++j) {
        const int buf = j & 1, x0 = w.slot0(j, TK);
        // P V of tile j - 2 is done: its scales are read, its values free
        if (!wait_all(&bars.v_free[buf], ((j >> 1) & 1) ^ 1u, abort, p.status)) break;
        if (w.any_ord) {
            const int ld = w.k_load(j), s = ld % C::slots;
            if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) break;
            const float* ks = reinterpret_cast<const float*>(sm + C::scales + s * TK * 4);
            if (warp == 0) *reinterpret_cast<float2*>(&sh.ks[buf][2 * lane]) = *reinterpret_cast<const float2*>(&ks[2 * lane]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.empty[s]);
        }
        const int ld = w.v_load(j), s = ld % C::slots;
        if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) break;
        float2 vs = *reinterpret_cast<const float2*>(sm + C::scales + s * TK * 4 + 8 * lane);
        // codes and scales of slots that no row sees may be anything: zeros, for 0 * NaN is none
        const bool lost = *(volatile int*)&sh.lost != 0;
        uint32_t seen0 = 0xffffffffu, seen1 = 0xffffffffu;   // keys 2 lane, 2 lane + 1
        const bool cut = lost || x0 + TK > w.g.hi || (x0 < w.g.lo && x0 + TK > w.g.sink);
        if (cut) {
            auto seen = [&](int k) {
                const int x = x0 + k, bx = x0 + k / P.box * P.box;
                return x < w.g.hi && (x >= w.g.lo || x < w.g.sink) && !(lost && paged_page(p, w.it, bx) < 0);
            };
            const bool a = seen(2 * lane), b = seen(2 * lane + 1);
            seen0 = __ballot_sync(0xffffffffu, a);
            seen1 = __ballot_sync(0xffffffffu, b);
            if (!a) vs.x = 0.f;
            if (!b) vs.y = 0.f;
        }
        // (scales are not negative: their bits have their order)
        const float vmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vs.x, vs.y))));
        if (vmax > vtop) {
            int ex = (int)((__float_as_uint(vmax) >> 23) & 255u) - 126;   // vmax < 2^ex
            vexp = ex < -110 ? -110 : ex > 127 ? 127 : ex;
            vtop = pow2i(vexp);
        }
        if (warp == 0) {
            const float f = pow2i(kWeightExp - vexp);
            *reinterpret_cast<float2*>(&sh.vs[buf][2 * lane]) = make_float2(vs.x * f, vs.y * f);
            if (lane == 0) sh.vexp[buf] = vtop > 0.f ? vexp : -1000;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.sc_ready[buf]);
        }
        // A warp takes 16 keys, 4 at a time; lane: 16 codes of a key.
        const uint8_t* src = sm + C::ring + s * TK * 128;
        uint8_t* dst = sm + C::v16 + buf * C::v16_tile;
        constexpr int kChunks = kD / 16;            // of 16 codes in a row
        constexpr int kKeys = 32 / kChunks;         // keys at a time
        const int c = lane % kChunks;
#pragma unroll
        for (int k0 = 0; k0 < 16; k0 += kKeys) {
            const int key = 16 * warp + k0 + lane / kChunks;
            uint4 x = *reinterpret_cast<const uint4*>(src + sw128_offset(key, 16 * c));
            if (cut && !(((key & 1 ? seen1 : seen0) >> (key >> 1)) & 1u)) x = make_uint4(0, 0, 0, 0);
            const uint4 a = make_uint4(codes_f16(x.x), codes_f16(x.x >> 16), codes_f16(x.y), codes_f16(x.y >> 16));
            const uint4 b = make_uint4(codes_f16(x.z), codes_f16(x.z >> 16), codes_f16(x.w), codes_f16(x.w >> 16));
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
            if (warp == 0) mbar_arrive(&bars.empty[s]);   // (a slot's barrier counts the MMAs of K too)
        }
    }
}

// Warps 0-7 of a group that has rows: thread = row.
template <int kD>
__device__ __forceinline__ void row_warps(const Q8Params& P, const RowsWork& w, const PagedRow& row, float qscale,
                                          uint8_t* sm, Shared& sh) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    Bars& bars = sh.bars;
    volatile int* abort = &sh.abort_flag;
    const int t = threadIdx.x, g = t >> 7, warp = (t >> 5) & 3, lane = t & 31;
    const uint32_t tmem = sh.tmem_base + g * C::group + ((uint32_t)(warp * 32) << 16);
    const int box_log2 = __ffs(P.box) - 1;
    const int i = row.i < 0 ? -1 : row.i - w.off;   // my last visible slot of the part
    const bool frozen = row.frozen && i >= 0;
    const float sc = row.frozen ? kLog2e : qscale;
    const bool any_frozen = __any_sync(0xffffffffu, frozen), any_scaled = __any_sync(0xffffffffu, i >= 0 && !row.frozen);
    const float* ra = p.a + (size_t)row.h * p.ld + w.off;
    const float* rr = p.r + (size_t)row.h * p.ld;
    // my staged pattern: a of the tile's keys, and r from the far end on (entry k - c for key c)
    const float* pat_a = reinterpret_cast<const float*>(sm + C::pat) + (frozen ? row.gi - w.fz0 : 0) * w.pitch();
    const float* pat_r = pat_a + TK + (TK - 1) + (frozen ? row.i - w.imin : 0);
    float m = -INFINITY, l = 0.f;
    int vexp = -1000;
    bool ok = true;

    const int tiles = w.e1 - w.e0;
    int n = 0;
    for (; n < tiles; ++n) {
        const int x0 = w.slot0(n, TK), buf = n & 1;
        uint32_t sv[TK];
        if (w.any_ord) {
            if (!(ok = mbar_wait(&bars.s_full[g], n & 1, abort, p.status, kStatusTimeout))) break;
            tc_fence_after();
            tmem_ld32(tmem, sv);
            tmem_ld32(tmem + 32, sv + 32);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.s_empty[g]);
        }
        if (!(ok = mbar_wait(&bars.sc_ready[buf], (n >> 1) & 1, abort, p.status, kStatusTimeout))) break;
        if (w.any_ord && any_scaled) {
#pragma unroll
            for (int c = 0; c < TK; c += 4) {
                const float4 ks = *reinterpret_cast<const float4*>(&sh.ks[buf][c]);
                const float2 a = fmul2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), make_float2(ks.x, ks.y));
                const float2 b = fmul2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), make_float2(ks.z, ks.w));
                sv[c] = __float_as_uint(a.x);
                sv[c + 1] = __float_as_uint(a.y);
                sv[c + 2] = __float_as_uint(b.x);
                sv[c + 3] = __float_as_uint(b.y);
            }
        }
        if (any_frozen) {   // the fixed pattern's logits (Eq. 3)
            if (w.staged) {
                if (!(ok = mbar_wait(&bars.pat_full[buf], (n >> 1) & 1, abort, p.status, kStatusTimeout))) break;
                if (frozen) {
                    const float* qa = pat_a + buf * kPatFloats;
                    const float* qr = pat_r + buf * kPatFloats;
#pragma unroll
                    for (int c = 0; c < TK; c += 4) {
                        const float4 a4 = *reinterpret_cast<const float4*>(qa + c);
                        sv[c] = __float_as_uint(a4.x + qr[-c]);
                        sv[c + 1] = __float_as_uint(a4.y + qr[-c - 1]);
                        sv[c + 2] = __float_as_uint(a4.z + qr[-c - 2]);
                        sv[c + 3] = __float_as_uint(a4.w + qr[-c - 3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.pat_empty[buf]);
            } else if (frozen) {   // (keys past my own position are masked below)
#pragma unroll
                for (int c = 0; c < TK; ++c) {
                    const int y = min(x0 + c, i);
                    sv[c] = __float_as_uint(__ldg(ra + y) + __ldg(rr + i - y));
                }
            }
        }
        // masks, in tiles that some row does not see whole
        const bool lost = *(volatile int*)&sh.lost != 0;
        if (lost || x0 + TK > w.g.hi || x0 + TK - 1 > w.imin - w.off ||
            (p.window > 0 && x0 <= w.imax - w.off - p.window)) {
            uint32_t have = 0xffffffffu;   // boxes whose page is in the cache
            if (lost)
                for (int b = 0; b < TK / P.box; ++b) {
                    const int bx = x0 + b * P.box;
                    if (box_seen(w.g, bx, P.box) && paged_page(p, w.it, bx) < 0) have &= ~(1u << b);
                }
            const int lo = row.frozen || p.window == 0 ? -1 : i - p.window;   // slots <= lo: sinks only
            const int sink = p.sinks - w.off, last = min(i, w.g.hi - 1);   // (a prefix ends before i)
#pragma unroll
            for (int c = 0; c < TK; ++c) {
                const int x = x0 + c;
                const bool seen = x <= last && (x > lo || x < sink) && ((have >> (c >> box_log2)) & 1u);
                if (!seen) sv[c] = __float_as_uint(-INFINITY);
            }
        }
        float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
        for (int c = 0; c < TK; c += 4) {
            ma = fmax3(ma, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            mb = fmax3(mb, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
        }
        const float m_new = fmaxf(m, fmaxf(ma, mb) * sc);
        float f = 1.f;   // of O
        bool need = m_new > m + kRescaleThreshold;
        if (need) {
            f = fast_exp2(m - m_new);
            l *= f;
            m = m_new;
        }
        const int now = sh.vexp[buf];   // (the same for every row)
        if (now != vexp) {
            f *= vexp == -1000 ? 0.f : exp2f((float)(vexp - now));
            vexp = now;
            need = true;
        }
        const float ref = m == -INFINITY ? 0.f : m;   // a row that has seen no key yet: weights 2^-inf = 0
        const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-ref, -ref);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
        uint32_t pk[TK / 2];
#pragma unroll
        for (int c = 0; c < TK / 2; c += 2) {
            const float4 vs = *reinterpret_cast<const float4*>(&sh.vs[buf][2 * c]);
            const float2 x = ffma2(make_float2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sc2, nm2);
            const float2 y = ffma2(make_float2(__uint_as_float(sv[2 * c + 2]), __uint_as_float(sv[2 * c + 3])), sc2, nm2);
            const float2 ex = make_float2(fast_exp2(x.x), fast_exp2(x.y)), ey = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            acc0 = fadd2(acc0, ex);
            acc1 = fadd2(acc1, ey);
            const float2 wx = fmul2(ex, make_float2(vs.x, vs.y)), wy = fmul2(ey, make_float2(vs.z, vs.w));
            pk[c] = pack_f16(wx.x, wx.y);
            pk[c + 1] = pack_f16(wy.x, wy.y);
        }
        l += (acc0.x + acc1.x) + (acc0.y + acc1.y);
        if (n > 0) {   // P V of the previous tile is done: P is free, O is stable
            if (!(ok = mbar_wait(&bars.o_done[g], (n - 1) & 1, abort, p.status, kStatusTimeout))) break;
            tc_fence_after();
        }
        tmem_st32(tmem + C::col_p, pk);
        if (n > 0 && __any_sync(0xffffffffu, need)) {
            uint32_t ov[32];
#pragma unroll
            for (int q = 0; q < kD; q += 32) {
                tmem_ld32(tmem + C::col_o + q, ov);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * f);
                tmem_st32(tmem + C::col_o + q, ov);
            }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_ready[g]);
    }
    // (a lane whose wait ran out leaves its warp's loop alone; the warp meets again here)
    __syncwarp();
    ok = __all_sync(0xffffffffu, ok) && mbar_wait_warp(&bars.o_done[g], (n - 1) & 1, abort, p.status, kStatusTimeout);
    tc_fence_after();
    if (!ok) return;
    // my row
    const bool sees = row.i >= 0 && l != 0.f;   // (a NaN sum is one)
    const size_t at = paged_out_row(p, row);
    const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
    const float back = vexp == -1000 ? 0.f : pow2i(vexp - kWeightExp);
    const float mul = p.nsplit > 1 ? back : back * (1.f / l);
#pragma unroll
    for (int q = 0; q < kD; q += 32) {
        uint32_t ov[32];
        tmem_ld32(tmem + C::col_o + q, ov);
        tmem_ld_wait();
        if (!row.there || q >= p.d) continue;
        float y[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) y[c] = sees ? __uint_as_float(ov[c]) * mul : 0.f;
        if (p.nsplit > 1) {
            float4* out = reinterpret_cast<float4*>(p.po + (at * p.nsplit + split) * p.d + q);
#pragma unroll
            for (int c = 0; c < 8; ++c) out[c] = make_float4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
        } else {
            uint4* out = reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + at * p.d + q);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                out[c] = make_uint4(pack_bf16(y[8 * c], y[8 * c + 1]), pack_bf16(y[8 * c + 2], y[8 * c + 3]),
                                    pack_bf16(y[8 * c + 4], y[8 * c + 5]), pack_bf16(y[8 * c + 6], y[8 * c + 7]));
        }
    }
    if (!row.there) return;
    if (p.nsplit > 1) p.ml[at * p.nsplit + split] = sees ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
    else p.lse[at] = sees ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Every warp but the loading one: q's terms and tensor memory are there.
__device__ __forceinline__ void set_up_done() {
    tc_fence_before();
    asm volatile("bar.sync 2, 480;" ::: "memory");
    tc_fence_after();
}

// q's terms, one row per thread (zeros for frozen rows and those without a token); the row's scale.
template <int kD>
__device__ __forceinline__ float put_q(const Q8Params& P, const PagedRow& row, uint8_t* sm) {
    using C = Cfg<kD>;
    const PagedArgs& p = P.a;
    const int t = threadIdx.x;
    const bool have = row.i >= 0 && !row.frozen;
    const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.q + paged_out_row(p, row) * p.d);
    uint4 x[kD / 8];
#pragma unroll
    for (int c = 0; c < kD / 8; ++c) x[c] = have && 8 * c < p.d ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
    // the row's largest magnitude as bits: above 0x7f7f it holds an infinity or a NaN
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kD / 8; ++c) {
        const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = __vmaxu2(top, v[k] & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
    const bool bad = top >= 0x7f80u;
    // 448 = 1.75 x 2^8
    int e = 8 - ((int)(top >> 7) - 127) - ((top & 0x7fu) > 0x60u);
    e = bad ? 0 : e < -120 ? -120 : e > 120 ? 120 : e;
    const float f = pow2i(e);
    uint8_t* hi = sm + C::q + (t >> 7) * 2 * 128 * 128;
    uint8_t* lo = hi + 128 * 128;
#pragma unroll
    for (int c = 0; c < kD / 16; ++c) {
        const uint32_t v[8] = {x[2 * c].x, x[2 * c].y, x[2 * c].z, x[2 * c].w,
                               x[2 * c + 1].x, x[2 * c + 1].y, x[2 * c + 1].z, x[2 * c + 1].w};
        uint32_t h[4], r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t hp[2], rp[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float y0 = __uint_as_float(v[2 * k + b] << 16) * f, y1 = __uint_as_float(v[2 * k + b] & 0xffff0000u) * f;
                hp[b] = pack_e4m3(y0, y1);
                const float2 z = unpack_e4m3(hp[b]);
                rp[b] = pack_e4m3(y0 - z.x, y1 - z.y);
            }
            h[k] = hp[0] | hp[1] << 16;
            r[k] = rp[0] | rp[1] << 16;
            if (bad) h[k] = r[k] = 0x7f7f7f7fu;   // (saturation would hide an infinity)
        }
        *reinterpret_cast<uint4*>(hi + sw128_offset(t & 127, 16 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + sw128_offset(t & 127, 16 * c)) = make_uint4(r[0], r[1], r[2], r[3]);
    }
    fence_proxy_async_smem();
    return p.scale_log2 * pow2i(-e);
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
    if (warp == 0) {
        if (lane == 0) {
            sh.abort_flag = 0;
            sh.imin = 0x7fffffff;
            sh.imax = -1;
            sh.kinds = sh.frozen_warps = sh.lost = 0;
        }
        if (lane < C::slots) {
            mbar_init(&bars.full[lane], 1);
            mbar_init(&bars.empty[lane], 5);   // K: its MMAs and the four warps that read its scales; V: those warps
        } else if (lane < C::slots + 2) {
            const int i = lane - C::slots;
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.s_empty[i], 4);
            mbar_init(&bars.p_ready[i], 4);
            mbar_init(&bars.o_done[i], 1);
            mbar_init(&bars.sc_ready[i], 1);
            mbar_init(&bars.v_ready[i], 4);
            mbar_init(&bars.v_free[i], 1);
            mbar_init(&bars.pat_full[i], 1);
            mbar_init(&bars.mma_idle[i], 1);
        }
        fence_mbar_init();
    }
    RowsWork w;
    w.it = paged_item(p, blockIdx.x);
    const PagedBlock block = paged_block(p, w.it);
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    PagedRow row;
    if (t < 256) {
        row = paged_row(p, w.it, block, t);
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
    w.there = block.there;
    w.groups = block.there > 128 ? 2 : 1;
    w.g = paged_range(p, w.it, w.imin, w.imax, (sh.kinds & 2) != 0 || p.window == 0);
    const int per = p.per_chunk[w.it.part];
    w.e0 = min(w.it.chunk * per, w.g.n);
    w.e1 = min(w.e0 + per, w.g.n);
    if (w.e0 >= w.e1) {   // no keys: nothing but the rows' empty sums
        if (t < 256 && row.there) {
            const int split = w.it.part ? p.chunks[0] + w.it.chunk : w.it.chunk;
            const size_t at = paged_out_row(p, row);
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
    w.nf = (block.first + w.there - 1) / block.per_head - w.fz0 + 1;
    w.staged = (long long)w.nf * ((long long)w.imax - w.imin + 2 * TK + 3) <= kPatFloats;
    const int n = w.e1 - w.e0;
    volatile int* abort = &sh.abort_flag;

    // one setmaxnreg for each warpgroup
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
        float qscale = 0.f;
        if (w.any_ord && (t >> 7) < w.groups) qscale = put_q<kD>(P, row, sm);
        if (t == 0 && sh.frozen_warps > 0) {
            mbar_init(&bars.pat_empty[0], sh.frozen_warps);
            mbar_init(&bars.pat_empty[1], sh.frozen_warps);
            fence_mbar_init();
        }
        set_up_done();
        if ((t >> 7) < w.groups) row_warps<kD>(P, w, row, qscale, sm, sh);
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
            const uint32_t tmem = sh.tmem_base;
            if (warp == 13) {
                // S of tile j, when K is there and the group has read S of tile j - 1
                constexpr uint32_t id_s = idesc_e4m3(128, TK, 0, 0);
                const uint64_t d_q = sdesc_sw128(smem_u32(sm + C::q), 16, 1024);   // K-major, as K
                const uint64_t d_ring = sdesc_sw128(smem_u32(sm + C::ring), 16, 1024);
                const int steps = p.d / 32;
                for (int j = 0; j < n && w.any_ord; ++j) {
                    const int ld = w.k_load(j), s = ld % C::slots;
                    if (!wait_all(&bars.full[s], (ld / C::slots) & 1, abort, p.status)) break;
                    const uint64_t d_k = sdesc_advance(d_ring, s * TK * 128);
                    bool ok = true;
                    for (int g = 0; g < w.groups && ok; ++g) {
                        ok = j == 0 || wait_all(&bars.s_empty[g], (j - 1) & 1, abort, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        for (int k = 0; k < 2 * steps; ++k) {   // hi, then lo
                            const int term = k >= steps, kk = k - term * steps;
                            mma_ss_e4m3_warp(tmem + g * C::group, sdesc_advance(d_q, (2 * g + term) * 16384 + 32 * kk),
                                             sdesc_advance(d_k, 32 * kk), id_s, k > 0);
                        }
                        mma_commit_warp(&bars.s_full[g]);
                    }
                    if (!ok) break;
                    mma_commit_warp(&bars.empty[s]);
                }
            } else if (warp == 14) {
                // O += P V of tile j, when V is unpacked and the group's weights are there
                constexpr uint32_t id_o = idesc_f16(128, kD, 0, 1);
                const uint64_t d_v16 = sdesc_sw128(smem_u32(sm + C::v16), C::v16_atom, 1024);   // MN-major
                for (int j = 0; j < n; ++j) {
                    if (!wait_all(&bars.v_ready[j & 1], (j >> 1) & 1, abort, p.status)) break;
                    const uint64_t d_v = sdesc_advance(d_v16, (j & 1) * C::v16_tile);
                    bool ok = true;
                    for (int g = 0; g < w.groups && ok; ++g) {
                        ok = wait_all(&bars.p_ready[g], j & 1, abort, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t base = tmem + g * C::group;
#pragma unroll
                        for (int k = 0; k < TK / 16; ++k)
                            mma_ts_warp(base + C::col_o, base + C::col_p + 8 * k, sdesc_advance(d_v, k * 2048), id_o,
                                        (j > 0 || k > 0) ? 1u : 0u);
                        mma_commit_warp(&bars.o_done[g]);
                    }
                    if (!ok) break;
                    mma_commit_warp(&bars.v_free[j & 1]);
                }
            } else if (sh.frozen_warps > 0 && w.staged) {
                pattern_warp<kD>(P, w, sm, sh);
            }
            if (warp < 15) {   // every MMA issued here is done before tensor memory is freed
                mma_commit_warp(&bars.mma_idle[warp - 13]);
                if (lane == 0) mbar_wait_bounded(&bars.mma_idle[warp - 13], 0, kWaitLimitNs);
                __syncwarp();
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
