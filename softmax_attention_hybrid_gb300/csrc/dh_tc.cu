// The layer in bf16 on the tensor cores at head dimensions 96 and 128 (the
// paper's 1B model uses d_h = 96, App. C.5; App. D.2 tests d_h in {64, 96, 128}).
//
// A [128 rows x d] tile is held in shared memory as two 128-byte-swizzled atoms of
// 64 columns, the layout of the d = 64 kernels twice over. At d = 96 the second
// atom's TMA box reaches past the row end, and TMA fills columns 96..127 with
// zeros: they add nothing to Q K^T, and the outputs' columns 96..127 are never
// stored. So one code path serves both head dimensions, padded to 128.
//
// Launches (all with programmatic dependent launch after the layer's call_init
// and, in the forward, lognorm kernels):
//   forward     dh_fwd_kernel        one CTA per (query block, slice): online
//                                    softmax (ordinary) or Eq. 3 in its exact
//                                    form (frozen), O in tensor memory
//   backward    dh_rowvec_kernel     -lse * log2(e) and D = dO . O per query block
//               dh_bwd_kv_kernel     one CTA per (key block, slice): dV, dK
//               dh_bwd_q_kernel      one CTA per (query block, slice): dQ
// Each CTA: in the forward warps 0-3 own one tile row per thread (the TMEM lanes), warp 4
// loads with TMA, warp 5 owns tensor memory and issues the MMAs from one thread; in the
// backward passes warps 0-7 are the row warps (half of a row each), 8 and 9 the other two.
// Every wait is bounded (mbar_wait): on expiry the CTA records the timeout in the
// call's status word, every role gives up, and tensor memory is freed.
#include <math.h>
#include <string.h>

#include "saf_internal.h"
#include "tc_common.cuh"

namespace saf {
namespace {

using namespace tc;

constexpr int kAtom = 128 * 64 * 2;    // 128 rows x 64 bf16, 128-byte swizzle
constexpr int kTile = 2 * kAtom;       // 128 rows x 128 (d padded to 128)
constexpr int kThreads = 192;      // forward: 4 row warps, a TMA warp, an MMA warp
constexpr int kThreadsBwd = 320;   // backward: 8 row warps (a row's columns in two halves), TMA, MMA
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Descriptors of a [128 x 128] tile, formed once per tile, and of its k-steps, which add a
// constant: an MMA then takes a few instructions of the issuing thread and not twenty.
// K-major: k-step k is 16 columns of d.
__device__ __forceinline__ uint64_t kmaj_tile(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t kmaj(uint64_t tile, int k) {
    return sdesc_advance(tile, (uint32_t)(k >> 2) * kAtom + (uint32_t)(k & 3) * 32);
}
// Read MN-major (d as the N dimension), k-step k is 16 rows: the leading-dimension offset steps
// from the first 64 columns of d (atom 0) to the next (atom 1), so one N = 128 MMA covers the
// whole padded head dimension.
__device__ __forceinline__ uint64_t mnmaj_tile(uint32_t tile) { return sdesc_sw128(tile, kAtom, 1024); }
__device__ __forceinline__ uint64_t mnmaj(uint64_t tile, int k) { return sdesc_advance(tile, (uint32_t)k * 2048); }

// Load a [128 x 128] tile (two atoms) of tensor map `map` at row y of slice z.
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int y, int z) {
    tma_load_3d(dst, map, bar, 0, y, z);
    tma_load_3d(dst + kAtom, map, bar, 64, y, z);
}

// Columns c0 .. c0 + n - 1 (n a multiple of 32, at most 128, the same in every lane) of a
// warp's 32 bf16 output rows of d elements: lane l holds row row0 + l as n fp32 values, which
// are scaled and rounded; rows l < nrows only. Whole 32-byte sectors per store instruction.
__device__ __forceinline__ void store_rows_cols(__nv_bfloat16* row0, int d, int nrows, int c0, int n,
                                                const uint32_t* v, float scale) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (32 * q < n) {
            uint4 x[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t* w = v + 32 * q + 8 * c;
                x[c] = make_uint4(pack_bf16(__uint_as_float(w[0]) * scale, __uint_as_float(w[1]) * scale),
                                  pack_bf16(__uint_as_float(w[2]) * scale, __uint_as_float(w[3]) * scale),
                                  pack_bf16(__uint_as_float(w[4]) * scale, __uint_as_float(w[5]) * scale),
                                  pack_bf16(__uint_as_float(w[6]) * scale, __uint_as_float(w[7]) * scale));
            }
            store_rows64(reinterpret_cast<uint8_t*>(row0 + c0 + 32 * q), 2 * (size_t)d, nrows, x);
        }
    }
}

// Head kinds of a key-block item, as a compile-time tag so that each kind gets its own
// tile loop: 0 every query head ordinary, 1 every one frozen, 2 mixed.
template <int M>
struct HeadKinds {
    static constexpr int value = M;
};

struct DhParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    __nv_bfloat16* o;
    float* lse;
    __nv_bfloat16 *dq, *dk, *dv;
    const __nv_bfloat16* o_in;
    const __nv_bfloat16* dO;
    const float* lse_in;
    const float* lz;       // [H, T]: log Z of frozen heads
    const float* a2p;      // [H, Tp]: a * log2(e), -inf padded
    const float* r2p;      // [H, Tp + 256]: r * log2(e) shifted by 127, -inf padded
    float* rowvec;         // [B, H, nqb, 256]: -lse * log2(e) | D per query block
    SinkParts sp;          // key-block pass, windowed
    uint32_t* status;
    int B, H, T, d, Tp, nqb;
    int Hkv, G;            // key/value heads; query head h reads key/value head h / G
    int window, sinks;     // ordinary heads (kWin kernels)
    bool q_waits;          // query-block pass: dq lies over what the key-block pass reads
    float scale_log2;      // log2(e) / sqrt(d)
    float scale;           // 1 / sqrt(d)
    HeadMask mask;
    int n_ord, n_frz;
    uint8_t ord_heads[SAF_MAX_HEADS], frz_heads[SAF_MAX_HEADS];
};

// ---------------------------------------------------------------------------
// Forward. Two CTAs share an SM (about 99 KB of shared memory and 256 TMEM
// columns each), so that one CTA's MMAs run while the other's rows are in the
// softmax. K and V have a buffer each: K(j + 1) loads while the rows work on
// S(j), V(j + 1) while they work on S(j + 1). A frozen head, which needs no K, has
// its odd blocks' V in the K buffer, and their W in the second half of S's columns: its
// loads and its MMAs run beside the rows. (All heads frozen, H32/Hkv8 d128, B2 T4096:
// 264 us with one buffer, 206 us so: a load takes about 2000 cycles, a tile of W 1500.)
// TMEM: S [0, 128) fp32, P written over S[0, 64) as bf16 pairs (frozen: W of even
// blocks, and [64, 128) of odd ones) | O [128, 256).
// ---------------------------------------------------------------------------
struct FwdSmem {
    static constexpr int q = 0;
    static constexpr int k = kTile;
    static constexpr int v = 2 * kTile;
    static constexpr int vec = 3 * kTile;   // frozen, two: a2 slice [128] | r2 band [256]
    static constexpr int vec_bytes = 1536;
    static constexpr int total = vec + 2 * vec_bytes;
};

struct FwdBars {
    // v: frozen heads' even blocks, k: their odd ones; p_ready: two for a frozen head's blocks in
    // turn, since its warps may be a block ahead of one another
    uint64_t q_full, k_full, k_empty, v_full, v_empty, s_full, p_ready[2], o_done, mma_idle;
};

template <bool kWin>
__global__ void __launch_bounds__(kThreads, 2) dh_fwd_kernel(const __grid_constant__ DhParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ FwdBars bars;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Over the whole launch the frozen heads' blocks, longest first, then the ordinary ones': one
    // slice after the other, the last slices' long blocks begin late and the launch ends on a few
    // SMs. (H32/Hkv8 d128, B2 T4096, forward and backward: 1273 us slice by slice, 1092 us so.)
    long long u = (long long)blockIdx.y * p.nqb + blockIdx.x;
    const long long n_frz = (long long)p.B * p.n_frz * p.nqb;
    const bool first = u < n_frz;
    if (!first) u -= n_frz;
    const int heads = first ? p.n_frz : p.n_ord, slices = p.B * heads;
    const int level = (int)(u / slices), slice = (int)(u - (long long)level * slices);
    const int qb = p.nqb - 1 - level;
    const int bh = slice / heads * p.H + (first ? p.frz_heads : p.ord_heads)[slice % heads];
    const int h = bh % p.H;
    const int bkv = (bh / p.H) * p.Hkv + h / p.G;   // key/value slice
    const bool frz = head_frozen(p.mask, h);
    // the key blocks that the rows see (every causal one for a frozen head)
    const KeyBlocks<kWin> blocks(qb * 128, qb, kWin && frz ? p.T : p.window, p.sinks, 128);
    const int nblk = blocks.n;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(&bars.q_full, 1);
        mbar_init(&bars.k_full, 1);
        mbar_init(&bars.k_empty, 1);
        mbar_init(&bars.v_full, 1);
        mbar_init(&bars.v_empty, 1);
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.p_ready[0], 4);
        mbar_init(&bars.p_ready[1], 4);
        mbar_init(&bars.o_done, 1);
        mbar_init(&bars.mma_idle, 1);
        fence_mbar_init();
    }
    if (warp == 5) {
        tmem_alloc(&tmem_base_sh, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    volatile int* abort = &abort_flag;
    uint32_t* status = p.status;

    if (warp == 4) {
        // ---------------------------------------------------------------- producer
        if (lane == 0) {
            if (!frz) {
                mbar_expect_tx(&bars.q_full, kTile);
                load_tile(sm + FwdSmem::q, &p.tm_q, &bars.q_full, qb * 128, bh);
            }
            for (int j = 0; j < nblk; ++j) {
                // the K buffer is free once S(j - 1) has been computed, the V buffer
                // once P(j - 1) V has; a frozen head's buffers, with the vectors, once W(j - 2) V has
                if (!frz) {
                    if (!mbar_wait(&bars.k_empty, (j & 1) ^ 1u, abort, status, kStatusTimeout)) break;
                    mbar_expect_tx(&bars.k_full, kTile);
                    load_tile(sm + FwdSmem::k, &p.tm_k, &bars.k_full, blocks.id(j) * 128, bkv);
                    if (!mbar_wait(&bars.v_empty, (j & 1) ^ 1u, abort, status, kStatusTimeout)) break;
                    mbar_expect_tx(&bars.v_full, kTile);
                    load_tile(sm + FwdSmem::v, &p.tm_v, &bars.v_full, blocks.id(j) * 128, bkv);
                } else {   // (it visits block j as its j-th)
                    const bool odd = j & 1;
                    uint64_t* full = odd ? &bars.k_full : &bars.v_full;
                    float* vec = reinterpret_cast<float*>(sm + FwdSmem::vec + odd * FwdSmem::vec_bytes);
                    if (!mbar_wait(odd ? &bars.k_empty : &bars.v_empty, ((j >> 1) & 1) ^ 1u, abort, status,
                                   kStatusTimeout))
                        break;
                    mbar_expect_tx(full, kTile + 512 + 1024);
                    bulk_load(vec, p.a2p + (size_t)h * p.Tp + (size_t)j * 128, 512, full);
                    bulk_load(vec + 128, p.r2p + (size_t)h * (p.Tp + 256) + (size_t)(qb - j) * 128, 1024, full);
                    load_tile(sm + (odd ? FwdSmem::k : FwdSmem::v), &p.tm_v, full, j * 128, bkv);
                }
            }
        }
    } else if (warp == 5) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16(128, 128, 0, 0);   // S = Q K^T
            const uint32_t id_o = idesc_bf16(128, 128, 0, 1);   // O += P V, V MN-major
            const uint32_t d_s = tmem, d_o = tmem + 128;
            const uint64_t sq = kmaj_tile(smem_u32(sm + FwdSmem::q)), sk = kmaj_tile(smem_u32(sm + FwdSmem::k));
            const uint64_t sv = mnmaj_tile(smem_u32(sm + FwdSmem::v));
            bool ok = true;
            auto issue_s = [&](int j) -> bool {
                if (!mbar_wait(&bars.k_full, j & 1, abort, status, kStatusTimeout)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_ss(d_s, kmaj(sq, k), kmaj(sk, k), id_s, k > 0);
                mma_commit(&bars.s_full);
                mma_commit(&bars.k_empty);
                return true;
            };
            if (!frz) {
                ok = mbar_wait(&bars.q_full, 0, abort, status, kStatusTimeout) && issue_s(0);
                for (int j = 0; j < nblk && ok; ++j) {
                    if (!(ok = mbar_wait(&bars.v_full, j & 1, abort, status, kStatusTimeout))) break;
                    if (!(ok = mbar_wait(&bars.p_ready[0], j & 1, abort, status, kStatusTimeout))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(d_o, d_s + 8 * k, mnmaj(sv, k), id_o, (j > 0 || k > 0) ? 1u : 0u);
                    mma_commit(&bars.o_done);
                    mma_commit(&bars.v_empty);
                    // S(j + 1) overwrites the columns P(j) is read from; MMAs run in issue order
                    if (j + 1 < nblk) ok = issue_s(j + 1);
                }
            } else {
                const uint64_t sv1 = mnmaj_tile(smem_u32(sm + FwdSmem::k));
                for (int j = 0; j < nblk; ++j) {
                    const bool odd = j & 1;
                    const uint32_t parity = (j >> 1) & 1;
                    if (!mbar_wait(odd ? &bars.k_full : &bars.v_full, parity, abort, status, kStatusTimeout)) break;
                    if (!mbar_wait(&bars.p_ready[odd], parity, abort, status, kStatusTimeout)) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(d_o, d_s + 64 * odd + 8 * k, mnmaj(odd ? sv1 : sv, k), id_o, (j > 0 || k > 0) ? 1u : 0u);
                    mma_commit(odd ? &bars.k_empty : &bars.v_empty);
                }
            }
            mma_commit(&bars.mma_idle);
            mbar_wait_bounded(&bars.mma_idle, 0, kWaitLimitNs);
        }
    } else {
        // ---------------------------------------------------------------- softmax / pattern rows
        const int t = threadIdx.x;   // row of the tile = TMEM lane
        const int row = qb * 128 + t;
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        float m = -INFINITY, l = 0.f;
        const float lz2 = (frz && row < p.T) ? p.lz[(size_t)h * p.T + row] * kLog2e : INFINITY;
        bool ok = true;
        for (int j = 0; j < nblk; ++j) {
            uint32_t pk[64];
            uint32_t p_base = lane_base;
            if (!frz) {
                if (!(ok = mbar_wait(&bars.s_full, j & 1, abort, status, kStatusTimeout))) break;
                tc_fence_after();
                uint32_t sr[128];   // this row of S, raw scores; hidden keys -inf
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(lane_base + 32 * c4, sr + 32 * c4);
                tmem_ld_wait();
                const int kb = blocks.id(j);
                if (kWin && window_cuts(qb, kb, p.window, 128)) {
                    // hidden past the diagonal, and before the window unless a sink
                    const int hi = (qb - kb) * 128 + t, lo = hi - p.window + 1, sink = p.sinks - kb * 128;
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > hi || (c < lo && c >= sink)) sr[c] = __float_as_uint(-INFINITY);
                } else if (kb == qb) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > t) sr[c] = __float_as_uint(-INFINITY);
                }
                // row max of the raw scores (the scale is positive): two chains of 3-input max
                float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; c += 4) {
                    ma = fmax3(ma, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                    mb = fmax3(mb, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
                }
                const float mx = fmaxf(m, fmaxf(ma, mb) * p.scale_log2);
                // a row of a windowed layer that has seen no key yet: weights 2^-inf = 0 with any
                // finite reference
                const float m_ref = kWin && mx == -INFINITY ? 0.f : mx;
                const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-m_ref, -m_ref);
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 128; c += 2) {
                    const float2 x =
                        ffma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc2, nm2);
                    const float e0 = fast_exp2(x.x), e1 = fast_exp2(x.y);
                    sum += e0 + e1;
                    pk[c >> 1] = pack_bf16(e0, e1);
                }
                const float corr = fast_exp2(m - m_ref);   // 0 on the first block (m = -inf)
                l = l * corr + sum;
                // P(j - 1) V has been added before O is rescaled (S(j) was computed after it,
                // so its columns are free for P(j) already)
                if (j > 0) {
                    if (!(ok = mbar_wait(&bars.o_done, (j - 1) & 1, abort, status, kStatusTimeout))) break;
                    tc_fence_after();
                    // tcgen05.ld/st are warp-collective: when any row of the warp has a new
                    // maximum, every lane rescales (by exactly 1 where its maximum held)
                    if (__any_sync(0xffffffffu, mx > m)) {
#pragma unroll
                        for (int c4 = 0; c4 < 4; ++c4) {
                            uint32_t u[32];
                            tmem_ld32(lane_base + 128 + 32 * c4, u);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * corr);
                            tmem_st32(lane_base + 128 + 32 * c4, u);
                        }
                    }
                }
                m = mx;
            } else {
                // the block's vectors, and W(j - 2) V done, which read the columns of this W
                const bool odd = j & 1;
                const uint32_t parity = (j >> 1) & 1;
                if (!(ok = mbar_wait(odd ? &bars.k_full : &bars.v_full, parity, abort, status, kStatusTimeout))) break;
                if (j > 1 &&
                    !(ok = mbar_wait(odd ? &bars.k_empty : &bars.v_empty, parity ^ 1u, abort, status, kStatusTimeout)))
                    break;
                tc_fence_after();
                p_base = lane_base + 64 * odd;
                const float* vec = reinterpret_cast<const float*>(sm + FwdSmem::vec + odd * FwdSmem::vec_bytes);
                // W(row, key) = exp2(a2[key] + r2[row - key] - log2 Z(row)) (Eq. 3); the band
                // holds r at distance (qb - j) 128 + t - c at entry 127 + t - c
                const float* band = vec + 128 + 127 + t;
                const float2 lz22 = make_float2(lz2, lz2);
#pragma unroll
                for (int c = 0; c < 128; c += 2) {
                    const float2 x = fsub2(fadd2(*reinterpret_cast<const float2*>(vec + c),
                                                 make_float2(band[-c], band[-c - 1])), lz22);
                    pk[c >> 1] = pack_bf16(fast_exp2(x.x), fast_exp2(x.y));
                }
            }
            tmem_st32(p_base, pk);
            tmem_st32(p_base + 32, pk + 32);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.p_ready[frz ? j & 1 : 0]);
        }
        uint64_t* done = !frz ? &bars.o_done : (nblk - 1) & 1 ? &bars.k_empty : &bars.v_empty;
        const uint32_t parity = (frz ? (nblk - 1) >> 1 : nblk - 1) & 1;
        if (ok && mbar_wait_warp(done, parity, abort, status, kStatusTimeout)) {
            tc_fence_after();
            const float inv = frz ? 1.f : 1.f / l;
            uint32_t ov[128];
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(lane_base + 128 + 32 * c4, ov + 32 * c4);
            tmem_ld_wait();
            const int row0 = row - lane;
            store_rows_cols(p.o + ((size_t)bh * p.T + row0) * p.d, p.d, p.T - row0, 0, p.d, ov, inv);
            if (row < p.T) p.lse[(size_t)bh * p.T + row] = frz ? lz2 * kLn2 : (m + log2f(l)) * kLn2;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ---------------------------------------------------------------------------
// Backward prep: rowvec[bh, qb, 0..127] = -lse * log2(e) (-inf past T),
// rowvec[bh, qb, 128..255] = D = sum_c dO_c O_c (0 past T, and for frozen heads,
// which do not use it). Grid (Tp / 128, B H). Bound by reading o and dO: 16 lanes read a row
// of them (a thread per row read every line twice), two rows a warp, eight rows' loads in
// flight. (H32 d128, B2 T4096: 21.6 us, 35 us with a thread per row, and the layer's forward and
// backward with window 512 478 us for 533.)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) dh_rowvec_kernel(const __grid_constant__ DhParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int bh = blockIdx.y, qb = blockIdx.x;
    float* v = p.rowvec + ((size_t)bh * p.nqb + qb) * 256;
    const int i = qb * 128 + threadIdx.x;
    v[threadIdx.x] = i < p.T ? -(p.lse_in[(size_t)bh * p.T + i] * kLog2e) : -INFINITY;
    if (head_frozen(p.mask, bh % p.H)) {
        v[128 + threadIdx.x] = 0.f;
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane & 15;
#pragma unroll
    for (int it0 = 0; it0 < 16; it0 += 4) {
        uint4 x[4], y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int row = qb * 128 + 32 * warp + 2 * (it0 + u) + (lane >> 4);
            x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
            if (row < p.T && 8 * part < p.d) {
                const size_t at = ((size_t)bh * p.T + row) * p.d + 8 * part;
                x[u] = __ldg(reinterpret_cast<const uint4*>(p.o_in + at));
                y[u] = __ldg(reinterpret_cast<const uint4*>(p.dO + at));
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, ys[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
            float dd = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dd = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), dd);
                dd = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), dd);
            }
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, m);
            if (part == 0) v[128 + 32 * warp + 2 * (it0 + u) + (lane >> 4)] = dd;
        }
    }
}

// TMEM column of k-step k (16 rows of the contraction) of an operand written in
// chunks of 32 rows: chunk c holds its 16 packed pairs at [32 c, 32 c + 16) and the
// second operand's at [32 c + 16, 32 c + 32).
__device__ __forceinline__ uint32_t chunk_col(int k, int second) {
    return 32u * (uint32_t)(k >> 1) + 16u * (uint32_t)second + 8u * (uint32_t)(k & 1);
}

// ---------------------------------------------------------------------------
// Backward, key-block pass: dV, dK of key block kb of key/value slice bkv. The
// tiles run over the G query heads that share the slice (one head in the
// multi-head layer) and, for each, the query blocks kb .. nqb - 1; dV sums every
// head's share, dK the ordinary heads' (zeros when the group has none).
// TMEM: two regions of 128 columns, [0, 128) and [128, 256), which even and odd tiles take in
//       turn: S^T(i) fp32 is in region i % 2, overwritten chunk by chunk with P^T and dS^T as bf16
//       pairs (chunk c: P^T at [32 c, +16), dS^T at [32 c + 16, +16)), dP^T(i) in the other |
//       dV [256, 384) | dK [384, 512).
// So the MMAs and the rows work on two tiles at once: S^T(i + 1) overwrites dP^T(i) as soon as the
// rows have read it, then come dK(i) and, over the region that it has read, dP^T(i + 1), while the
// rows form P^T(i + 1); dV(i + 1) runs while they form dS^T(i + 1). MMAs run in the order in which
// they were issued, so a region is not overwritten before the products that read it.
// The two stages hand Q and dO back apart: dO(i) is free after dV(i). The row vectors, which the
// rows need first, are loaded two tiles earlier than Q and dO (a load takes about 2000 cycles).
// ---------------------------------------------------------------------------
struct KvSmem {
    static constexpr int k = 0, v = kTile;
    static constexpr int st = 2 * kTile;      // 2 stages: Q | dO
    static constexpr int st_q = 0, st_do = kTile, st_bytes = 2 * kTile;
    static constexpr int vec = st + 2 * st_bytes;   // 4: -lse2 [128] | D [128] | r2 band [256]
    static constexpr int vec_bytes = 2048;
    static constexpr int total = vec + 4 * vec_bytes;
};

struct KvBars {
    // q_empty: the tile's MMAs are all done
    uint64_t kv_full, q_full[2], q_empty[2], do_full[2], do_empty[2], vec_full[4];
    // p: P^T or W^T. Two, for the tiles in turn: with frozen heads a row warp may be a tile
    // ahead of another, and its arrival must not count for the other's tile.
    uint64_t s_full, dp_full, p_ready[2], ds_ready, mma_idle;
};

template <bool kWin>
__global__ void __launch_bounds__(kThreadsBwd, 1) dh_bwd_kv_kernel(const __grid_constant__ DhParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ KvBars bars;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Over the whole launch the longest first: blocks of sinks, which every query sees, and early
    // blocks, which have the most query blocks after them.
    long long u = (long long)blockIdx.y * gridDim.x + blockIdx.x;
    const int slices = p.B * p.Hkv;
    const long long n_parts = kWin ? (long long)p.sp.blocks * p.sp.parts * slices : 0;
    const bool in_parts = kWin && u < n_parts;
    if (!in_parts) u -= n_parts;
    const int level = (int)(u / slices);
    const int bkv = (int)(u - (long long)level * slices);   // key/value slice
    const int kb = in_parts ? level / p.sp.parts : (kWin ? p.sp.blocks : 0) + level;
    const int b = bkv / p.Hkv, h0 = (bkv - b * p.Hkv) * p.G;   // its query heads: h0 .. h0 + G - 1
    bool any_ord = false, any_frz = false;
    for (int gi = 0; gi < p.G; ++gi) (head_frozen(p.mask, h0 + gi) ? any_frz : any_ord) = true;
    // Query tiles kb + q0 .. of a head, those that see a key of the block through a window. A part
    // has a run of them (the first one all of them where every head is frozen: the block is then
    // like its neighbours).
    int q0 = 0, nq_frz = p.nqb - kb, nq_ord = query_blocks<kWin>(kb, p.nqb, p.window, p.sinks, 128);
    const bool split = in_parts && any_ord;
    const int part = in_parts ? level % p.sp.parts : 0;
    if (split) {
        const SinkParts::Range run = p.sp.range(kb, p.T, part);
        q0 = run.first - kb;
        nq_frz = nq_ord = run.n;
    }
    if (in_parts && (split ? nq_ord == 0 : part > 0)) return;
    int ntiles = 0;
    for (int gi = 0; gi < p.G; ++gi) ntiles += kWin && !head_frozen(p.mask, h0 + gi) ? nq_ord : nq_frz;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(&bars.kv_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], 1);
            mbar_init(&bars.do_full[i], 1);
            mbar_init(&bars.do_empty[i], 1);
            mbar_init(&bars.p_ready[i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars.vec_full[i], 1);
        mbar_init(&bars.s_full, 1);
        mbar_init(&bars.dp_full, 1);
        mbar_init(&bars.ds_ready, 8);
        mbar_init(&bars.mma_idle, 1);
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    volatile int* abort = &abort_flag;
    uint32_t* status = p.status;

    if (warp == 8) {
        if (lane == 0) {
            mbar_expect_tx(&bars.kv_full, any_ord ? 2 * kTile : kTile);
            if (any_ord) load_tile(sm + KvSmem::k, &p.tm_k, &bars.kv_full, kb * 128, bkv);
            load_tile(sm + KvSmem::v, &p.tm_v, &bars.kv_full, kb * 128, bkv);
            // tile i: query head h0 + gi, block kb + qi
            auto advance = [&](int& gi, int& qi) {
                if (++qi == q0 + (kWin && !head_frozen(p.mask, h0 + gi) ? nq_ord : nq_frz)) {
                    qi = q0;
                    ++gi;
                }
            };
            int vi = 0, vgi = 0, vqi = q0;
            auto load_vec = [&]() {   // the vectors of the next tile
                const int h = h0 + vgi;
                const bool frz = head_frozen(p.mask, h);
                uint64_t* bar = &bars.vec_full[vi & 3];
                float* vec = reinterpret_cast<float*>(sm + KvSmem::vec + (vi & 3) * KvSmem::vec_bytes);
                mbar_expect_tx(bar, 1024 + (frz ? 1024 : 0));
                bulk_load(vec, p.rowvec + ((size_t)(b * p.H + h) * p.nqb + kb + vqi) * 256, 1024, bar);
                if (frz) bulk_load(vec + 256, p.r2p + (size_t)h * (p.Tp + 256) + (size_t)vqi * 128, 1024, bar);
                advance(vgi, vqi);
                ++vi;
            };
            load_vec();
            if (ntiles > 1) load_vec();
            for (int i = 0, gi = 0, qi = q0; i < ntiles; ++i) {
                const int s = i & 1, y = (kb + qi) * 128, bh = b * p.H + h0 + gi;
                const bool frz = head_frozen(p.mask, h0 + gi);
                advance(gi, qi);
                const uint32_t parity = ((i >> 1) & 1) ^ 1u;
                uint8_t* st = sm + KvSmem::st + s * KvSmem::st_bytes;
                if (!mbar_wait(&bars.do_empty[s], parity, abort, status, kStatusTimeout)) break;
                mbar_expect_tx(&bars.do_full[s], kTile);
                load_tile(st + KvSmem::st_do, &p.tm_do, &bars.do_full[s], y, bh);
                if (!mbar_wait(&bars.q_empty[s], parity, abort, status, kStatusTimeout)) break;
                if (!frz) {
                    mbar_expect_tx(&bars.q_full[s], kTile);
                    load_tile(st + KvSmem::st_q, &p.tm_q, &bars.q_full[s], y, bh);
                } else {
                    mbar_arrive(&bars.q_full[s]);   // nothing to load: the phase passes
                }
                if (vi < ntiles) load_vec();   // of tile i + 2, over those of tile i - 2
            }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16(128, 128, 0, 0);   // S^T = K Q^T, dP^T = V dO^T
            const uint32_t id_n = idesc_bf16(128, 128, 0, 1);   // dV += P^T dO, dK += dS^T Q (B MN-major)
            const uint64_t sk = kmaj_tile(smem_u32(sm + KvSmem::k)), sv = kmaj_tile(smem_u32(sm + KvSmem::v));
            bool ok = mbar_wait(&bars.kv_full, 0, abort, status, kStatusTimeout);
            auto stage = [&](int i) { return smem_u32(sm + KvSmem::st + (i & 1) * KvSmem::st_bytes); };
            auto issue_s = [&](int i) -> bool {
                if (!mbar_wait(&bars.q_full[i & 1], (i >> 1) & 1, abort, status, kStatusTimeout)) return false;
                tc_fence_after();
                const uint64_t sq = kmaj_tile(stage(i) + KvSmem::st_q);
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_ss(tmem + 128 * (i & 1), kmaj(sk, k), kmaj(sq, k), id_s, k > 0);
                mma_commit(&bars.s_full);
                return true;
            };
            auto issue_dp = [&](int i) -> bool {
                if (!mbar_wait(&bars.do_full[i & 1], (i >> 1) & 1, abort, status, kStatusTimeout)) return false;
                tc_fence_after();
                const uint64_t sdo = kmaj_tile(stage(i) + KvSmem::st_do);
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_ss(tmem + 128 * (~i & 1), kmaj(sv, k), kmaj(sdo, k), id_s, k > 0);
                mma_commit(&bars.dp_full);
                return true;
            };
            auto tiles = [&](auto kinds) {
                constexpr int M = decltype(kinds)::value;
                int nord = 0;   // ordinary tiles so far (the first one starts dK)
                bool frz = M == 0 ? false : M == 1 ? true : head_frozen(p.mask, h0);
                if (!frz) ok = ok && issue_s(0) && issue_dp(0);
                for (int i = 0, gi = 0, qi = q0; i < ntiles && ok; ++i) {
                    const int s = i & 1;
                    if (++qi == q0 + (kWin && !frz ? nq_ord : nq_frz)) {
                        qi = q0;
                        ++gi;
                    }
                    // tile i + 1 is an ordinary one
                    const bool next = M != 1 && i + 1 < ntiles && (M == 0 || !head_frozen(p.mask, h0 + gi));
                    if (frz) {
                        // (no Q was loaded, but its phase is waited for: a later tile's wait on the barrier
                        // could otherwise take the end of the phase before this one for its own)
                        if (M == 2 && !(ok = mbar_wait(&bars.q_full[s], (i >> 1) & 1, abort, status, kStatusTimeout)))
                            break;
                        if (next && !(ok = issue_s(i + 1))) break;
                        if (!(ok = mbar_wait(&bars.do_full[s], (i >> 1) & 1, abort, status, kStatusTimeout))) break;
                    }
                    if (!(ok = mbar_wait(&bars.p_ready[s], (i >> 1) & 1, abort, status, kStatusTimeout))) break;
                    tc_fence_after();
                    const uint64_t sdon = mnmaj_tile(stage(i) + KvSmem::st_do);
                    const uint32_t region = tmem + 128 * s;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + 256, region + chunk_col(k, 0), mnmaj(sdon, k), id_n, (i > 0 || k > 0) ? 1u : 0u);
                    mma_commit(&bars.do_empty[s]);
                    if (!frz) {
                        // the rows have read dP^T, and dS^T is there
                        if (!(ok = mbar_wait(&bars.ds_ready, nord & 1, abort, status, kStatusTimeout))) break;
                        tc_fence_after();
                        if (next && !(ok = issue_s(i + 1))) break;
                        const uint64_t sqn = mnmaj_tile(stage(i) + KvSmem::st_q);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ts(tmem + 384, region + chunk_col(k, 1), mnmaj(sqn, k), id_n,
                                   (nord > 0 || k > 0) ? 1u : 0u);
                        ++nord;
                    }
                    mma_commit(&bars.q_empty[s]);
                    if (next && !(ok = issue_dp(i + 1))) break;
                    if (M == 2) frz = !next;
                }
            };
            if (!any_frz)
                tiles(HeadKinds<0>{});
            else if (!any_ord)
                tiles(HeadKinds<1>{});
            else
                tiles(HeadKinds<2>{});
            mma_commit(&bars.mma_idle);
            mbar_wait_bounded(&bars.mma_idle, 0, kWaitLimitNs);
        }
    } else {
        // warp w: key rows 32 (w % 4) .. + 31 (its TMEM lanes), query columns 64 (w / 4) .. + 63
        const int quarter = warp & 3, half = warp >> 2;
        const int t = quarter * 32 + lane;   // key row of the block = TMEM lane
        const int key = kb * 128 + t;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        bool ok = true;
        auto tiles = [&](auto kinds) {
            constexpr int M = decltype(kinds)::value;
            int nord = 0;     // ordinary tiles so far: phases of sdp_full
            float a2k = 0.f;  // a * log2(e) of my key for the current query head (frozen heads)
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
            for (int i = 0, gi = 0, qi = q0; i < ntiles; ++i) {
                const bool diag = qi == 0, first = qi == q0;   // query block kb; the head's first tile
                const int h = h0 + gi;
                const bool frz = M == 0 ? false : M == 1 ? true : head_frozen(p.mask, h);
                // queries of the tile from q_far on do not see my key through the window
                const int q_far = !kWin || key < p.sinks ? 128 : t + p.window - qi * 128;
                // some key of the block does not see some query of the tile through the window
                const bool cut = kWin && p.window < (qi + 1) * 128 && kb * 128 + 127 >= p.sinks;
                if (frz && first) a2k = p.a2p[(size_t)h * p.Tp + key];   // in flight during the wait below
                if (++qi == q0 + (kWin && !frz ? nq_ord : nq_frz)) {
                    qi = q0;
                    ++gi;
                }
                const int s = i & 1;
                const uint32_t region = lane_base + 128 * s;
                if (!(ok = mbar_wait(&bars.vec_full[i & 3], (i >> 2) & 1, abort, status, kStatusTimeout))) break;
                const float* vec = reinterpret_cast<const float*>(sm + KvSmem::vec + (i & 3) * KvSmem::vec_bytes);
                if (!frz) {
                    // the commit of S^T also means that the MMAs of tile i - 2 are done
                    if (!(ok = mbar_wait(&bars.s_full, nord & 1, abort, status, kStatusTimeout))) break;
                    tc_fence_after();
                    // the vector's element pairs of this warp's queries
                    const float2* nl2 = reinterpret_cast<const float2*>(vec) + 32 * half;
                    const float2* dd2 = nl2 + 64;
                    uint32_t su[64];
                    tmem_ld32(region + 64 * half, su);
                    tmem_ld32(region + 64 * half + 32, su + 32);
                    tmem_ld_wait();
                    float pr[64];
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        const float2 x = ffma2(make_float2(__uint_as_float(su[e]), __uint_as_float(su[e + 1])), sc2,
                                               nl2[e >> 1]);
                        pr[e] = fast_exp2(x.x);
                        pr[e + 1] = fast_exp2(x.y);
                    }
                    // only the diagonal and the window's end hide anything
                    if (diag) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (64 * half + e < t) pr[e] = 0.f;
                    }
                    if (kWin && cut) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (64 * half + e >= q_far) pr[e] = 0.f;
                    }
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {   // chunks of 32 queries: their own columns, already read
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pk[e] = pack_bf16(pr[32 * cc + 2 * e], pr[32 * cc + 2 * e + 1]);
                        tmem_st16(region + 64 * half + 32 * cc, pk);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.p_ready[s]);
                    if (!(ok = mbar_wait(&bars.dp_full, nord & 1, abort, status, kStatusTimeout))) break;
                    ++nord;
                    tc_fence_after();
                    tmem_ld32(lane_base + 128 * (s ^ 1) + 64 * half, su);
                    tmem_ld32(lane_base + 128 * (s ^ 1) + 64 * half + 32, su + 32);
                    tmem_ld_wait();
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t dk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int q = 32 * cc + 2 * e;
                            const float2 x = fmul2(
                                make_float2(pr[q], pr[q + 1]),
                                fsub2(make_float2(__uint_as_float(su[q]), __uint_as_float(su[q + 1])), dd2[q >> 1]));
                            dk[e] = pack_bf16(x.x, x.y);
                        }
                        tmem_st16(region + 64 * half + 32 * cc + 16, dk);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.ds_ready);
                } else {
                    // W^T(key, q) = exp2(a2[key] + r2[q - key] - log2 Z(q)); the band holds r at
                    // distance i 128 + c - t at entry 127 + c - t. The MMAs of tile i - 2 have
                    // read the region before it is written.
                    if (i > 1 && !(ok = mbar_wait(&bars.q_empty[s], ((i >> 1) & 1) ^ 1u, abort, status, kStatusTimeout)))
                        break;
                    tc_fence_after();
                    const float* band = vec + 256 + 127 - t;
    #pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        const int c4 = 2 * half + cc;
                        uint32_t pk[16];
    #pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const int c = 32 * c4 + e;
                            const float2 x = fadd2(fadd2(make_float2(a2k, a2k), make_float2(band[c], band[c + 1])),
                                                   *reinterpret_cast<const float2*>(vec + c));
                            pk[e >> 1] = pack_bf16(fast_exp2(x.x), fast_exp2(x.y));
                        }
                        tmem_st16(region + 32 * c4, pk);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.p_ready[s]);
                }
            }
        };
        if (!any_frz)
            tiles(HeadKinds<0>{});
        else if (!any_ord)
            tiles(HeadKinds<1>{});
        else
            tiles(HeadKinds<2>{});
        // tcgen05.ld is warp-collective: every lane loads, only rows inside T are stored;
        // each half of the warps writes its 64 columns of dV and dK (those inside d)
        ok = __all_sync(0xffffffffu, ok) &&
             mbar_wait_warp(&bars.q_empty[(ntiles - 1) & 1], ((ntiles - 1) >> 1) & 1, abort, status, kStatusTimeout);
        tc_fence_after();
        const int c0 = 64 * half, n = min(64, p.d - c0);
        const int key0 = key - lane;
        for (int i = 0; i < 2 && ok; ++i) {   // dV, dK
            uint32_t v[64];
            if (i == 0 || any_ord) {
                tmem_ld32(lane_base + 256 + 128 * i + c0, v);
                tmem_ld32(lane_base + 256 + 128 * i + c0 + 32, v + 32);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int c = 0; c < 64; ++c) v[c] = 0u;
            }
            if (!split) {
                store_rows_cols((i == 0 ? p.dv : p.dk) + ((size_t)bkv * p.T + key0) * p.d, p.d, p.T - key0, c0, n, v,
                                i == 0 ? 1.f : p.scale);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(p.sp.at(bkv, kb, part, i, p.d) + (size_t)t * p.d + c0);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (4 * c < n) dst[c] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Backward, query-block pass: dQ of query block qb of an ordinary slice (zeros
// for frozen slices). The scores of the next key block are computed while the rows
// work on this one's, and its dP before this block's dQ: the rows then find S(j + 1)
// ready, form P while dP(j + 1) and dQ(j) run, and only their dS waits for dP.
// K has three buffers (S(j + 1) comes before dQ(j), which reads K(j)), V two.
// The pass reads nothing that the key-block pass before it writes, so its blocks take the SMs
// that that launch leaves as it ends: a block that runs means that every block of that launch
// has begun, which each does after its own grid_dep_wait(), so the row vectors are there. Only
// block 0 waits for that launch, at its end, so that this one's completion implies it.
// (H32/Hkv8 d128, window 512, B2 T4096, forward and backward: 643 us with the wait at the
// beginning, 595 us so; T1024: 152 and 132 us.) Where dq lies over q or dO, which that launch
// still reads, every block waits at its beginning.
// TMEM: S of even blocks [0, 128) fp32 and of odd ones [384, 512), overwritten chunk by
//       chunk with dS as bf16 pairs (chunk c at [32 c, 32 c + 16)) | dP [128, 256) |
//       dQ [256, 384).
// ---------------------------------------------------------------------------
struct QSmem {
    static constexpr int q = 0, dO = kTile;
    static constexpr int k = 2 * kTile, v = k + 3 * kTile;
    static constexpr int total = v + 2 * kTile;
};

struct QBars {
    uint64_t q_full, k_full[3], k_empty[3], v_full[2], v_empty[2], s_full[2], dp_full, ds_ready, all_done, mma_idle;
};

template <bool kWin>
__global__ void __launch_bounds__(kThreadsBwd, 1) dh_bwd_q_kernel(const __grid_constant__ DhParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ QBars bars;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    if (p.q_waits) grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.y * p.nqb + blockIdx.x;
    const int slices = p.B * p.H;
    const int qb = p.nqb - 1 - (int)(u / slices), bh = (int)(u % slices);   // longest first
    const int h = bh % p.H;
    const int bkv = (bh / p.H) * p.Hkv + h / p.G;   // key/value slice
    if (head_frozen(p.mask, h)) {
        // dQ of a frozen head is exactly zero
        if (threadIdx.x < 128) {
            const int row = qb * 128 + threadIdx.x;
            if (row < p.T) {
                uint4* dst = reinterpret_cast<uint4*>(p.dq + ((size_t)bh * p.T + row) * p.d);
                for (int c = 0; c < p.d / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if (u == 0) grid_dep_wait();
        return;
    }
    const KeyBlocks<kWin> blocks(qb * 128, qb, p.window, p.sinks, 128);   // the key blocks that the rows see
    const int nblk = blocks.n;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(&bars.q_full, 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.v_full[i], 1);
            mbar_init(&bars.v_empty[i], 1);
            mbar_init(&bars.s_full[i], 1);
        }
        mbar_init(&bars.dp_full, 1);
        mbar_init(&bars.ds_ready, 8);
        mbar_init(&bars.all_done, 1);
        mbar_init(&bars.mma_idle, 1);
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    volatile int* abort = &abort_flag;
    uint32_t* status = p.status;

    if (warp == 8) {
        if (lane == 0) {
            mbar_expect_tx(&bars.q_full, 2 * kTile);
            load_tile(sm + QSmem::q, &p.tm_q, &bars.q_full, qb * 128, bh);
            load_tile(sm + QSmem::dO, &p.tm_do, &bars.q_full, qb * 128, bh);
            int sk = 0, pk = 1;   // K buffer, and the parity of its empty phase
            for (int j = 0; j < nblk; ++j) {
                const int sv = j & 1;
                if (!mbar_wait(&bars.k_empty[sk], pk, abort, status, kStatusTimeout)) break;
                mbar_expect_tx(&bars.k_full[sk], kTile);
                load_tile(sm + QSmem::k + sk * kTile, &p.tm_k, &bars.k_full[sk], blocks.id(j) * 128, bkv);
                if (!mbar_wait(&bars.v_empty[sv], ((j >> 1) & 1) ^ 1u, abort, status, kStatusTimeout)) break;
                mbar_expect_tx(&bars.v_full[sv], kTile);
                load_tile(sm + QSmem::v + sv * kTile, &p.tm_v, &bars.v_full[sv], blocks.id(j) * 128, bkv);
                if (++sk == 3) {
                    sk = 0;
                    pk ^= 1;
                }
            }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16(128, 128, 0, 0);   // S = Q K^T, dP = dO V^T
            const uint32_t id_n = idesc_bf16(128, 128, 0, 1);   // dQ += dS K (K MN-major)
            const uint64_t sq = kmaj_tile(smem_u32(sm + QSmem::q)), sdo = kmaj_tile(smem_u32(sm + QSmem::dO));
            const uint64_t k0 = kmaj_tile(smem_u32(sm + QSmem::k)), v0 = kmaj_tile(smem_u32(sm + QSmem::v));
            const uint64_t kn0 = mnmaj_tile(smem_u32(sm + QSmem::k));
            bool ok = mbar_wait(&bars.q_full, 0, abort, status, kStatusTimeout);
            int sk = 0, pk = 0;   // K buffer of the next S, and the parity of its full phase
            // S(j) may overwrite the columns of dS(j - 2): dQ(j - 2) was issued before it
            auto issue_s = [&](int j) -> bool {
                if (!mbar_wait(&bars.k_full[sk], pk, abort, status, kStatusTimeout)) return false;
                tc_fence_after();
                const uint64_t k_ = sdesc_advance(k0, sk * kTile);
                const uint32_t col = (j & 1) ? 384u : 0u;
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_ss(tmem + col, kmaj(sq, k), kmaj(k_, k), id_s, k > 0);
                mma_commit(&bars.s_full[j & 1]);
                if (++sk == 3) {
                    sk = 0;
                    pk ^= 1;
                }
                return true;
            };
            auto issue_dp = [&](int j) -> bool {
                const int s = j & 1;
                if (!mbar_wait(&bars.v_full[s], (j >> 1) & 1, abort, status, kStatusTimeout)) return false;
                tc_fence_after();
                const uint64_t v_ = sdesc_advance(v0, s * kTile);
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_ss(tmem + 128, kmaj(sdo, k), kmaj(v_, k), id_s, k > 0);
                mma_commit(&bars.dp_full);
                mma_commit(&bars.v_empty[s]);
                return true;
            };
            ok = ok && issue_s(0) && issue_dp(0);
            int sq_k = 0;   // K buffer of block j
            for (int j = 0; j < nblk && ok; ++j) {
                if (j + 1 < nblk && !(ok = issue_s(j + 1))) break;
                // the rows have read S(j) and dP(j), and dS(j) is there
                if (!(ok = mbar_wait(&bars.ds_ready, j & 1, abort, status, kStatusTimeout))) break;
                tc_fence_after();
                if (j + 1 < nblk && !(ok = issue_dp(j + 1))) break;
                const uint64_t k_ = sdesc_advance(kn0, sq_k * kTile);
                const uint32_t col = (j & 1) ? 384u : 0u;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ts(tmem + 256, tmem + col + chunk_col(k, 0), mnmaj(k_, k), id_n, (j > 0 || k > 0) ? 1u : 0u);
                mma_commit(&bars.k_empty[sq_k]);
                sq_k = sq_k == 2 ? 0 : sq_k + 1;
            }
            mma_commit(&bars.all_done);
            mma_commit(&bars.mma_idle);
            mbar_wait_bounded(&bars.mma_idle, 0, kWaitLimitNs);
        }
    } else {
        // warp w: query rows 32 (w % 4) .. + 31 (its TMEM lanes), key columns 64 (w / 4) .. + 63
        const int quarter = warp & 3, half = warp >> 2;
        const int t = quarter * 32 + lane;   // query row of the block = TMEM lane
        const int row = qb * 128 + t;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const float* rv = p.rowvec + ((size_t)bh * p.nqb + qb) * 256;
        const float nl2 = rv[t], dd = rv[128 + t];
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nl22 = make_float2(nl2, nl2), dd2 = make_float2(dd, dd);
        bool ok = true;
        for (int j = 0; j < nblk; ++j) {
            if (!(ok = mbar_wait(&bars.s_full[j & 1], (j >> 1) & 1, abort, status, kStatusTimeout))) break;
            tc_fence_after();
            const uint32_t s_base = lane_base + ((j & 1) ? 384u : 0u) + 64 * half;
            // keys of the block before k_near are hidden by the window unless they are sinks
            const int kb = blocks.id(j);
            const int k_near = kWin ? (qb - kb) * 128 + t - p.window + 1 : 0, sink = p.sinks - kb * 128;
            uint32_t su[64];
            tmem_ld32(s_base, su);
            tmem_ld32(s_base + 32, su + 32);
            tmem_ld_wait();
            float pr[64];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
                const float2 x = ffma2(make_float2(__uint_as_float(su[e]), __uint_as_float(su[e + 1])), sc2, nl22);
                pr[e] = fast_exp2(x.x);
                pr[e + 1] = fast_exp2(x.y);
            }
            // only the diagonal and the window's beginning hide anything
            if (kb == qb) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (64 * half + e > t) pr[e] = 0.f;
            }
            if (kWin && window_cuts(qb, kb, p.window, 128)) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (64 * half + e < k_near && 64 * half + e >= sink) pr[e] = 0.f;
            }
            if (!(ok = mbar_wait(&bars.dp_full, j & 1, abort, status, kStatusTimeout))) break;
            tc_fence_after();
            tmem_ld32(lane_base + 128 + 64 * half, su);
            tmem_ld32(lane_base + 128 + 64 * half + 32, su + 32);
            tmem_ld_wait();
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                uint32_t dk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int k0 = 32 * cc + 2 * e;
                    const float2 x =
                        fmul2(make_float2(pr[k0], pr[k0 + 1]),
                              fsub2(make_float2(__uint_as_float(su[k0]), __uint_as_float(su[k0 + 1])), dd2));
                    dk[e] = pack_bf16(x.x, x.y);
                }
                tmem_st16(s_base + 32 * cc, dk);   // the chunk's own columns, already read
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ds_ready);
        }
        if (ok && mbar_wait_warp(&bars.all_done, 0, abort, status, kStatusTimeout)) {
            tc_fence_after();
            const int c0 = 64 * half, n = min(64, p.d - c0);
            const int row0 = row - lane;
            uint32_t v[64];
            tmem_ld32(lane_base + 256 + c0, v);
            tmem_ld32(lane_base + 256 + c0 + 32, v + 32);
            tmem_ld_wait();
            store_rows_cols(p.dq + ((size_t)bh * p.T + row0) * p.d, p.d, p.T - row0, c0, n, v, p.scale);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (u == 0) grid_dep_wait();
}

DhParams make_params(const LayerArgs& a) {
    DhParams p;
    memset(&p, 0, sizeof(p));
    p.B = a.B;
    p.H = a.H;
    p.T = a.T;
    p.d = a.d;
    p.nqb = (a.T + 127) / 128;
    p.Tp = p.nqb * 128;
    p.scale = 1.f / sqrtf((float)a.d);
    p.scale_log2 = kLog2e * p.scale;
    p.mask = a.mask;
    p.status = a.status;
    p.lz = a.lz;
    p.a2p = a.a2p;
    p.r2p = a.r2p;
    p.rowvec = a.rowvec;
    p.Hkv = a.Hkv > 0 ? a.Hkv : a.H;
    p.G = a.H / p.Hkv;
    p.window = a.window;
    p.sinks = a.sinks;
    for (int h = 0; h < a.H; ++h) {
        if (head_frozen(a.mask, h))
            p.frz_heads[p.n_frz++] = (uint8_t)h;
        else
            p.ord_heads[p.n_ord++] = (uint8_t)h;
    }
    return p;
}

bool make_maps(DhParams& p, const LayerArgs& a, bool backward) {
    const int BH = a.B * a.H, BHkv = a.B * p.Hkv;
    bool ok = make_tmap_bf16_3d(&p.tm_v, a.v, a.d, a.T, BHkv, 64, 128);
    if (a.q) ok = ok && make_tmap_bf16_3d(&p.tm_q, a.q, a.d, a.T, BH, 64, 128);
    if (a.k) ok = ok && make_tmap_bf16_3d(&p.tm_k, a.k, a.d, a.T, BHkv, 64, 128);
    if (backward) ok = ok && make_tmap_bf16_3d(&p.tm_do, a.dO, a.d, a.T, BH, 64, 128);
    return ok;
}

}  // namespace

cudaError_t launch_dh_fwd(const LayerArgs& a, cudaStream_t s) {
    DhParams p = make_params(a);
    if (!make_maps(p, a, false)) return cudaErrorInvalidValue;
    p.o = (__nv_bfloat16*)a.out;
    p.lse = a.lse_out;
    const int smem = FwdSmem::total + 1024;
    void (*kernel)(DhParams) = a.window > 0 ? dh_fwd_kernel<true> : dh_fwd_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    before_launch(SAF_KERNEL_FWD, s);
    e = launch_ex(kernel, dim3((unsigned)p.nqb, (unsigned)(a.B * a.H)), dim3(kThreads), (size_t)smem, s,
                  true, 1, p);
    after_launch(SAF_KERNEL_FWD, s);
    return e;
}

cudaError_t launch_dh_bwd(const LayerArgs& a, cudaStream_t s) {
    DhParams p = make_params(a);
    if (!make_maps(p, a, true)) return cudaErrorInvalidValue;
    // (the accumulator of the d = 64 backward's dQ is not used here)
    p.sp = plan_sink_parts(a, 128, 128, 152, 16, a.dq_acc, (size_t)a.B * a.H * a.T * kHeadDim * sizeof(float));
    p.o_in = (const __nv_bfloat16*)a.o;
    p.dO = (const __nv_bfloat16*)a.dO;
    p.lse_in = a.lse;
    p.dq = (__nv_bfloat16*)a.dq;
    p.dk = (__nv_bfloat16*)a.dk;
    p.dv = (__nv_bfloat16*)a.dv;
    p.q_waits = dq_over_inputs(a, sizeof(__nv_bfloat16));
    const dim3 grid((unsigned)p.nqb, (unsigned)(a.B * a.H));
    before_launch(SAF_KERNEL_BWD_DELTA, s);
    cudaError_t e = launch_ex(dh_rowvec_kernel, grid, dim3(128), 0, s, true, 1, p);
    after_launch(SAF_KERNEL_BWD_DELTA, s);
    if (e == cudaSuccess) e = launch_narrow_d(a, s);
    if (e != cudaSuccess) return e;
    const int smem_kv = KvSmem::total + 1024, smem_q = QSmem::total + 1024;
    void (*kv_kernel)(DhParams) = a.window > 0 ? dh_bwd_kv_kernel<true> : dh_bwd_kv_kernel<false>;
    void (*q_kernel)(DhParams) = a.window > 0 ? dh_bwd_q_kernel<true> : dh_bwd_q_kernel<false>;
    e = cudaFuncSetAttribute(kv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_kv);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(q_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_q);
    if (e != cudaSuccess) return e;
    before_launch(SAF_KERNEL_BWD_KV, s);
    const unsigned levels = (unsigned)(p.nqb + p.sp.blocks * (p.sp.parts - 1));
    e = launch_ex(kv_kernel, dim3(levels, (unsigned)(a.B * p.Hkv)), dim3(kThreadsBwd),
                  (size_t)smem_kv, s, true, 1, p);
    after_launch(SAF_KERNEL_BWD_KV, s);
    if (e != cudaSuccess) return e;
    before_launch(SAF_KERNEL_BWD_Q, s);
    e = launch_ex(q_kernel, grid, dim3(kThreadsBwd), (size_t)smem_q, s, true, 1, p);
    after_launch(SAF_KERNEL_BWD_Q, s);
    if (e == cudaSuccess && p.sp.blocks > 0) e = launch_join_parts<__nv_bfloat16>(a, p.sp, s);
    return e;
}

}  // namespace saf
