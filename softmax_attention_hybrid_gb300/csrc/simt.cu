// fp32-arithmetic kernels of the hybrid attention layer (CUDA cores).
//
// These serve fp32 inputs, where the layer is computed in fp32 throughout
// (tensor cores have no fp32-input mode of full precision). They follow the
// same plan as the tensor-core path:
//   forward  : one launch; each program = (batch, head, 64-row query block);
//              the head's frozen flag picks ordinary online-softmax attention
//              (App. A.1 Eqs. 5-7, FlashAttention-2 tiling) or the frozen
//              pattern rebuilt from a, r and the precomputed log Z (§3.2 Eq. 3,
//              §3.3 "Fused computation"). Causal key blocks only.
//   backward : a key-block pass (dV for every head, dK for ordinary heads)
//              and a query-block pass (dQ for ordinary heads), as App. D.2
//              describes; frozen heads get dV = W^T dO and exact-zero dQ, dK.
//
// kWin instances serve ordinary heads with a sliding window and sinks: they visit the key
// (query) blocks that some row of the block sees and hide the other pairs.
//
// Tile: 16 RT own rows (query rows, or keys in the key-block pass) x 64 of the
// other axis, head dimension D = 64, 96 or 128, 256 threads, RT = 4. Thread
// (ty, tx), ty = tid / 16, tx = tid % 16, owns rows RT ty .. RT ty + RT - 1 and
// the columns tx, tx + 16, ... of the other axis (4 of them) or D / 16 columns
// of the head dimension, in vectors of 4 (2 at D = 96). Windowed calls that
// would leave most of the GPU idle take RT = 1: four times the programs, each
// with a quarter of the rows, and the same sums in the same order.
#include <math.h>

#include "saf_internal.h"

namespace saf {
namespace {

constexpr int kB = 64;          // rows per tile (queries and keys)
constexpr int kLd = kB + 4;     // padded fp32 row stride of a (key x query) tile
constexpr int kThreads = 256;
// A windowed launch of fewer blocks of 64 rows takes blocks of 16. A training step with a window of 100
// takes, with 64 and 16 rows: T 250, 4 heads, d 64 (16 blocks) 115 and 80 us; T 250, 16 heads over 4, d 96
// (64 and 16 blocks) 337 and 262; T 512, 12 heads, d 64 (96) 167 and 170; T 500, 12 heads, d 128 (96)
// 339 and 473; T 1000, 12 heads, d 64 (192) 334 and 343.
constexpr long long kFewBlocks = 76;
// floats per tile slot: every tile, (rows x D) or (key x query), fits one slot
template <int D>
__host__ __device__ constexpr int tile_floats() { return kB * ((D > kB ? D : kB) + 4); }

// rows r0 .. r0 + R - 1 of a [T, D] slice into shared memory, row stride D + 4
template <int D, int R>
__device__ __forceinline__ void load_tile(float* s, const float* g, int r0, int T) {
#pragma unroll 4
    for (int e = 4 * threadIdx.x; e < R * D; e += 4 * kThreads) {
        const int rr = e / D, c = e - rr * D;
        const int row = r0 + rr;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < T) x = *reinterpret_cast<const float4*>(g + (size_t)row * D + c);
        *reinterpret_cast<float4*>(s + rr * (D + 4) + c) = x;
    }
}

// Whether query i of an ordinary head sees key j <= i.
template <bool kWin>
__device__ __forceinline__ bool in_window(const LayerArgs& p, int i, int j) {
    return !kWin || i - j < p.window || j < p.sinks;
}

// dot[i][c] += x_i . y_c over D, x_i row RT ty + i of X, y_c row tx + 16 c of Y: each element is read
// once for all of its products, 16 bytes at a time. (Every sum runs over e in order.)
template <int D, int RT>
__device__ __forceinline__ void tile_dots(const float* X, const float* Y, int ty, int tx, float (&dot)[RT][4]) {
    constexpr int LdD = D + 4;
#pragma unroll 2
    for (int e = 0; e < D; e += 4) {
        float4 x[RT], y[4];
#pragma unroll
        for (int i = 0; i < RT; ++i) x[i] = *reinterpret_cast<const float4*>(X + (ty * RT + i) * LdD + e);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4*>(Y + (tx + 16 * c) * LdD + e);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                dot[i][c] = fmaf(x[i].x, y[c].x, dot[i][c]);
                dot[i][c] = fmaf(x[i].y, y[c].y, dot[i][c]);
                dot[i][c] = fmaf(x[i].z, y[c].z, dot[i][c]);
                dot[i][c] = fmaf(x[i].w, y[c].w, dot[i][c]);
            }
    }
}

// A thread's columns of the head dimension: NV vectors of VW, vector u at column at(u).
template <int D>
struct Cols {
    static constexpr int VW = D == 96 ? 2 : 4, NV = D / 16 / VW;
    static __device__ __forceinline__ int at(int u, int tx) { return VW * (tx + 16 * u); }
    static __device__ __forceinline__ void load(float* x, const float* row, int tx) {   // row of a tile
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if constexpr (VW == 4) {
                const float4 y = *reinterpret_cast<const float4*>(row + at(u, tx));
                x[4 * u] = y.x, x[4 * u + 1] = y.y, x[4 * u + 2] = y.z, x[4 * u + 3] = y.w;
            } else {
                const float2 y = *reinterpret_cast<const float2*>(row + at(u, tx));
                x[2 * u] = y.x, x[2 * u + 1] = y.y;
            }
        }
    }
    static __device__ __forceinline__ void store(float* row, const float* x, float f, int tx) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int e = 0; e < VW; ++e) row[at(u, tx) + e] = x[VW * u + e] * f;
    }
};

// acc[i][c] += sum over the 64 rows j of Y of w_ij Y[j][column c], w_ij row RT ty + i of W (stride
// kLd); j in order.
template <int D, int RT>
__device__ __forceinline__ void tile_sums(const float* W, const float* Y, int ty, int tx, float (&acc)[RT][D / 16]) {
    constexpr int NC = D / 16, LdD = D + 4;
#pragma unroll 2
    for (int j = 0; j < kB; j += 4) {
        float w[RT][4], y[4][NC];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(W + (ty * RT + i) * kLd + j);
            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) Cols<D>::load(y[u], Y + (j + u) * LdD, tx);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(w[i][u], y[u][c], acc[i][c]);
    }
}

__device__ __forceinline__ float quad16_max(float x) {
    for (int o = 1; o < 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float quad16_sum(float x) {
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Programmatic dependent launch. The next launch's blocks may come in early only where this one
// leaves every block an SM of its own: beside a larger grid's last blocks they would crowd two to
// an SM while others idle (H8/Hkv1 d64, T2048, forward and backward: 852 us so, 668 us otherwise;
// H4 T250, window 100: 60 us with it, 80 us without).
constexpr int kSms = 152;   // GB300
__device__ __forceinline__ bool one_block_an_sm() { return gridDim.x * gridDim.y <= kSms; }
__device__ __forceinline__ void begin_block() {
    grid_dep_wait();
    if (one_block_an_sm()) grid_dep_launch();
}

// ---------------------------------------------------------------------------
// Forward. Grid (ceil(T / 16 RT), B*H).
// ---------------------------------------------------------------------------
template <int D, bool kWin, int RT>
__global__ void __launch_bounds__(kThreads) fwd_kernel(LayerArgs p) {
    begin_block();
    extern __shared__ float sm[];
    float* Qs = sm;
    constexpr int NC = D / 16, kT = tile_floats<D>(), kR = 16 * RT;
    float* Ks = Qs + kT;
    float* Vs = Ks + kT;
    float* Ps = Vs + kT;

    const int T = p.T;
    const int qb = blockIdx.x, bh = blockIdx.y, h = bh % p.H;
    const bool frozen = head_frozen(p.mask, h);
    const size_t base = (size_t)bh * T * D;
    // key/value slice of this query head (grouped-query layout: head h reads h / (H / Hkv))
    const size_t kvbase = ((size_t)(bh / p.H) * p.Hkv + h / (p.H / p.Hkv)) * T * D;
    const float* q = (const float*)p.q + base;
    const float* k = (const float*)p.k + kvbase;
    const float* v = (const float*)p.v + kvbase;
    const float* a = p.a + (size_t)h * p.ld_prior;
    const float* r = p.r + (size_t)h * p.ld_prior;
    const int q0 = qb * kR;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const float scale = 1.f / sqrtf((float)D);

    if (!frozen) load_tile<D, kR>(Qs, q, q0, T);
    float m[RT], l[RT], lzr[RT], acc[RT][NC];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = q0 + ty * RT + i;
        m[i] = -INFINITY;
        l[i] = 0.f;
        lzr[i] = (frozen && row < T) ? p.lz[(size_t)h * T + row] : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = 0.f;
    }

    const KeyBlocks<kWin> blocks(q0, (q0 + kR - 1) / kB, kWin && frozen ? T : p.window, p.sinks, kB);
    for (int jj = 0; jj < blocks.n; ++jj) {
        const int kb = blocks.id(jj);
        __syncthreads();
        if (!frozen) load_tile<D, kB>(Ks, k, kb * kB, T);
        load_tile<D, kB>(Vs, v, kb * kB, T);
        __syncthreads();
        float s[RT][4], dot[RT][4] = {};
        if (!frozen) tile_dots<D, RT>(Qs, Ks, ty, tx, dot);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = q0 + ty * RT + i;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int key = kb * kB + tx + 16 * c;
                if (frozen) {
                    // W(i, j) = exp(a[j] + r[i-j] - log Z(i)), causal (Eq. 3)
                    const bool ok = key <= row && row < T;
                    s[i][c] = ok ? expf(a[key] + r[row - key] - lzr[i]) : 0.f;
                } else {
                    s[i][c] = (key <= row && key < T && in_window<kWin>(p, row, key)) ? dot[i][c] * scale : -INFINITY;
                }
            }
        }
        if (!frozen) {
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
                const float mnew = fmaxf(m[i], quad16_max(mx));
                // a row of a windowed layer that has seen no key yet: any finite reference
                const float ref = kWin && mnew == -INFINITY ? 0.f : mnew;
                const float corr = expf(m[i] - ref);
                float ls = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[i][c] = expf(s[i][c] - ref);
                    ls += s[i][c];
                }
                l[i] = l[i] * corr + quad16_sum(ls);
                m[i] = mnew;
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[i][c] *= corr;
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) Ps[(ty * RT + i) * kLd + tx + 16 * c] = s[i][c];
        __syncthreads();
        tile_sums<D, RT>(Ps, Vs, ty, tx, acc);
    }

    float* o = (float*)p.out + base;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = q0 + ty * RT + i;
        if (row >= T) continue;
        Cols<D>::store(o + (size_t)row * D, acc[i], frozen ? 1.f : 1.f / l[i], tx);
        if (tx == 0) p.lse_out[(size_t)bh * T + row] = frozen ? lzr[i] : m[i] + logf(l[i]);
    }
}

// ---------------------------------------------------------------------------
// Backward, key-block pass. Grid (ceil(T / 16 RT), B*Hkv). Program owns keys
// k0 .. k0 + 16 RT - 1 of one key/value slice; loops over the query heads that share it
// (grouped-query layout; one head in the multi-head layer) and, for each, over
// query blocks qb >= kb, so that the slice's dV and dK are group sums formed
// without atomics. Thread rows = keys. With a window the grid begins with the parts of
// the key blocks that hold sinks (SinkParts), each of which has a run of the query blocks
// (H8/Hkv2 d64, T4096, window 512, 16 sinks, forward and backward: 2979 us whole, 1047 us so).
// ---------------------------------------------------------------------------
template <int D, bool kWin, int RT>
__global__ void __launch_bounds__(kThreads) bwd_kv_kernel(LayerArgs p, SinkParts sp) {
    begin_block();
    extern __shared__ float sm[];
    constexpr int NC = D / 16, kT = tile_floats<D>(), kR = 16 * RT;
    float* Ks = sm;
    float* Vs = Ks + kT;
    float* Qs = Vs + kT;
    float* dOs = Qs + kT;
    float* Pt = dOs + kT;    // P^T  [key][query]
    float* dSt = Pt + kT;    // dS^T [key][query]
    __shared__ float rowstat[kB];  // lse (ordinary) or log Z (frozen) per query
    __shared__ float rowD[kB];

    const int T = p.T;
    const int G = p.H / p.Hkv;
    const int bkv = blockIdx.y, b = bkv / p.Hkv, hk = bkv % p.Hkv;
    bool any_ordinary = false;
    for (int gi = 0; gi < G; ++gi) any_ordinary |= !head_frozen(p.mask, hk * G + gi);
    const int n_parts = kWin ? sp.blocks * sp.parts : 0, x = blockIdx.x;
    const bool in_parts = kWin && x < n_parts, split = in_parts && any_ordinary;
    const int kb = in_parts ? x / sp.parts : x - n_parts + (kWin ? sp.blocks : 0);
    const int part = in_parts ? x % sp.parts : 0;
    SinkParts::Range run{0, 0};
    if (split) run = sp.range(kb, T, part);
    if (in_parts && (split ? run.n == 0 : part > 0)) return;   // (a frozen group's block is not split)
    const size_t kvbase = (size_t)bkv * T * D;
    const float* k = (const float*)p.k + kvbase;
    const float* v = (const float*)p.v + kvbase;
    const int k0 = kb * kR;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const float scale = 1.f / sqrtf((float)D);
    if (any_ordinary) load_tile<D, kR>(Ks, k, k0, T);
    load_tile<D, kR>(Vs, v, k0, T);
    float dv[RT][NC], dk[RT][NC];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) dv[i][c] = dk[i][c] = 0.f;

    const int nqb = (T + kB - 1) / kB;
    for (int gi = 0; gi < G; ++gi) {
    const int h = hk * G + gi, bh = b * p.H + h;
    const bool frozen = head_frozen(p.mask, h);
    const size_t base = (size_t)bh * T * D;
    const float* q = (const float*)p.q + base;
    const float* dO = (const float*)p.dO + base;
    const float* a = p.a + (size_t)h * p.ld_prior;
    const float* r = p.r + (size_t)h * p.ld_prior;
    // query blocks from the one of my first key on; with a window to the one of the last query that
    // sees my last key
    int q_end = nqb;
    if (kWin && !frozen && k0 >= p.sinks) {
        const long long last = ((long long)k0 + kR - 1 + p.window - 1) / kB;
        q_end = last < nqb - 1 ? (int)last + 1 : nqb;
    }
    int qb = k0 / kB;
    if (split) {
        qb = run.first;
        q_end = run.first + run.n;
    }
    for (; qb < q_end; ++qb) {
        const int q0 = qb * kB;
        __syncthreads();
        if (!frozen) load_tile<D, kB>(Qs, q, q0, T);
        load_tile<D, kB>(dOs, dO, q0, T);
        if (tid < kB) {
            const int qi = q0 + tid;
            if (frozen) {
                rowstat[tid] = qi < T ? p.lz[(size_t)h * T + qi] : 0.f;
            } else {
                rowstat[tid] = qi < T ? p.lse[(size_t)bh * T + qi] : 0.f;
                rowD[tid] = qi < T ? p.delta[(size_t)bh * T + qi] : 0.f;
            }
        }
        __syncthreads();
        float dot[RT][4] = {}, dpt[RT][4] = {};
        if (!frozen) {
            tile_dots<D, RT>(Ks, Qs, ty, tx, dot);
            tile_dots<D, RT>(Vs, dOs, ty, tx, dpt);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int key = k0 + ty * RT + i;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int qq = tx + 16 * c;
                const int qi = q0 + qq;
                const bool ok = key <= qi && qi < T;
                float pt, dst = 0.f;
                if (frozen) {
                    pt = ok ? expf(a[key] + r[qi - key] - rowstat[qq]) : 0.f;
                } else {
                    pt = ok && in_window<kWin>(p, qi, key) ? expf(fmaf(dot[i][c], scale, -rowstat[qq])) : 0.f;
                    dst = pt * (dpt[i][c] - rowD[qq]);
                }
                Pt[(ty * RT + i) * kLd + qq] = pt;
                dSt[(ty * RT + i) * kLd + qq] = dst;
            }
        }
        __syncthreads();
        tile_sums<D, RT>(Pt, dOs, ty, tx, dv);
        if (!frozen) tile_sums<D, RT>(dSt, Qs, ty, tx, dk);
    }
    }

    if constexpr (kWin) {
        if (split) {
            float* sums = sp.at(bkv, kb, part, 0, D);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                Cols<D>::store(sums + (ty * RT + i) * D, dv[i], 1.f, tx);
                Cols<D>::store(sums + (kR + ty * RT + i) * D, dk[i], 1.f, tx);
            }
            return;
        }
    }
    float* dvp = (float*)p.dv + kvbase;
    float* dkp = (float*)p.dk + kvbase;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int key = k0 + ty * RT + i;
        if (key >= T) continue;
        Cols<D>::store(dvp + (size_t)key * D, dv[i], 1.f, tx);
        if (!any_ordinary)
#pragma unroll
            for (int c = 0; c < NC; ++c) dk[i][c] = 0.f;
        Cols<D>::store(dkp + (size_t)key * D, dk[i], scale, tx);
    }
}

// ---------------------------------------------------------------------------
// Backward, query-block pass (dQ). Grid (ceil(T / 16 RT), B*H). Frozen heads
// write zeros. beside: the pass reads nothing that the key-block pass before it writes, and runs
// beside it; every block of that launch has begun, after its own grid_dep_wait(), before one of
// this runs, and block (0, 0) waits for it at its end, so that this launch's completion implies
// that one's. (Where both grids together leave every block an SM of its own, and dq neither holds
// parts' sums nor lies over q or dO, which the key-block pass reads.)
// ---------------------------------------------------------------------------
template <int D, bool kWin, int RT>
__global__ void __launch_bounds__(kThreads) bwd_q_kernel(LayerArgs p, bool beside) {
    if (!beside) grid_dep_wait();
    if (one_block_an_sm()) grid_dep_launch();
    extern __shared__ float sm[];
    constexpr int NC = D / 16, kT = tile_floats<D>(), kR = 16 * RT;
    float* Qs = sm;
    float* dOs = Qs + kT;
    float* Ks = dOs + kT;
    float* Vs = Ks + kT;
    float* dSs = Vs + kT;

    const int T = p.T;
    const int qb = blockIdx.x, bh = blockIdx.y, h = bh % p.H;
    const bool frozen = head_frozen(p.mask, h);
    const size_t base = (size_t)bh * T * D;
    float* dq = (float*)p.dq + base;
    const int q0 = qb * kR;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    if (frozen) {
        for (int e = tid; e < kR * D; e += kThreads) {
            const int row = q0 + e / D;
            if (row < T) dq[(size_t)row * D + e % D] = 0.f;
        }
        if (beside && blockIdx.x == 0 && blockIdx.y == 0) grid_dep_wait();
        return;
    }
    const size_t kvbase = ((size_t)(bh / p.H) * p.Hkv + h / (p.H / p.Hkv)) * T * D;
    const float* q = (const float*)p.q + base;
    const float* k = (const float*)p.k + kvbase;
    const float* v = (const float*)p.v + kvbase;
    const float* dO = (const float*)p.dO + base;
    const float scale = 1.f / sqrtf((float)D);

    load_tile<D, kR>(Qs, q, q0, T);
    load_tile<D, kR>(dOs, dO, q0, T);
    float lse[RT], Dr[RT], acc[RT][NC];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = q0 + ty * RT + i;
        lse[i] = row < T ? p.lse[(size_t)bh * T + row] : 0.f;
        Dr[i] = row < T ? p.delta[(size_t)bh * T + row] : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = 0.f;
    }
    const KeyBlocks<kWin> blocks(q0, (q0 + kR - 1) / kB, p.window, p.sinks, kB);
    for (int jj = 0; jj < blocks.n; ++jj) {
        const int kb = blocks.id(jj);
        __syncthreads();
        load_tile<D, kB>(Ks, k, kb * kB, T);
        load_tile<D, kB>(Vs, v, kb * kB, T);
        __syncthreads();
        float dot[RT][4] = {}, dp[RT][4] = {};
        tile_dots<D, RT>(Qs, Ks, ty, tx, dot);
        tile_dots<D, RT>(dOs, Vs, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = q0 + ty * RT + i;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int key = kb * kB + tx + 16 * c;
                const bool ok = key <= row && row < T && in_window<kWin>(p, row, key);
                const float pij = ok ? expf(dot[i][c] * scale - lse[i]) : 0.f;
                dSs[(ty * RT + i) * kLd + tx + 16 * c] = pij * (dp[i][c] - Dr[i]);
            }
        }
        __syncthreads();
        tile_sums<D, RT>(dSs, Ks, ty, tx, acc);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = q0 + ty * RT + i;
        if (row < T) Cols<D>::store(dq + (size_t)row * D, acc[i], scale, tx);
    }
    if (beside && blockIdx.x == 0 && blockIdx.y == 0) grid_dep_wait();
}

template <int D, int RT, typename K, typename... Args>
cudaError_t launch(K kernel, int id, int tiles, const LayerArgs& p, cudaStream_t s, int slices, int extra, Args... args) {
    const int smem = tiles * tile_floats<D>() * (int)sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    dim3 grid((p.T + 16 * RT - 1) / (16 * RT) + extra, slices);
    before_launch(id, s);
    e = launch_ex(kernel, grid, dim3(kThreads), (size_t)smem, s, true, 1, p, args...);
    after_launch(id, s);
    return e;
}

template <int D, bool kWin, int RT>
cudaError_t fwd_d(const LayerArgs& p, cudaStream_t s) {
    return launch<D, RT>(fwd_kernel<D, kWin, RT>, SAF_KERNEL_FWD, 4, p, s, p.B * p.H, 0);
}

// parts: whether dq was used for the parts' sums
template <int D, bool kWin, int RT>
cudaError_t bwd_kv_d(const LayerArgs& p, cudaStream_t s, bool* parts) {
    // dq serves as scratch until the query-block pass writes it, unless it lies over what is read till
    // then; two blocks of threads an SM
    const size_t scratch = dq_over_inputs(p, sizeof(float)) ? 0 : (size_t)p.B * p.H * p.T * p.d * sizeof(float);
    const SinkParts sp = plan_sink_parts(p, 16 * RT, kB, 304, 4, p.dq, scratch);
    const cudaError_t e = launch<D, RT>(bwd_kv_kernel<D, kWin, RT>, SAF_KERNEL_BWD_KV, 6, p, s, p.B * p.Hkv,
                                        sp.blocks * (sp.parts - 1), sp);
    *parts = sp.blocks > 0;
    return e == cudaSuccess && *parts ? launch_join_parts<float>(p, sp, s) : e;
}

template <int D, bool kWin, int RT>
cudaError_t bwd_q_d(const LayerArgs& p, cudaStream_t s, bool beside) {
    return launch<D, RT>(bwd_q_kernel<D, kWin, RT>, SAF_KERNEL_BWD_Q, 5, p, s, p.B * p.H, 0, beside);
}

template <bool kWin, int RT>
cudaError_t fwd_f32(const LayerArgs& p, cudaStream_t s) {
    switch (p.d) {
        case 96: return fwd_d<96, kWin, RT>(p, s);
        case 128: return fwd_d<128, kWin, RT>(p, s);
        default: return fwd_d<64, kWin, RT>(p, s);
    }
}

template <bool kWin, int RT>
cudaError_t bwd_kv_f32(const LayerArgs& p, cudaStream_t s, bool* parts) {
    switch (p.d) {
        case 96: return bwd_kv_d<96, kWin, RT>(p, s, parts);
        case 128: return bwd_kv_d<128, kWin, RT>(p, s, parts);
        default: return bwd_kv_d<64, kWin, RT>(p, s, parts);
    }
}

template <bool kWin, int RT>
cudaError_t bwd_q_f32(const LayerArgs& p, cudaStream_t s, bool beside) {
    switch (p.d) {
        case 96: return bwd_q_d<96, kWin, RT>(p, s, beside);
        case 128: return bwd_q_d<128, kWin, RT>(p, s, beside);
        default: return bwd_q_d<64, kWin, RT>(p, s, beside);
    }
}

// Whether blocks of 64 rows of `slices` slices leave most SMs without a program.
bool few_blocks(const LayerArgs& p, int slices) { return (long long)((p.T + kB - 1) / kB) * slices < kFewBlocks; }

}  // namespace

cudaError_t launch_simt_fwd(const LayerArgs& p, cudaStream_t s) {
    if (p.window == 0) return fwd_f32<false, 4>(p, s);
    return few_blocks(p, p.B * p.H) ? fwd_f32<true, 1>(p, s) : fwd_f32<true, 4>(p, s);
}

cudaError_t launch_simt_bwd(const LayerArgs& p, cudaStream_t s) {
    cudaError_t e;
    bool parts = false;
    if (p.window == 0) e = bwd_kv_f32<false, 4>(p, s, &parts);
    else e = few_blocks(p, p.B * p.Hkv) ? bwd_kv_f32<true, 1>(p, s, &parts) : bwd_kv_f32<true, 4>(p, s, &parts);
    if (e != cudaSuccess) return e;
    const auto blocks = [&](int slices) {
        const int rows = p.window > 0 && few_blocks(p, slices) ? 16 : 64;
        return (long long)((p.T + rows - 1) / rows) * slices;
    };
    const bool beside = !parts && !dq_over_inputs(p, sizeof(float)) && blocks(p.B * p.Hkv) + blocks(p.B * p.H) <= kSms;
    if (p.window == 0) return bwd_q_f32<false, 4>(p, s, beside);
    return few_blocks(p, p.B * p.H) ? bwd_q_f32<true, 1>(p, s, beside) : bwd_q_f32<true, 4>(p, s, beside);
}

}  // namespace saf
