// Paged attention over 8-bit caches for fp32 q and o, on the CUDA cores (see paged.h for the split).
//
// An item holds up to 8 query rows and walks tiles of 128 keys, of which the next one's codes are copied
// into shared memory as they lie in the cache (cp.async) while this one is used:
//   scores   a thread per key, for all rows: sum q c over its codes c, two products to an instruction, then the key's
//            scale. q's rows are read from shared memory (the same 16 bytes for every lane), scaled by a
//            power of two to [1, 2) for their largest, so that sums over codes up to 448 do not overflow
//            where q k would not. A frozen row's logit is a[j] + r[i - j] instead, loaded before the tile is there.
//   softmax  base 2, a running maximum per row for the whole block: a tile whose scores stay below m + 4 leaves it
//            (one barrier with an OR); each thread keeps its own part of the sum
//   output   a thread per 4 columns of d and every 128 / (d / 4)-th key: weight times the value's scale (rounded once),
//            times the codes, for all rows; the threads of a column are added at the end
// A code is turned into fp32 once for all rows (exactly). Everything else is fp32.
// Blocks of 2, 4, 6 or 8 rows: instructions bound the kernel, and their number goes with the rows.
// (Five tokens each of four sequences of up to 2000, 16 heads of their own, d 96: 19.1 us, 0.86 TB/s. Tiles of 32 keys
// written to shared memory as fp32, a warp for every two rows: 39.6 us.)
#include <cuda_fp8.h>

#include "paged_tc.cuh"

namespace saf {
namespace {

using namespace paged_tc;

constexpr int kThreads = 128;
constexpr int TK = kQ8SimtTile;
static_assert(TK == kThreads, "a thread per key");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 4.0f;                // scores may pass the maximum by this much (base 2)
constexpr float kNoMax = -3.402823466e38f;    // a row that has seen no key yet: no finite score is below it

template <int D, int R>
struct Smem {
    static constexpr int k_pitch = D + 16;    // (16 more bytes: 8 keys' 16-byte reads lie in other banks)
    static constexpr int quads = D / 4, groups = kThreads / quads;
    union {
        struct {
            uint8_t k[2][TK * k_pitch];
            uint8_t v[2][TK * D];
        };
        float sums[groups][R][D];             // at the end
    };
    float q[R][D];
    float w[TK][R];                           // weights of the tile, times the values' scales
    long long at[2][TK];                      // a key's row in the caches, -1: nothing to read
    alignas(16) float scale[R], m[R], fall[R];   // of the scores; running maxima; 2^(old maximum - new one)
    float part[4][R];
    int pos[R], head[R], out[R];              // out: the row's place in o, -1: none
    int frozen[R];
};

__device__ __forceinline__ void copy16(void* dst, const uint8_t* src, bool have) {   // zeros without a source
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(have ? 16 : 0)
                 : "memory");
}

// Two codes (the low 16 bits) as fp32: exact.
__device__ __forceinline__ float2 codes2(uint32_t codes) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3)));
}

// Whether any thread says so; a barrier of the block.
__device__ __forceinline__ bool any_thread(bool x) { return __syncthreads_or(x) != 0; }

// Largest of a warp's values (NaN left out), by integers that have the order of the floats.
__device__ __forceinline__ float warp_max(float x) {
    int k = x == x ? __float_as_int(x) : (int)0xff800000;
    k ^= (k >> 31) & 0x7fffffff;
    k = __reduce_max_sync(0xffffffffu, k);
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// R rows of a row of shared memory, in pairs.
template <int R>
__device__ __forceinline__ void read_rows(const float* src, float2* x) {
    static_assert(R % 2 == 0, "pairs");
    if constexpr (R % 4 == 0) {
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            const float4 y = *reinterpret_cast<const float4*>(src + r);
            x[r / 2] = make_float2(y.x, y.y);
            x[r / 2 + 1] = make_float2(y.z, y.w);
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; r += 2) x[r / 2] = *reinterpret_cast<const float2*>(src + r);
    }
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, paged_q8_simt_ctas(D)) paged_q8_simt_kernel(const __grid_constant__ PagedArgs p) {
    using S = Smem<D, R>;
    extern __shared__ __align__(16) uint8_t raw[];
    S& sm = *reinterpret_cast<S*>(raw);
    grid_dep_wait();
    grid_dep_launch();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const PagedItem it = paged_item(p, blockIdx.x);
    const PagedBlock block = paged_block(p, it);
    // every warp finds the rows for itself, a lane each
    const PagedRow row = paged_place(p, it, block, lane);
    int i = -1;
    if (row.there) {
        int c;
        bool bad;
        const int n = paged_tokens(p, row.b, &c, &bad);
        if (row.t < n) i = p.P + c + row.t;
        // each sequence's counts are checked once
        if (bad && t == 0 && it.part == 1 && it.chunk == 0 && it.rb == 0 && it.hk == 0) atomicOr(p.status, kStatusPage);
    }
    const int imin = __reduce_min_sync(0xffffffffu, i >= 0 ? i : 0x7fffffff), imax = __reduce_max_sync(0xffffffffu, i);
    const bool any_ord = __ballot_sync(0xffffffffu, i >= 0 && !row.frozen) != 0;
    const uint32_t fz = __ballot_sync(0xffffffffu, i >= 0 && row.frozen);
    const uint32_t ord = __ballot_sync(0xffffffffu, i >= 0 && !row.frozen);
    const PagedRange g = paged_range(p, it, imin, imax, fz != 0 || p.window == 0);
    const int e0 = min(it.chunk * p.per_chunk[it.part], g.n), e1 = min(e0 + p.per_chunk[it.part], g.n);
    const int off = it.part ? p.P : 0;
    if (t < R) {
        sm.pos[t] = i;
        sm.head[t] = row.h;
        sm.out[t] = row.there ? (int)paged_out_row(p, row) : -1;
        sm.frozen[t] = row.frozen;
        sm.m[t] = kNoMax;
        sm.scale[t] = 0.f;
    }
    const uint8_t* kc = (const uint8_t*)p.k_cache;
    const uint8_t* vc = (const uint8_t*)p.v_cache;
    // where key t of tile e lies; keys that no row sees, and those of pages outside the cache, are read as zeros
    auto look = [&](int e) -> long long {
        if (e >= e1) return -1;
        const int x = paged_tile(g, e) * TK + t;
        if (!(x < g.hi && (x >= g.lo || x < g.sink))) return -1;
        const int pg = paged_page(p, it, x);
        if (pg < 0) {
            atomicOr(p.status, kStatusPage);
            return -1;
        }
        return (((long long)pg * p.Hkv + it.hk) << p.page_log2) + (x & ((1 << p.page_log2) - 1));
    };
    auto copy_tile = [&](int s) {
#pragma unroll
        for (int u = t; u < TK * (D / 16); u += kThreads) {
            const int kk = u / (D / 16), c = 16 * (u - kk * (D / 16));
            const long long at = sm.at[s][kk];
            const long long from = at < 0 ? 0 : at * D + c;
            if (any_ord) copy16(&sm.k[s][kk * S::k_pitch + c], kc + from, at >= 0);
            copy16(&sm.v[s][kk * D + c], vc + from, at >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // my key of this tile and of the next, and their scales
    long long mine = look(e0), next = look(e0 + 1);
    float ks = 0.f, vs = 0.f;
    if (mine >= 0) {
        if (any_ord) ks = __ldg(p.k_scale + mine);
        vs = __ldg(p.v_scale + mine);
    }
    sm.at[0][t] = mine;
    sm.at[1][t] = next;
    __syncthreads();
    if (e0 < e1) copy_tile(0);
    if (any_ord && e0 < e1)
        for (int r = warp; r < R; r += 4) {   // a warp a row
            if (!((ord >> r) & 1u)) {
                if (lane < D / 4) *reinterpret_cast<float4*>(&sm.q[r][4 * lane]) = make_float4(0.f, 0.f, 0.f, 0.f);
                continue;
            }
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < D / 4) x = *reinterpret_cast<const float4*>((const float*)p.q + (size_t)sm.out[r] * D + 4 * lane);
            uint32_t top = max(max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu),
                               max(__float_as_uint(x.z) & 0x7fffffffu, __float_as_uint(x.w) & 0x7fffffffu));
            top = __reduce_max_sync(0xffffffffu, top);
            // 2^e <= the largest < 2^(e + 1); a row with an infinity or a NaN stays as it is
            int e = (int)(top >> 23) - 127;
            e = top >= 0x7f800000u ? 0 : e < -120 ? -120 : e > 120 ? 120 : e;
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
            if (lane < D / 4) *reinterpret_cast<float4*>(&sm.q[r][4 * lane]) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
            if (lane == 0) sm.scale[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
        }

    const int quad = t % S::quads, grp = t / S::quads;   // my columns and keys of the output
    float2 acc[4][R / 2];
    float l[R];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int r = 0; r < R / 2; ++r) acc[c][r] = make_float2(0.f, 0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) l[r] = 0.f;

    for (int e = e0, n = 0; e < e1; ++e, ++n) {
        const int s = n & 1;
        const int x = paged_tile(g, e) * TK + t, j = off + x;   // my key's slot and position
        float sc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sc[r] = -INFINITY;
            if ((fz >> r) & 1u) {
                const int pi = sm.pos[r];
                const size_t h = (size_t)sm.head[r] * p.ld;
                if (j <= pi) sc[r] = (__ldg(p.a + h + j) + __ldg(p.r + h + pi - j)) * kLog2e;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();   // the tile is there, and everyone is done with the one before
        const bool live = mine >= 0;
        const float ks1 = ks, vs1 = vs;
        mine = next;
        if (e + 1 < e1) {
            copy_tile(s ^ 1);
            ks = vs = 0.f;
            if (mine >= 0) {
                if (any_ord) ks = __ldg(p.k_scale + mine);
                vs = __ldg(p.v_scale + mine);
            }
        }
        next = look(e + 2);
        if (any_ord) {
            float2 dot[R];
#pragma unroll
            for (int r = 0; r < R; ++r) dot[r] = make_float2(0.f, 0.f);
#pragma unroll 2
            for (int c = 0; c < D; c += 16) {
                const uint4 y = *reinterpret_cast<const uint4*>(&sm.k[s][t * S::k_pitch + c]);
                const uint32_t wd[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float2 k0 = codes2(wd[b] & 0xffffu), k1 = codes2(wd[b] >> 16);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float4 q = *reinterpret_cast<const float4*>(&sm.q[r][c + 4 * b]);
                        dot[r] = ffma2(make_float2(q.x, q.y), k0, dot[r]);
                        dot[r] = ffma2(make_float2(q.z, q.w), k1, dot[r]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int pi = sm.pos[r];
                const bool sees = ((ord >> r) & 1u) && j <= pi && (p.window == 0 || pi - j < p.window || j < p.sinks);
                if (sees) sc[r] = (dot[r].x + dot[r].y) * (ks1 * sm.scale[r]);
            }
        }
        float past = 0.f;   // by how much a score passes its row's maximum (a NaN does not)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!live) sc[r] = -INFINITY;
            past = fmaxf(past, sc[r] - sm.m[r]);
        }
        if (any_thread(past > kSlack)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float mx = warp_max(sc[r]);
                if (lane == 0) sm.part[warp][r] = mx;
            }
            __syncthreads();
            if (t < R) {
                const float old = sm.m[t];
                const float now = fmaxf(fmaxf(fmaxf(sm.part[0][t], sm.part[1][t]), fmaxf(sm.part[2][t], sm.part[3][t])), old);
                sm.m[t] = now;
                sm.fall[t] = now > old ? exp2f(old - now) : 1.f;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r) l[r] *= sm.fall[r];
#pragma unroll
            for (int r = 0; r < R; r += 2) {
                const float2 f = *reinterpret_cast<const float2*>(&sm.fall[r]);
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c][r / 2] = fmul2(acc[c][r / 2], f);
            }
        }
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            const float y0 = exp2f(sc[r] - sm.m[r]), y1 = exp2f(sc[r + 1] - sm.m[r + 1]);
            l[r] += y0;
            l[r + 1] += y1;
            *reinterpret_cast<float2*>(&sm.w[t][r]) = make_float2(y0 * vs1, y1 * vs1);
        }
        __syncthreads();
        sm.at[s][t] = next;   // (this tile's copies were issued before it began)
        if (grp < S::groups) {
#pragma unroll 4
            for (int kk = grp; kk < TK; kk += S::groups) {
                const uint32_t y = *reinterpret_cast<const uint32_t*>(&sm.v[s][kk * D + 4 * quad]);
                float2 w[R / 2];
                read_rows<R>(sm.w[kk], w);
                const float2 v0 = codes2(y & 0xffffu), v1 = codes2(y >> 16);
                const float v[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int r = 0; r < R / 2; ++r) acc[c][r] = ffma2(w[r], make_float2(v[c], v[c]), acc[c][r]);
            }
        }
    }

#pragma unroll
    for (int r = 0; r < R; ++r) {
        for (int o = 16; o; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        if (lane == 0) sm.part[warp][r] = l[r];
    }
    __syncthreads();   // (the tiles are no longer read)
    if (grp < S::groups) {
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            *reinterpret_cast<float4*>(&sm.sums[grp][2 * r][4 * quad]) =
                make_float4(acc[0][r].x, acc[1][r].x, acc[2][r].x, acc[3][r].x);
            *reinterpret_cast<float4*>(&sm.sums[grp][2 * r + 1][4 * quad]) =
                make_float4(acc[0][r].y, acc[1][r].y, acc[2][r].y, acc[3][r].y);
        }
    }
    __syncthreads();
    const int split = it.part ? p.chunks[0] + it.chunk : it.chunk;
    if (t >= D) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (sm.out[r] < 0) continue;
        const size_t at = (size_t)sm.out[r];
        const float lr = (sm.part[0][r] + sm.part[1][r]) + (sm.part[2][r] + sm.part[3][r]);
        float o = 0.f;
#pragma unroll
        for (int k = 0; k < S::groups; ++k) o += sm.sums[k][r][t];
        if (p.nsplit == 1) {
            ((float*)p.o)[at * D + t] = lr != 0.f ? o / lr : 0.f;
            if (t == 0) p.lse[at] = lr != 0.f ? (sm.m[r] + log2f(lr)) * kLn2 : -INFINITY;
        } else {
            p.po[(at * p.nsplit + split) * D + t] = o;
            if (t == 0) p.ml[at * p.nsplit + split] = make_float2(lr != 0.f ? sm.m[r] : -INFINITY, lr);
        }
    }
}

template <int D, int R>
cudaError_t launch_r(const PagedArgs& p, cudaStream_t s) {
    const size_t smem = sizeof(Smem<D, R>);
    const cudaError_t e =
        cudaFuncSetAttribute(paged_q8_simt_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_ex(paged_q8_simt_kernel<D, R>, dim3(p.items), dim3(kThreads), smem, s, true, 1, p);
}

template <int D>
cudaError_t launch_d(const PagedArgs& p, cudaStream_t s) {
    const int rows = p.rows[0] > p.rows[1] ? p.rows[0] : p.rows[1];
    switch (rows) {
        case 2: return launch_r<D, 2>(p, s);
        case 4: return launch_r<D, 4>(p, s);
        case 6: return launch_r<D, 6>(p, s);
        default: return launch_r<D, 8>(p, s);
    }
}

}  // namespace

cudaError_t launch_paged_q8_simt(const PagedArgs& p, cudaStream_t s) {
    switch (p.d) {
        case 96: return launch_d<96>(p, s);
        case 128: return launch_d<128>(p, s);
        default: return launch_d<64>(p, s);
    }
}

}  // namespace saf
