// Paged attention of fp32 caches on the CUDA cores (see paged.h for the split).
//
// An item holds up to 8 query rows and walks its tiles of 32 keys, of which the next one is
// copied into shared memory (cp.async) while this one is used:
//   scores   a warp per two rows, a lane per key: the products from shared memory, 16 bytes at a
//            time; a frozen row's logit is a[j] + r[i - j] instead, loaded before the tile is there
//   softmax  base 2, the running maximum per row; each lane keeps its own part of the sum
//   output   a thread per column of d: the rows' weights (broadcast) times the column's values
// Bound by shared memory and the cache's bytes alike: a tile at d = 96 is 24 KB, 1000 cycles of an
// SM's share of the memory, and about as many of shared-memory reads.
#include "paged.h"

namespace saf {
namespace {

constexpr int kThreads = 128;
constexpr int R = kSimtRows, TK = kSimtTile;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
    float q[R][D];
    float k[2][TK][D + 4];   // 16 more bytes a row: 8 keys' 16-byte reads spread over the banks
    float v[2][TK][D];
    float p[TK][R];          // weights of the tile, [key][row]
    long long at[2][TK];     // first element of a key's row in the caches, -1: nothing to read
    float corr[R], m[R], l[R];
    int pos[R], head[R], out[R];   // out: the row's place in o, -1: none
    uint8_t frozen[R];
    int imin, imax, full, any_ord;
};

__device__ __forceinline__ void copy16(void* dst, const float* src, bool have) {   // zeros without a source
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(have ? 16 : 0)
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(const __grid_constant__ PagedArgs p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedItem it = paged_item(p, blockIdx.x);
    const PagedBlock block = paged_block(p, it);

    if (tid == 0) {
        sm.imin = 0x7fffffff;
        sm.imax = -1;
        sm.full = sm.any_ord = 0;
    }
    __syncthreads();
    if (tid < R) {
        const PagedRow w = paged_row(p, it, block, tid);
        sm.pos[tid] = w.i;
        sm.head[tid] = w.h;
        sm.out[tid] = w.there ? (int)paged_out_row(p, w) : -1;
        sm.frozen[tid] = w.frozen;
        if (w.i >= 0) {
            atomicMin(&sm.imin, w.i);
            atomicMax(&sm.imax, w.i);
            if (w.frozen) atomicOr(&sm.full, 1);
            else atomicOr(&sm.any_ord, 1);
        }
    } else if (tid == 32 && it.part == 1 && it.chunk == 0 && it.rb == 0 && it.hk == 0) {
        int c;   // each sequence's counts are checked once
        bool bad;
        paged_tokens(p, it.b, &c, &bad);
        if (bad) atomicOr(p.status, kStatusPage);
    }
    __syncthreads();
    const PagedRange g = paged_range(p, it, sm.imin, sm.imax, sm.full || p.window == 0);
    const int e0 = min(it.chunk * p.per_chunk[it.part], g.n), e1 = min(e0 + p.per_chunk[it.part], g.n);
    const int off = it.part ? p.P : 0;
    const float* kc = (const float*)p.k_cache;
    const float* vc = (const float*)p.v_cache;
    const bool any_ord = sm.any_ord != 0;

    // where key `lane` of tile e lies (warp 0); keys that no row sees, and those of pages outside
    // the cache, are read as zeros
    auto look = [&](int e) -> long long {
        if (e >= e1) return -1;
        const int x = paged_tile(g, e) * TK + lane;
        if (!(x < g.hi && (x >= g.lo || x < g.sink))) return -1;
        const int pg = paged_page(p, it, x);
        if (pg < 0) {
            atomicOr(p.status, kStatusPage);
            return -1;
        }
        return ((((long long)pg * p.Hkv + it.hk) << p.page_log2) + (x & ((1 << p.page_log2) - 1))) * D;
    };
    auto copy_tile = [&](int s) {
        for (int u = tid; u < TK * (D / 4); u += kThreads) {
            const int kk = u / (D / 4), c = 4 * (u - kk * (D / 4));
            const long long at = sm.at[s][kk];
            const long long from = at < 0 ? 0 : at + c;
            if (any_ord) copy16(&sm.k[s][kk][c], kc + from, at >= 0);
            copy16(&sm.v[s][kk][c], vc + from, at >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (warp == 0) {
        sm.at[0][lane] = look(e0);
        sm.at[1][lane] = look(e0 + 1);
    }
    if (any_ord && e0 < e1)
        for (int u = tid; u < R * (D / 4); u += kThreads) {
            const int rr = u / (D / 4), c = 4 * (u - rr * (D / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (sm.pos[rr] >= 0 && !sm.frozen[rr])
                x = *reinterpret_cast<const float4*>((const float*)p.q + (size_t)sm.out[rr] * D + c);
            *reinterpret_cast<float4*>(&sm.q[rr][c]) = x;
        }
    __syncthreads();
    if (e0 < e1) copy_tile(0);

    // this warp's two rows
    int ri[2];
    bool fz[2];
    const float* ra[2];
    const float* rr[2];
    float m[2], l[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int x = 2 * warp + u;
        ri[u] = sm.pos[x];
        fz[u] = sm.frozen[x] && ri[u] >= 0;
        ra[u] = p.a + (size_t)sm.head[x] * p.ld;
        rr[u] = p.r + (size_t)sm.head[x] * p.ld;
        m[u] = -INFINITY;
        l[u] = 0.f;
    }
    // output columns: thread c of D holds column c; with D = 64 two threads share a column's keys
    constexpr int NK = D == 64 ? 2 : 1;
    const int col = NK == 2 ? (tid & 63) : tid, kh = NK == 2 ? (tid >> 6) : 0;
    float acc[R];
#pragma unroll
    for (int x = 0; x < R; ++x) acc[x] = 0.f;

    for (int e = e0, n = 0; e < e1; ++e, ++n) {
        const int s = n & 1;
        const int j = off + paged_tile(g, e) * TK + lane;   // my key's position
        float lg[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (fz[u] && j <= ri[u]) lg[u] = __ldg(ra[u] + j) + __ldg(rr[u] + ri[u] - j);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();   // the tile is there, and everyone is done with the one before
        if (e + 1 < e1) copy_tile(s ^ 1);
        const long long live = sm.at[s][lane];
        const long long next = warp == 0 ? look(e + 2) : -1;
        float dot[2] = {0.f, 0.f};
        if (any_ord) {
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 kx = *reinterpret_cast<const float4*>(&sm.k[s][lane][c]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 qx = *reinterpret_cast<const float4*>(&sm.q[2 * warp + u][c]);
                    dot[u] = fmaf(qx.x, kx.x, dot[u]);
                    dot[u] = fmaf(qx.y, kx.y, dot[u]);
                    dot[u] = fmaf(qx.z, kx.z, dot[u]);
                    dot[u] = fmaf(qx.w, kx.w, dot[u]);
                }
            }
        }
        float2 w;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = ri[u];
            float x = -INFINITY;
            if (live >= 0 && j <= i) {
                if (fz[u]) x = lg[u] * kLog2e;
                else if (p.window == 0 || i - j < p.window || j < p.sinks) x = dot[u] * p.scale_log2;
            }
            float mx = x;
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m[u], mx);
            const float base = m_new == -INFINITY ? 0.f : m_new;   // a row that has seen nothing yet
            const float f = exp2f(m[u] - base), y = exp2f(x - base);
            l[u] = l[u] * f + y;
            m[u] = m_new;
            if (lane == 0) sm.corr[2 * warp + u] = f;
            (u ? w.y : w.x) = y;
        }
        *reinterpret_cast<float2*>(&sm.p[lane][2 * warp]) = w;
        __syncthreads();
        if (warp == 0) sm.at[s][lane] = next;   // (this tile's are in registers or used)
        if (col < D) {
#pragma unroll
            for (int x = 0; x < R; ++x) acc[x] *= sm.corr[x];
#pragma unroll 4
            for (int kk = kh * (TK / NK); kk < (kh + 1) * (TK / NK); ++kk) {
                const float vx = sm.v[s][kk][col];
                const float4 pa = *reinterpret_cast<const float4*>(&sm.p[kk][0]);
                const float4 pb = *reinterpret_cast<const float4*>(&sm.p[kk][4]);
                acc[0] = fmaf(pa.x, vx, acc[0]);
                acc[1] = fmaf(pa.y, vx, acc[1]);
                acc[2] = fmaf(pa.z, vx, acc[2]);
                acc[3] = fmaf(pa.w, vx, acc[3]);
                acc[4] = fmaf(pb.x, vx, acc[4]);
                acc[5] = fmaf(pb.y, vx, acc[5]);
                acc[6] = fmaf(pb.z, vx, acc[6]);
                acc[7] = fmaf(pb.w, vx, acc[7]);
            }
        }
    }

#pragma unroll
    for (int u = 0; u < 2; ++u) {
        for (int o = 16; o; o >>= 1) l[u] += __shfl_xor_sync(0xffffffffu, l[u], o);
        if (lane == 0) {
            sm.m[2 * warp + u] = m[u];
            sm.l[2 * warp + u] = l[u];
        }
    }
    __syncthreads();
    if (NK == 2) {   // the two halves of a column's keys
        float* half = &sm.v[0][0][0];
        if (kh == 1)
#pragma unroll
            for (int x = 0; x < R; ++x) half[x * D + col] = acc[x];
        __syncthreads();
        if (kh == 0)
#pragma unroll
            for (int x = 0; x < R; ++x) acc[x] += half[x * D + col];
    }
    const int split = it.part ? p.chunks[0] + it.chunk : it.chunk;
    if (kh == 0 && col < D) {
#pragma unroll
        for (int x = 0; x < R; ++x) {
            if (sm.out[x] < 0) continue;
            const size_t row = (size_t)sm.out[x];
            const float lx = sm.l[x];
            if (p.nsplit == 1) {
                ((float*)p.o)[row * D + col] = lx != 0.f ? acc[x] / lx : 0.f;
                if (col == 0) p.lse[row] = lx != 0.f ? (sm.m[x] + log2f(lx)) * kLn2 : -INFINITY;
            } else {
                p.po[(row * p.nsplit + split) * D + col] = acc[x];
                if (col == 0) p.ml[row * p.nsplit + split] = make_float2(sm.m[x], lx);
            }
        }
    }
}

template <int D>
cudaError_t launch_d(const PagedArgs& p, cudaStream_t s) {
    const size_t smem = sizeof(Smem<D>);
    cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_ex(paged_simt_kernel<D>, dim3(p.items), dim3(kThreads), smem, s, true, 1, p);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedArgs& p, cudaStream_t s) {
    switch (p.d) {
        case 96: return launch_d<96>(p, s);
        case 128: return launch_d<128>(p, s);
        default: return launch_d<64>(p, s);
    }
}

}  // namespace saf
