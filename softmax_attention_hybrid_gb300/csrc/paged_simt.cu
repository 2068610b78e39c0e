// Paged attention of fp32 caches on the CUDA cores (see paged.h for the split).
//
// An item holds up to 8 query rows and walks its tiles of 64 keys:
//   scores   thread (key, half): the key's products with four rows, K and q from shared memory;
//            a frozen row's logit is a[j] + r[i - j] instead
//   softmax  a warp per two rows: running maximum and sum, base 2
//   output   thread per column of d: rows' weights (broadcast) times the column's values
// Bound by the cache's bytes with up to 8 rows: a 64-key tile at d = 128 is 64 KB of fp32
// and 131 K multiply-adds, 1024 cycles of an SM's 128 lanes, while 64 KB take about 2800
// cycles of an SM's share of the memory.
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
    float k[TK][D + 4];   // 16 more bytes a row: the 64 keys' float4 reads spread over the banks
    float v[TK][D];
    float p[TK][R];       // weights of the tile, [key][row]
    float s[R][TK + 1];
    float corr[R], m[R], l[R];
    int pos[R], head[R], out[R];   // out: the row's place in o, -1: none
    uint8_t frozen[R], live[TK];
    int imin, imax, full, any_ord;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(const __grid_constant__ PagedArgs p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedItem it = paged_item(p, blockIdx.x);
    const int r0 = it.rb * R;

    if (tid == 0) {
        sm.imin = 0x7fffffff;
        sm.imax = -1;
        sm.full = sm.any_ord = 0;
    }
    __syncthreads();
    PagedRow w;
    if (tid < R) {
        w = paged_row(p, it, r0 + tid);
        sm.pos[tid] = w.i;
        sm.head[tid] = w.h;
        sm.out[tid] = w.there ? (int)paged_out_row(p, w) : -1;
        sm.frozen[tid] = w.frozen;
        sm.m[tid] = -INFINITY;
        sm.l[tid] = 0.f;
        if (w.i >= 0) {
            atomicMin(&sm.imin, w.i);
            atomicMax(&sm.imax, w.i);
            if (w.frozen) atomicOr(&sm.full, 1);
            else atomicOr(&sm.any_ord, 1);
        }
    }
    // each sequence's counts are checked once, by the first item that has it
    if (it.part == 1 && it.chunk == 0 && it.rb == 0 && it.hk == 0 && tid == 0) {
        int c;
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

    if (any_ord && e0 < e1)
        for (int e = tid; e < R * (D / 4); e += kThreads) {
            const int rr = e / (D / 4), c = 4 * (e - rr * (D / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (sm.pos[rr] >= 0 && !sm.frozen[rr]) x = load4((const float*)p.q + (size_t)sm.out[rr] * D + c);
            *reinterpret_cast<float4*>(&sm.q[rr][c]) = x;
        }

    // output columns: thread c of D holds column c; with D = 64 two threads share a column's keys
    constexpr int NK = D == 64 ? 2 : 1;
    const int col = NK == 2 ? (tid & 63) : tid, kh = NK == 2 ? (tid >> 6) : 0;
    float acc[R];
#pragma unroll
    for (int x = 0; x < R; ++x) acc[x] = 0.f;

    for (int e = e0; e < e1; ++e) {
        const int x0 = paged_tile(g, e) * TK;
        __syncthreads();
        // K and V of the tile; keys that no row sees, and those of pages outside the cache, as zeros
        if (tid < TK) {
            const int x = x0 + tid;
            const bool seen = x < g.hi && (x >= g.lo || x < g.sink);
            const bool page = seen && paged_page(p, it, x) >= 0;
            if (seen && !page) atomicOr(p.status, kStatusPage);
            sm.live[tid] = page;
        }
        __syncthreads();
        for (int u = tid; u < TK * (D / 4); u += kThreads) {
            const int kk = u / (D / 4), c = 4 * (u - kk * (D / 4));
            float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
            if (sm.live[kk]) {
                const int x = x0 + kk;
                const size_t row = (((size_t)paged_page(p, it, x) * p.Hkv + it.hk) << p.page_log2) +
                                   (x & ((1 << p.page_log2) - 1));
                if (any_ord) kx = load4(kc + row * D + c);
                vx = load4(vc + row * D + c);
            }
            *reinterpret_cast<float4*>(&sm.k[kk][c]) = kx;
            *reinterpret_cast<float4*>(&sm.v[kk][c]) = vx;
        }
        __syncthreads();
        {
            const int kk = tid & 63, rh = 4 * (tid >> 6);
            float dot[4] = {0.f, 0.f, 0.f, 0.f};
            if (any_ord) {
#pragma unroll 8
                for (int c = 0; c < D; c += 4) {
                    const float4 kx = *reinterpret_cast<const float4*>(&sm.k[kk][c]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float4 qx = *reinterpret_cast<const float4*>(&sm.q[rh + u][c]);
                        dot[u] = fmaf(qx.x, kx.x, dot[u]);
                        dot[u] = fmaf(qx.y, kx.y, dot[u]);
                        dot[u] = fmaf(qx.z, kx.z, dot[u]);
                        dot[u] = fmaf(qx.w, kx.w, dot[u]);
                    }
                }
            }
            const int j = off + x0 + kk;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = sm.pos[rh + u];
                float s = -INFINITY;
                if (sm.live[kk] && j <= i) {
                    if (sm.frozen[rh + u]) {
                        const size_t hr = (size_t)sm.head[rh + u] * p.ld;
                        s = (p.a[hr + j] + p.r[hr + i - j]) * kLog2e;
                    } else if (p.window == 0 || i - j < p.window || j < p.sinks) {
                        s = dot[u] * p.scale_log2;
                    }
                }
                sm.s[rh + u][kk] = s;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int rr = 2 * warp + u;
            const float s0 = sm.s[rr][lane], s1 = sm.s[rr][lane + 32];
            float mx = fmaxf(s0, s1);
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_old = sm.m[rr], m_new = fmaxf(m_old, mx);
            const float base = m_new == -INFINITY ? 0.f : m_new;   // a row that has seen nothing yet
            const float w0 = exp2f(s0 - base), w1 = exp2f(s1 - base);
            float sum = w0 + w1;
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sm.p[lane][rr] = w0;
            sm.p[lane + 32][rr] = w1;
            __syncwarp();
            if (lane == 0) {
                const float f = exp2f(m_old - base);
                sm.corr[rr] = f;
                sm.l[rr] = sm.l[rr] * f + sum;
                sm.m[rr] = m_new;
            }
        }
        __syncthreads();
        if (col < D) {
#pragma unroll
            for (int x = 0; x < R; ++x) acc[x] *= sm.corr[x];
#pragma unroll 4
            for (int kk = kh * (TK / NK); kk < (kh + 1) * (TK / NK); ++kk) {
                const float vx = sm.v[kk][col];
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

    __syncthreads();
    if (NK == 2) {   // the two halves of a column's keys
        float* half = &sm.v[0][0];
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
            if (p.nsplit == 1) {
                const float l = sm.l[x];
                ((float*)p.o)[row * D + col] = l > 0.f ? acc[x] / l : 0.f;
                if (col == 0) p.lse[row] = l > 0.f ? (sm.m[x] + log2f(l)) * kLn2 : -INFINITY;
            } else {
                p.po[(row * p.nsplit + split) * D + col] = acc[x];
                if (col == 0) p.ml[row * p.nsplit + split] = make_float2(sm.m[x], sm.l[x]);
            }
        }
    }
}

template <int D>
cudaError_t launch_d(const PagedArgs& p, cudaStream_t s) {
    const size_t smem = sizeof(Smem<D>);
    cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_ex(paged_simt_kernel<D>, dim3((unsigned)p.items), dim3(kThreads), smem, s, true, 1, p);
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
