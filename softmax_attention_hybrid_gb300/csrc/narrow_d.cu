// Windowed backward in bf16: D of rows that see few keys.
//
// dS(i, j) = P(i, j) (dP(i, j) - D(i)), D(i) = sum_j P(i, j) dP(i, j) = dO(i) . o(i). The backward takes
// D from the forward's o, which is rounded to bf16: over many keys that is lost in the rounding of
// dS, over two to sixteen it is the largest error of dq and dk (against 64 bits, relative, windows of 2, 4,
// 16 keys: 0.0037, 0.0030, 0.0025 from the rounded o, 0.0023, 0.0024, 0.0024 from the sum over j). So
// where no row sees more than kNarrow keys, and in sequences of at most kShort tokens, whose rows
// see half of that on the average, the sum is formed here in fp32, over the D that the pass
// before wrote. Four lanes to a row, a quarter of its elements each; neighbouring rows' keys come
// from the L1. Bound by the conversions and products of 2 d kNarrow a row: a layer of 12 heads of 64,
// B8 T4096, window 16, takes 472 us forward and backward where the D of the pass before leaves 368.
#include <algorithm>

#include "saf_internal.h"

namespace saf {
namespace {

constexpr int kNarrow = 16, kShort = 32;   // keys of a row; tokens of a sequence

template <int D>
__global__ void __launch_bounds__(128)
narrow_d_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ dO,
                const float* __restrict__ lse, float* __restrict__ rowvec, HeadMask mask, int H, int Hkv, int T,
                int window, int sinks) {
    grid_dep_wait();
    grid_dep_launch();
    const int bh = blockIdx.y, h = bh % H;
    if (head_frozen(mask, h)) return;
    constexpr int N = D / 4, kVec = N / 8;   // my elements of a row, in 16-byte pieces
    const int part = threadIdx.x & 3, i = blockIdx.x * 32 + (threadIdx.x >> 2);
    const int row = min(i, T - 1);   // rows past the end do the last one's work and store nothing
    auto load = [&](const __nv_bfloat16* p, size_t r, float* x) {
        const uint4* src = reinterpret_cast<const uint4*>(p + r * D + part * N);
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            const uint4 y = __ldg(src + c);
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[8 * c + 2 * e] = __uint_as_float(w[e] << 16);
                x[8 * c + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
        }
    };
    const size_t at = (size_t)bh * T + row;
    const size_t kv = ((size_t)(bh / H) * Hkv + h / (H / Hkv)) * T;
    float qr[N], dr[N];
    load(q, at, qr);
    load(dO, at, dr);
    const float scale = rsqrtf((float)D), l = lse[at];
    const int first = max(0, row - window + 1), recent = row - first + 1;   // the window's keys
    const int n = recent + min(sinks, first);                              // and the sinks before them
    const int most = min(T, window + min(sinks, T));
    float sum = 0.f;
    for (int e = 0; e < most; ++e) {
        const int j = e < recent ? first + e : min(e - recent, T - 1);
        float x[N], s = 0.f, t = 0.f;
        load(k, kv + j, x);
#pragma unroll
        for (int c = 0; c < N; ++c) s = fmaf(qr[c], x[c], s);
        load(v, kv + j, x);
#pragma unroll
        for (int c = 0; c < N; ++c) t = fmaf(dr[c], x[c], t);
#pragma unroll
        for (int m = 1; m < 4; m <<= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, m);
            t += __shfl_xor_sync(0xffffffffu, t, m);
        }
        if (e < n) sum = fmaf(expf(fmaf(s, scale, -l)), t, sum);
    }
    if (part == 0 && i < T) {
        const int nqb = (T + 127) / 128;
        rowvec[((size_t)bh * nqb + (i >> 7)) * 256 + 128 + (i & 127)] = sum;
    }
}

template <int D>
cudaError_t launch_d(const LayerArgs& a, int window, cudaStream_t s) {
    note_launch();
    const dim3 grid((unsigned)((a.T + 31) / 32), (unsigned)(a.B * a.H));
    return launch_ex(narrow_d_kernel<D>, grid, dim3(128), 0, s, true, 1, (const __nv_bfloat16*)a.q,
                     (const __nv_bfloat16*)a.k, (const __nv_bfloat16*)a.v, (const __nv_bfloat16*)a.dO, a.lse, a.rowvec,
                     a.mask, a.H, a.Hkv, a.T, window, a.sinks);
}

}  // namespace

cudaError_t launch_narrow_d(const LayerArgs& a, cudaStream_t s) {
    const int window = a.window > 0 ? a.window : a.T;
    if (!a.exact_d || (a.T > kShort && (long long)window + std::min(a.sinks, a.T) > kNarrow)) return cudaSuccess;
    bool ordinary = false;
    for (int h = 0; h < a.H; ++h) ordinary = ordinary || !head_frozen(a.mask, h);
    if (!ordinary) return cudaSuccess;
    return a.d == 96 ? launch_d<96>(a, window, s) : a.d == 128 ? launch_d<128>(a, window, s) : launch_d<64>(a, window, s);
}

}  // namespace saf
