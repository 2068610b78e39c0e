// Windowed backward: key blocks that hold sinks, in parts.
//
// Every query sees a sink, so the key block of a sink is visited by every query block where
// another is visited by the few that its window reaches: as one work item it would be the length
// of the launch (H8 over one key/value head, d 64, T 32768, window 512, 16 sinks: 3.9 ms forward
// and backward, 0.38 ms in parts, 0.29 ms without sinks). Its query blocks are therefore shared by several items,
// each of which leaves its dV and dK (unscaled) in fp32, and the kernel here adds them up in the
// order of the parts: the result does not depend on which ended first.
#include <algorithm>
#include <cmath>

#include "saf_internal.h"
#include "tc_common.cuh"

namespace saf {
namespace {

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16(x.x, x.y), tc::pack_bf16(x.z, x.w));
}

// One thread per four columns of a key's dV or dK; the sums are read once (bound: their bytes, from
// L2 as a rule). Grid: items x 2 * rows * d / 1024. A key/value head whose query heads are all
// frozen was not split.
template <typename E>
__global__ void __launch_bounds__(256) join_parts_kernel(SinkParts sp, E* __restrict__ dv, E* __restrict__ dk,
                                                         HeadMask mask, int Hkv, int G, int T, int d, float scale) {
    grid_dep_wait();
    grid_dep_launch();
    const int elems = sp.rows * d, per = 2 * elems / 1024;
    const int item = (int)(blockIdx.x / per);
    int e = (int)(blockIdx.x % per) * 1024 + threadIdx.x * 4;
    const int which = e >= elems;
    e -= which * elems;
    const int bkv = item / sp.blocks, kb = item - bkv * sp.blocks, hk = bkv % Hkv;
    if (kb * sp.rows + e / d >= T) return;
    bool frozen = true;
    for (int gi = 0; gi < G; ++gi) frozen = frozen && head_frozen(mask, hk * G + gi);
    if (frozen) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < sp.parts; ++k) {
        if (sp.range(kb, T, k).n == 0) break;
        const float4 x = __ldcg(reinterpret_cast<const float4*>(sp.at(bkv, kb, k, which, d) + e));
        acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
    }
    const float f = which ? scale : 1.f;
    store4((which ? dk : dv) + ((size_t)bkv * T + (size_t)kb * sp.rows) * d + e,
           make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
}

}  // namespace

// Each part gets about half of a slot's share of the launch's tiles (a frozen head's counted as half
// an ordinary one's), at least `few`; at most 32 parts and what `bytes` hold (0: nothing is split).
SinkParts plan_sink_parts(const LayerArgs& a, int rows, int q_rows, int slots, int few, void* sums, size_t bytes) {
    const SinkParts none{0, 1, rows, q_rows, nullptr};
    if (a.window == 0 || a.sinks == 0) return none;
    const int Hkv = a.Hkv > 0 ? a.Hkv : a.H, G = a.H / Hkv;
    const int nkb = (a.T + rows - 1) / rows, nqb = (a.T + q_rows - 1) / q_rows;
    int n_ord = 0;
    for (int h = 0; h < a.H; ++h) n_ord += head_frozen(a.mask, h) ? 0 : 1;
    if (n_ord == 0) return none;
    const int blocks = a.sinks >= a.T ? nkb : (a.sinks + rows - 1) / rows;
    const double reach = std::min<double>(nqb, (rows - 2.0 + a.window) / q_rows + 1);   // of another key block
    const double ord = blocks * (double)nqb + (nkb - blocks) * reach, frz = 0.5 * nkb * (nqb + 1.0);
    const double share = a.B * (n_ord * ord + 0.5 * (a.H - n_ord) * frz) / slots;
    const double longest = G * (double)nqb * (n_ord + 0.5 * (a.H - n_ord)) / a.H;
    const size_t items = (size_t)a.B * Hkv * blocks, part_bytes = (size_t)2 * rows * a.d * sizeof(float);
    const double want = std::ceil(longest / std::max(0.5 * share, (double)few));
    const int parts = (int)std::min({want, 32.0, (double)nqb, (double)(bytes / (items * part_bytes))});
    if (parts < 2) return none;
    return SinkParts{blocks, parts, rows, q_rows, (float*)sums};
}

template <typename E>
cudaError_t launch_join_parts(const LayerArgs& a, const SinkParts& sp, cudaStream_t s) {
    const int Hkv = a.Hkv > 0 ? a.Hkv : a.H;
    const unsigned grid = (unsigned)((size_t)a.B * Hkv * sp.blocks * (2 * sp.rows * a.d / 1024));
    note_launch();
    return launch_ex(join_parts_kernel<E>, dim3(grid), dim3(256), 0, s, true, 1, sp, (E*)a.dv, (E*)a.dk, a.mask, Hkv,
                     a.H / Hkv, a.T, a.d, 1.f / sqrtf((float)a.d));
}
template cudaError_t launch_join_parts<float>(const LayerArgs&, const SinkParts&, cudaStream_t);
template cudaError_t launch_join_parts<__nv_bfloat16>(const LayerArgs&, const SinkParts&, cudaStream_t);

}  // namespace saf
