// Windowed backward on the tensor cores: key blocks that hold sinks, in parts.
//
// Every query sees a sink, so the key block of a sink is visited by all T / 128 query blocks where
// another is visited by the few that its window reaches: as one work item it would be the length
// of the launch (H8 over one key/value head, d 64, T 32768, window 512, 16 sinks: 3.9 ms forward
// and backward, 0.29 ms without sinks). Its query blocks are therefore shared by several items,
// each of which leaves its dV and dK (unscaled) in fp32, and the kernel here adds them up in the
// order of the parts: the result does not depend on which ended first.
#include <algorithm>
#include <cmath>

#include "saf_internal.h"
#include "tc_common.cuh"

namespace saf {
namespace {

// One thread per four columns of a key's dV or dK; the sums are read once (bound: their bytes, from
// L2 as a rule). Grid: items x 2 * 128 * d / 1024. A key/value head whose query heads are all
// frozen was not split.
__global__ void __launch_bounds__(256)
join_parts_kernel(SinkParts sp, __nv_bfloat16* __restrict__ dv, __nv_bfloat16* __restrict__ dk, HeadMask mask, int Hkv,
                  int G, int T, int d, int nqb, float scale) {
    grid_dep_wait();
    grid_dep_launch();
    const int block_elems = 128 * d, per = 2 * block_elems / 1024;
    const int item = (int)(blockIdx.x / per);
    int e = (int)(blockIdx.x % per) * 1024 + threadIdx.x * 4;
    const bool is_k = e >= block_elems;
    if (is_k) e -= block_elems;
    const int bkv = item / sp.blocks, kb = item - bkv * sp.blocks, hk = bkv % Hkv;
    if (kb * 128 + e / d >= T) return;
    bool frozen = true;
    for (int gi = 0; gi < G; ++gi) frozen = frozen && head_frozen(mask, hk * G + gi);
    if (frozen) return;
    const float* src = sp.sums + ((size_t)item * sp.parts * 2 + is_k) * block_elems + e;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < sp.parts; ++k) {
        if (sp.range(kb, nqb, k).n == 0) break;
        const float4 x = __ldcg(reinterpret_cast<const float4*>(src + (size_t)k * 2 * block_elems));
        acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
    }
    const float f = is_k ? scale : 1.f;
    __nv_bfloat16* dst = (is_k ? dk : dv) + ((size_t)bkv * T + (size_t)kb * 128) * d + e;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(tc::pack_bf16(acc.x * f, acc.y * f), tc::pack_bf16(acc.z * f, acc.w * f));
}

}  // namespace

// Each part gets about half of an SM's share of the launch's tiles (a frozen head's counted as half
// an ordinary one's), at least 16, at most 32 parts and what `bytes` hold.
SinkParts plan_sink_parts(const LayerArgs& a, float* sums, size_t bytes) {
    SinkParts sp{0, 1, nullptr};
    if (a.window == 0 || a.sinks == 0) return sp;
    const int Hkv = a.Hkv > 0 ? a.Hkv : a.H, G = a.H / Hkv, nqb = (a.T + 127) / 128;
    int n_ord = 0;
    for (int h = 0; h < a.H; ++h) n_ord += head_frozen(a.mask, h) ? 0 : 1;
    if (n_ord == 0) return sp;
    const int blocks = a.sinks >= a.T ? nqb : (a.sinks + 127) / 128;
    const double reach = std::min<double>(nqb, (126.0 + a.window) / 128 + 1);   // query blocks of another block
    const double ord = blocks * (double)nqb + (nqb - blocks) * reach, frz = 0.5 * nqb * (nqb + 1.0);
    const double share = a.B * (n_ord * ord + 0.5 * (a.H - n_ord) * frz) / 152;
    const double longest = G * (double)nqb * (n_ord + 0.5 * (a.H - n_ord)) / a.H;
    const size_t items = (size_t)a.B * Hkv * blocks, part_bytes = (size_t)2 * 128 * a.d * sizeof(float);
    const double want = std::ceil(longest / std::max(0.5 * share, 16.0));
    const int parts = (int)std::min({want, 32.0, (double)nqb, (double)(bytes / (items * part_bytes))});
    if (parts < 2) return sp;
    return SinkParts{blocks, parts, sums};
}

cudaError_t launch_join_parts(const LayerArgs& a, const SinkParts& sp, cudaStream_t s) {
    const int Hkv = a.Hkv > 0 ? a.Hkv : a.H;
    const unsigned grid = (unsigned)((size_t)a.B * Hkv * sp.blocks * (2 * 128 * a.d / 1024));
    note_launch();
    return launch_ex(join_parts_kernel, dim3(grid), dim3(256), 0, s, true, 1, sp, (__nv_bfloat16*)a.dv,
                     (__nv_bfloat16*)a.dk, a.mask, Hkv, a.H / Hkv, a.T, a.d, (a.T + 127) / 128,
                     1.f / sqrtf((float)a.d));
}

}  // namespace saf
