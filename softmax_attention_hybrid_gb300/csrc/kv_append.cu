// Keys and values of new tokens into a paged cache, with the rotary position rotation of
// k (and of q, for the attention that follows) on the way.
//
// Token t of sequence b goes to slot x = ctx[b] + t of the sequence: row x mod page of page
// table[b][x / page]. Pair c of a row's first `rope_dim` elements is turned by the angle
// pos * f_c with pos = pos_base + x:
//     (y0, y1) = (x0 cos - x1 sin, x0 sin + x1 cos),
// in fp32, rounded once to the cache's type. Angles of far positions keep their digits: the
// host turns f_c into F_c = (f_c / 2 pi mod 1) 2^64, rounded to an integer from two doubles, and
// pos * F_c in 64-bit integers is the angle in turns, modulo one, off by pos 2^-64 at most: by
// 2^-24 of a turn, what fp32 leaves anyway, at the last position that is taken, 2^40.
//
// Bound by memory: every element is read once and written once; the angles cost one
// sincospif per pair and token for several heads. Thread = 16 elements of a row (8 pairs) of
// `per` heads of a token, so that neighbouring threads read whole rows. The prompts of eight
// sequences (105 MB) take 23 us, 4.6 TB/s, 67% of a plain copy's rate: a thread waits for its
// counts, then its page, then its rows. (The angles of a block's tokens computed once, into
// shared memory, took 2 us more: they are not what bounds it.)
//
// 8-bit caches (saf_kv_append_quant). A row y is held as codes and one scale,
//     scale = max(max_c |y_c| / 448, 2^-126),   code_c = y_c / scale, rounded to e4m3,
// with y rotated but not rounded before. The threads of a row are then neighbouring lanes (4, or
// 8 of which 6 work at d = 96) that find the row's maximum by shuffles, and the reciprocal of the scale is
// the hardware's, off by a step of fp32. The prompts of eight sequences (111 MB, 12 heads of 64)
// take 32 us, 3.4 TB/s, twice what the bytes take: the chain of loads is the same (most stalls are waits for memory, 24
// warps to an SM at 80 registers), and rotation, maximum and conversion fill 58% of the issue slots beside it.
#include <cuda_fp8.h>
#include <math.h>
#include <string.h>

#include "saf_internal.h"

namespace saf {
namespace {

constexpr int kThreads = 128;
constexpr long long kFullGpu = 152ll * 2048;   // threads that the GPU holds

struct AppendArgs {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    float *k_scale, *v_scale;        // 8-bit caches: [num_pages, Hkv, page]
    const int32_t *ctx, *n_new, *table;
    uint32_t* status;
    long long sq[3], sk[3], sv[3];   // element strides (sequence, head, token)
    long long pos_base;
    int B, H, Hkv, T, d, max_pages, num_pages, page_log2;
    int rope, interleaved;
    int units;                       // d / 16
    int lanes;                       // threads of a row: units, or for 8-bit caches 4 or 8
    int nq, nk, slots;               // heads of q, of k, and all with v's that are moved
    int per, groups;                 // slots of a thread; ceil(slots / per)
    uint64_t freq[64];               // F_c
    uint8_t heads[2 * SAF_MAX_HEADS];   // nq query heads, then nk key heads
};

// 8 elements as they lie in memory.
template <typename E>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ void store(float* p) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(p + 4) = b;
    }
    __device__ void get(float* x) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ void set(const float* x) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint32_t w[4];
    __device__ void load(const __nv_bfloat16* p) { *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p); }
    __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w); }
    __device__ void get(float* x) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    __device__ void set(const float* x) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
};

__device__ __forceinline__ float max3_abs(float m, float x, float y) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x)), "f"(fabsf(y)));
    return r;
}
__device__ __forceinline__ float reciprocal(float x) {   // to a step of fp32; x at least 2^-126
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 8 values as codes of e4m3 (out of range: the largest; NaN stays NaN).
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c[e] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e] * inv, x[2 * e + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

template <typename E, bool kQ8>
__device__ __forceinline__ void append_token(const AppendArgs& p, int b, int t, int group, int u) {
    const int c = p.ctx[b];
    const int n = p.n_new ? p.n_new[b] : p.T;
    const long long room = (long long)p.max_pages << p.page_log2;
    if (c < 0 || n < 0 || n > p.T || c + (long long)n > room) {
        if (t == 0 && group == 0 && u == 0 && p.status) atomicOr(p.status, kStatusPage);
        if (c < 0) return;
    }
    if (t >= n) return;
    const long long slot = (long long)c + t;
    if (slot >= room) return;   // no token: the count is cut to the room
    int page = p.table[(size_t)b * p.max_pages + (slot >> p.page_log2)];
    if (page < 0 || page >= p.num_pages) {
        if (group == 0 && u == 0 && p.status) atomicOr(p.status, kStatusPage);
        page = -1;
    }
    const size_t page_row = (size_t)(slot & ((1 << p.page_log2) - 1));

    // my 16 elements: two runs of 8, for a rotated row's pairs (8u + e, rope / 2 + 8u + e) when
    // the pairs are halves apart
    const bool mine = !kQ8 || u < p.units;   // (a lane without elements still takes part in the shuffles)
    const bool turn = 16 * u < p.rope;
    const int c0 = turn && !p.interleaved ? 8 * u : 16 * u;
    const int c1 = turn && !p.interleaved ? (p.rope >> 1) + 8 * u : 16 * u + 8;
    float cs[8], sn[8];
    if (turn && group < p.nq + p.nk) {
        const uint64_t pos = (uint64_t)(p.pos_base + slot);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // the angle in half turns, in [-1, 1)
            const int32_t x = (int32_t)((pos * p.freq[8 * u + e]) >> 32);
            sincospif((float)x * 4.656612873077393e-10f, &sn[e], &cs[e]);   // 2^-31
        }
    }
    // My heads are group, group + groups, ...: the threads of a token then read rows that lie next to
    // each other. Several rows are on their way at a time.
    constexpr int kBatch = sizeof(E) == 2 && !kQ8 ? 4 : 2;
    for (int s0 = group; s0 < p.slots; s0 += kBatch * p.groups) {
        Raw<E> x[kBatch], y[kBatch];
        E* dst[kBatch];          // the row in q_out or in the cache
        size_t at[kQ8 ? kBatch : 1];   // 8-bit caches: the row's number
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int s = s0 + k * p.groups;
            dst[k] = nullptr;
            if (s >= p.slots) continue;
            const bool is_v = s >= p.nq + p.nk;
            const int h = is_v ? s - p.nq - p.nk : p.heads[s];
            const E* src;
            if (s < p.nq) {
                src = (const E*)p.q + b * p.sq[0] + h * p.sq[1] + t * p.sq[2];
                dst[k] = (E*)p.q_out + (((size_t)b * p.H + h) * p.T + t) * p.d;
            } else {
                if (page < 0) continue;
                const long long* st = is_v ? p.sv : p.sk;
                src = (const E*)(is_v ? p.v : p.k) + b * st[0] + h * st[1] + t * st[2];
                const size_t row = (((size_t)page * p.Hkv + h) << p.page_log2) + page_row;
                if constexpr (kQ8) {
                    at[k] = row;
                    dst[k] = (E*)(is_v ? p.v_cache : p.k_cache);
                } else {
                    dst[k] = (E*)(is_v ? p.v_cache : p.k_cache) + row * p.d;
                }
            }
            if (!mine) continue;
            x[k].load(src + (is_v ? 16 * u : c0));
            y[k].load(src + (is_v ? 16 * u + 8 : c1));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!dst[k]) continue;
            const bool is_v = s0 + k * p.groups >= p.nq + p.nk;
            const bool coded = kQ8 && s0 + k * p.groups >= p.nq;
            if (!coded && !mine) continue;
            float a[8], z[8];
            if (coded || (turn && !is_v)) {
                if (!mine) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = z[e] = 0.f;
                } else {
                    x[k].get(a);
                    y[k].get(z);
                }
            }
            if (turn && !is_v) {
                if (!p.interleaved) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a0 = a[e], z0 = z[e];
                        a[e] = a0 * cs[e] - z0 * sn[e];
                        z[e] = a0 * sn[e] + z0 * cs[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a0 = a[2 * e], z0 = a[2 * e + 1];
                        a[2 * e] = a0 * cs[e] - z0 * sn[e];
                        a[2 * e + 1] = a0 * sn[e] + z0 * cs[e];
                        a0 = z[2 * e], z0 = z[2 * e + 1];
                        z[2 * e] = a0 * cs[4 + e] - z0 * sn[4 + e];
                        z[2 * e + 1] = a0 * sn[4 + e] + z0 * cs[4 + e];
                    }
                }
                if (!coded) {
                    x[k].set(a);
                    y[k].set(z);
                }
            }
            if constexpr (kQ8) {
                if (coded) {
                    float m = 0.f;   // (a NaN is left out)
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = max3_abs(m, a[e], z[e]);
                    const unsigned first = threadIdx.x & 31u & ~(unsigned)(p.lanes - 1);
                    const unsigned mask = ((1u << p.lanes) - 1u) << first;
                    for (int o = p.lanes >> 1; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
                    const float scale = fmaxf(m * (1.f / 448.f), 0x1p-126f), inv = reciprocal(scale);
                    if (mine) {
                        uint8_t* row = (uint8_t*)dst[k] + at[k] * p.d;
                        *reinterpret_cast<uint2*>(row + (is_v ? 16 * u : c0)) = codes8(a, inv);
                        *reinterpret_cast<uint2*>(row + (is_v ? 16 * u + 8 : c1)) = codes8(z, inv);
                    }
                    if (u == 0) (is_v ? p.v_scale : p.k_scale)[at[k]] = scale;
                    continue;
                }
            }
            x[k].store(dst[k] + (is_v ? 16 * u : c0));
            y[k].store(dst[k] + (is_v ? 16 * u + 8 : c1));
        }
    }
}

template <typename E, bool kQ8>
__device__ __forceinline__ void append_threads(const AppendArgs& p) {
    grid_dep_wait();
    grid_dep_launch();
    const unsigned id = blockIdx.x * kThreads + threadIdx.x;   // (token, group of slots, unit) of a sequence
    const unsigned lanes = (unsigned)(kQ8 ? p.lanes : p.units);
    const unsigned w = id / lanes;
    const int u = (int)(id - w * lanes);
    const int t = (int)(w / (unsigned)p.groups), group = (int)(w - (unsigned)t * (unsigned)p.groups);
    if (t >= p.T) return;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) append_token<E, kQ8>(p, b, t, group, u);
}
template <typename E>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs p) {
    append_threads<E, false>(p);
}
// (six blocks to an SM: more loads on their way than with the 128 registers that it would take)
template <typename E>
__global__ void __launch_bounds__(kThreads, 6) append_codes_kernel(const __grid_constant__ AppendArgs p) {
    append_threads<E, true>(p);
}

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

// x modulo 1 in units of 2^-64, to the nearest (x - trunc(x) and the scaling are exact).
uint64_t turn_units(double x) {
    const double y = (x - trunc(x)) * 18446744073709551616.0;
    const uint64_t n = (uint64_t)nearbyint(fabs(y));
    return y < 0.0 ? 0 - n : n;
}

// f / (2 pi) modulo 1 in units of 2^-64. 1 / (2 pi) is taken as a sum of two doubles (off by 2^-110)
// and the product's rounding error as a third: a single double would leave f / (2 pi) with 53 bits,
// 2^-56 for f near 1, which positions in the billions show.
uint64_t frequency(double f) {
    constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
    const double p = f * hi, e = fma(f, hi, -p) + f * lo;
    return turn_units(p) + turn_units(e);
}

constexpr int64_t kLastBase = 1ll << 40;   // of pos_base

int append(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* ctx,
           const int32_t* n_new, const int32_t* page_table, int max_pages, const double* inv_freq,
           int rope_dim, int interleaved, int64_t pos_base, const uint8_t* frozen, int B, int H,
           int Hkv, int T, int d, int num_pages, int page_size, saf_dtype_t dt, bool coded, void* q_out, void* k_cache,
           void* v_cache, float* k_scale, float* v_scale, uint32_t* status, void* stream) {
    if (B < 0 || H <= 0 || T < 0 || H > SAF_MAX_HEADS || Hkv <= 0 || H % Hkv != 0) return SAF_EINVAL;
    if (dt != SAF_BF16 && dt != SAF_FP32) return SAF_EINVAL;
    if (!head_dim_supported(d, dt)) return SAF_EUNSUPPORTED;
    if (rope_dim < 0 || rope_dim > d || rope_dim % 16 != 0 || (rope_dim > 0 && !inv_freq)) return SAF_EINVAL;
    if (interleaved != 0 && interleaved != 1) return SAF_EINVAL;
    if (pos_base < 0 || pos_base > kLastBase || T > (1 << 21) || (long long)B * T > (1ll << 30)) return SAF_EINVAL;
    if (B == 0 || T == 0) return SAF_OK;
    if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return SAF_EINVAL;
    if (num_pages < 1 || max_pages < 1) return SAF_EINVAL;
    AppendArgs p;
    memset(&p, 0, sizeof(p));
    const int G = H / Hkv;
    if (q)
        for (int h = 0; h < H; ++h)
            if (!(frozen && frozen[h])) p.heads[p.nq++] = (uint8_t)h;
    for (int hk = 0; hk < Hkv; ++hk) {   // keys that an ordinary query head reads
        bool live = false;
        for (int gi = 0; gi < G; ++gi) live |= !(frozen && frozen[hk * G + gi]);
        if (live) p.heads[p.nq + p.nk++] = (uint8_t)hk;
    }
    if (!v || !v_cache || !ctx || !page_table || (p.nq > 0 && !q_out)) return SAF_EINVAL;
    if (p.nk > 0 && (!k || !k_cache)) return SAF_EINVAL;
    if (coded && (!v_scale || (p.nk > 0 && !k_scale))) return SAF_EINVAL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(ctx, 4) || !aligned(n_new, 4) || !aligned(page_table, 4) ||
        !aligned(status, 4) || (coded && (!aligned(k_scale, 16) || !aligned(v_scale, 16))))
        return SAF_EALIGN;
    const long long row = d, e = dt == SAF_BF16 ? 2 : 4;
    long long* st[3] = {p.sq, p.sk, p.sv};
    for (int i = 0; i < 3; ++i) {
        const long long full[3] = {(i ? Hkv : H) * (long long)T * row, T * row, row};
        const int n[3] = {B, i ? Hkv : H, T};
        for (int x = 0; x < 3; ++x) {
            st[i][x] = n[x] == 1 ? 0 : strides ? strides[3 * i + x] : full[x];
            if (st[i][x] * e % 16 != 0) return SAF_EALIGN;
        }
        // in place only where q is laid out as q_out
        if (i == 0 && p.nq > 0 && q == q_out)
            for (int x = 0; x < 3; ++x)
                if (n[x] != 1 && st[i][x] != full[x]) return SAF_EINVAL;
    }
    for (int c = 0; c < rope_dim / 2; ++c) {
        if (!isfinite(inv_freq[c])) return SAF_EINVAL;
        p.freq[c] = frequency(inv_freq[c]);
    }
    int s = check_device();
    if (s != SAF_OK) return s;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.ctx = ctx;
    p.n_new = n_new;
    p.table = page_table;
    p.status = status;
    p.pos_base = pos_base;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.T = T;
    p.d = d;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    while ((1 << p.page_log2) < page_size) ++p.page_log2;
    p.rope = rope_dim;
    p.interleaved = interleaved;
    p.units = d / 16;
    p.lanes = !coded ? p.units : p.units <= 4 ? 4 : 8;
    p.slots = p.nq + p.nk + Hkv;
    // A thread takes several heads of its token, so that its angles serve them all, once the call
    // has threads enough for the whole GPU. The prompts of eight sequences of 4096 tokens (12 heads,
    // d 64) take 62, 38, 28, 23, 24 us with 1, 2, 4, 8, 16 heads per thread; one token of 32
    // sequences (32 + 2 x 8 heads, d 128) 3.4, 3.6, 4.0, 5.1, 6.7 us, one call behind another.
    const long long all = (long long)B * T * p.slots * p.lanes;
    // (8-bit caches, the same prompts: 40, 35, 36, 32, 39 us with 4, 6, 8, 12, 18.)
    const int most = coded ? 12 : 8;
    p.per = all > most * kFullGpu ? most : all > kFullGpu ? (int)(all / kFullGpu) : 1;
    p.groups = (p.slots + p.per - 1) / p.per;
    const long long threads = (long long)T * p.groups * p.lanes;   // of a sequence: at most 2^21 x 96 x 8
    const long long blocks = (threads + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)blocks, (unsigned)(B < 65535 ? B : 65535));
    cudaStream_t cs = (cudaStream_t)stream;
    before_launch(SAF_KERNEL_KV_APPEND, cs);
    const cudaError_t err =
        launch_ex(coded ? (dt == SAF_BF16 ? append_codes_kernel<__nv_bfloat16> : append_codes_kernel<float>)
                        : (dt == SAF_BF16 ? append_kernel<__nv_bfloat16> : append_kernel<float>),
                  grid, dim3(kThreads), 0, cs, true, 1, p);
    after_launch(SAF_KERNEL_KV_APPEND, cs);
    return launch_status(err);
}

}  // namespace
}  // namespace saf

using namespace saf;

extern "C" {

int saf_kv_append(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* ctx,
                  const int32_t* n_new, const int32_t* page_table, int max_pages, const double* inv_freq, int rope_dim,
                  int interleaved, int64_t pos_base, const uint8_t* frozen, int B, int H, int Hkv, int T, int d,
                  int num_pages, int page_size, saf_dtype_t dt, void* q_out, void* k_cache, void* v_cache,
                  uint32_t* status, void* stream) {
    return append(q, k, v, strides, ctx, n_new, page_table, max_pages, inv_freq, rope_dim, interleaved, pos_base,
                  frozen, B, H, Hkv, T, d, num_pages, page_size, dt, false, q_out, k_cache, v_cache, nullptr, nullptr,
                  status, stream);
}

int saf_kv_append_quant(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* ctx,
                       const int32_t* n_new, const int32_t* page_table, int max_pages, const double* inv_freq,
                       int rope_dim, int interleaved, int64_t pos_base, const uint8_t* frozen, int B, int H, int Hkv,
                       int T, int d, int num_pages, int page_size, saf_dtype_t dt, void* q_out, void* k_cache,
                       void* v_cache, float* k_scale, float* v_scale, uint32_t* status, void* stream) {
    return append(q, k, v, strides, ctx, n_new, page_table, max_pages, inv_freq, rope_dim, interleaved, pos_base,
                  frozen, B, H, Hkv, T, d, num_pages, page_size, dt, true, q_out, k_cache, v_cache, k_scale, v_scale,
                  status, stream);
}

}  // extern "C"
