// Rows of the 8-bit paged cache (see kv_append.cu) back as bf16 or fp32: token t of sequence b
// is slot x = first[b] + t, value code_c * scale, rounded once.
//
// Bound by memory: a row is read once (d + 4 bytes) and written once. Thread = 16 codes of a row
// of k and of v; a block's threads hold neighbouring tokens of one key/value head.
#include <cuda_fp8.h>
#include <string.h>

#include "saf_internal.h"

namespace saf {
namespace {

constexpr int kThreads = 128;

struct ReadArgs {
    const uint8_t *k_cache, *v_cache;   // k_cache may be NULL: values only
    const float *k_scale, *v_scale;
    const int32_t *first, *count, *table;
    void *k_out, *v_out;                // [B, Hkv, T, d]
    uint32_t* status;
    int B, Hkv, T, d, max_pages, num_pages, page_log2;
    int units;                          // d / 16
};

// 16 codes of e4m3, times their row's scale.
__device__ __forceinline__ void values16(const uint4& c, float scale, float* x) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e >> 1] >> (16 * (e & 1))), __NV_E4M3));
        const float2 f = __half22float2(h);
        x[2 * e] = f.x * scale;
        x[2 * e + 1] = f.y * scale;
    }
}

__device__ __forceinline__ void put16(float* p, const float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        reinterpret_cast<float4*>(p)[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
}
__device__ __forceinline__ void put16(__nv_bfloat16* p, const float* x) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename E>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs p) {
    grid_dep_wait();
    grid_dep_launch();
    const unsigned id = blockIdx.x * kThreads + threadIdx.x;   // (token, unit)
    const int t = (int)(id / (unsigned)p.units), u = (int)(id - (unsigned)t * (unsigned)p.units);
    if (t >= p.T) return;
    for (unsigned z = blockIdx.y; z < (unsigned)p.B * (unsigned)p.Hkv; z += gridDim.y) {
        const int b = (int)(z / (unsigned)p.Hkv), hk = (int)(z - (unsigned)b * (unsigned)p.Hkv);
        const int c = p.first ? p.first[b] : 0, n = p.count ? p.count[b] : p.T;
        const long long room = (long long)p.max_pages << p.page_log2;
        if ((c < 0 || n < 0 || n > p.T || c + (long long)n > room) && t == 0 && u == 0 && hk == 0 && p.status)
            atomicOr(p.status, kStatusPage);
        const long long slot = (long long)c + t;
        uint4 ck = make_uint4(0, 0, 0, 0), cv = ck;   // rows without a token are zeros
        float sk = 0.f, sv = 0.f;
        if (c >= 0 && t < n && slot < room) {
            const int page = p.table[(size_t)b * p.max_pages + (slot >> p.page_log2)];
            if (page >= 0 && page < p.num_pages) {
                const size_t row = (((size_t)page * p.Hkv + hk) << p.page_log2) + (slot & ((1 << p.page_log2) - 1));
                if (p.k_cache) {
                    ck = *reinterpret_cast<const uint4*>(p.k_cache + row * p.d + 16 * u);
                    sk = p.k_scale[row];
                }
                cv = *reinterpret_cast<const uint4*>(p.v_cache + row * p.d + 16 * u);
                sv = p.v_scale[row];
            } else if (u == 0 && hk == 0 && p.status) {
                atomicOr(p.status, kStatusPage);
            }
        }
        const size_t out = ((size_t)z * p.T + t) * p.d + 16 * u;
        float x[16];
        if (p.k_cache) {
            values16(ck, sk, x);
            put16((E*)p.k_out + out, x);
        }
        values16(cv, sv, x);
        put16((E*)p.v_out + out, x);
    }
}

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace
}  // namespace saf

using namespace saf;

extern "C" int saf_kv_read_quant(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                                const int32_t* page_table, int max_pages, const int32_t* first, const int32_t* count,
                                int B, int Hkv, int T, int d, int num_pages, int page_size, saf_dtype_t dt,
                                void* k_out, void* v_out, uint32_t* status, void* stream) {
    if (B < 0 || Hkv <= 0 || Hkv > SAF_MAX_HEADS || T < 0) return SAF_EINVAL;
    if (dt != SAF_BF16 && dt != SAF_FP32) return SAF_EINVAL;
    if (!head_dim_supported(d, dt)) return SAF_EUNSUPPORTED;
    if (T > (1 << 21) || (long long)B * T > (1ll << 30)) return SAF_EINVAL;
    if (B == 0 || T == 0) return SAF_OK;
    if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return SAF_EINVAL;
    if (num_pages < 1 || max_pages < 1) return SAF_EINVAL;
    if (!v_cache || !v_scale || !v_out || !page_table) return SAF_EINVAL;
    if (k_cache ? (!k_scale || !k_out) : k_out != nullptr) return SAF_EINVAL;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16) ||
        !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(page_table, 4) || !aligned(first, 4) ||
        !aligned(count, 4) || !aligned(status, 4))
        return SAF_EALIGN;
    const int st = check_device();
    if (st != SAF_OK) return st;
    ReadArgs p;
    memset(&p, 0, sizeof(p));
    p.k_cache = (const uint8_t*)k_cache;
    p.v_cache = (const uint8_t*)v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.first = first;
    p.count = count;
    p.table = page_table;
    p.k_out = k_out;
    p.v_out = v_out;
    p.status = status;
    p.B = B;
    p.Hkv = Hkv;
    p.T = T;
    p.d = d;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    while ((1 << p.page_log2) < page_size) ++p.page_log2;
    p.units = d / 16;
    const long long blocks = ((long long)T * p.units + kThreads - 1) / kThreads;   // at most 2^21 x 8 / 128
    const long long rows = (long long)B * Hkv;
    const dim3 grid((unsigned)blocks, (unsigned)(rows < 65535 ? rows : 65535));
    cudaStream_t cs = (cudaStream_t)stream;
    before_launch(SAF_KERNEL_KV_READ, cs);
    const cudaError_t err = launch_ex(dt == SAF_BF16 ? read_kernel<__nv_bfloat16> : read_kernel<float>, grid,
                                      dim3(kThreads), 0, cs, true, 1, p);
    after_launch(SAF_KERNEL_KV_READ, cs);
    return launch_status(err);
}
