// Rows of the 8-bit paged cache (see kv_append.cu) back as bf16 or fp32: token t of sequence b
// is slot x = first[b] + t, value code_c * scale, rounded once.
//
// Bound by memory: a row is read once (d + 4 bytes) and written once. Thread = 16 bytes of a written row of k and
// of v (8 or 4 codes), so that a warp's stores are whole lines, for several tokens of one key/value
// head whose reads are on their way together. Four contexts of up to 16K tokens of 8 heads of 128 (354 MB) take
// 55 us, 95% of a plain copy's rate; 66 with 16 codes of one token to a thread.
#include <cuda_fp8.h>
#include <string.h>

#include "saf_internal.h"

namespace saf {
namespace {

constexpr int kThreads = 128;
constexpr long long kFullGpu = 152ll * 2048;   // threads that the GPU holds
constexpr int kManyRows = 2;                   // tokens of a thread, once the GPU is full without

struct ReadArgs {
    const uint8_t *k_cache, *v_cache;   // k_cache may be NULL: values only
    const float *k_scale, *v_scale;
    const int32_t *first, *count, *table;
    void *k_out, *v_out;                // [B, Hkv, T, d]
    uint32_t* status;
    int B, Hkv, T, d, max_pages, num_pages, page_log2;
    int units;                          // threads of a row
};

// The codes that make 16 bytes of a row, times their row's scale.
struct Eight {   // bf16
    using Codes = uint2;
    static constexpr int count = 8;
    __device__ __forceinline__ static uint4 values(Codes c, float scale) {
        return make_uint4(pair(c.x, scale), pair(c.x >> 16, scale), pair(c.y, scale), pair(c.y >> 16, scale));
    }
    __device__ __forceinline__ static uint32_t pair(uint32_t codes, float scale) {
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3)));
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
struct Four {   // fp32
    using Codes = uint32_t;
    static constexpr int count = 4;
    __device__ __forceinline__ static uint4 values(Codes c, float scale) {
        const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
        const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3)));
        return make_uint4(__float_as_uint(a.x * scale), __float_as_uint(a.y * scale), __float_as_uint(b.x * scale),
                          __float_as_uint(b.y * scale));
    }
};

// X: Eight or Four. kRows: tokens of a thread, a block's threads apart.
template <typename X, int kRows>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs p) {
    grid_dep_wait();
    grid_dep_launch();
    const unsigned id = blockIdx.x * (kThreads * kRows) + threadIdx.x;   // (token, unit)
    for (unsigned z = blockIdx.y; z < (unsigned)p.B * (unsigned)p.Hkv; z += gridDim.y) {
        const int b = (int)(z / (unsigned)p.Hkv), hk = (int)(z - (unsigned)b * (unsigned)p.Hkv);
        const int c = p.first ? p.first[b] : 0, n = p.count ? p.count[b] : p.T;
        const long long room = (long long)p.max_pages << p.page_log2;
        if ((c < 0 || n < 0 || n > p.T || c + (long long)n > room) && id == 0 && hk == 0 && p.status)
            atomicOr(p.status, kStatusPage);
        typename X::Codes ck[kRows], cv[kRows];
        float sk[kRows], sv[kRows];
        int page[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int t = (int)((id + k * kThreads) / (unsigned)p.units);
            const long long slot = (long long)c + t;
            page[k] = -2;   // no token
            if (c >= 0 && t < n && t < p.T && slot < room) {
                page[k] = p.table[(size_t)b * p.max_pages + (slot >> p.page_log2)];
                if (page[k] < 0 || page[k] >= p.num_pages) page[k] = -1;
            }
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {   // rows without a token are zeros
            const unsigned at = id + k * kThreads;
            const int t = (int)(at / (unsigned)p.units), u = (int)(at - (unsigned)t * (unsigned)p.units);
            ck[k] = cv[k] = typename X::Codes{};
            sk[k] = sv[k] = 0.f;
            if (page[k] >= 0) {
                const size_t row = (((size_t)page[k] * p.Hkv + hk) << p.page_log2) + (((unsigned)c + (unsigned)t) & ((1u << p.page_log2) - 1u));
                if (p.k_cache) {
                    ck[k] = *reinterpret_cast<const typename X::Codes*>(p.k_cache + row * p.d + X::count * u);
                    sk[k] = p.k_scale[row];
                }
                cv[k] = *reinterpret_cast<const typename X::Codes*>(p.v_cache + row * p.d + X::count * u);
                sv[k] = p.v_scale[row];
            } else if (page[k] == -1 && u == 0 && hk == 0 && p.status) {
                atomicOr(p.status, kStatusPage);
            }
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const unsigned at = id + k * kThreads;
            if (at / (unsigned)p.units >= (unsigned)p.T) continue;
            // (units of 16 bytes lie next to each other from token to token)
            const size_t out = (size_t)z * p.T * p.units + at;
            if (p.k_cache) reinterpret_cast<uint4*>(p.k_out)[out] = X::values(ck[k], sk[k]);
            reinterpret_cast<uint4*>(p.v_out)[out] = X::values(cv[k], sv[k]);
        }
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
    p.units = d / (dt == SAF_BF16 ? Eight::count : Four::count);
    const long long threads = (long long)T * p.units;   // of a sequence and head: at most 2^21 x 32
    const bool many = threads * B * Hkv > 4ll * kFullGpu;
    const long long per_block = kThreads * (many ? kManyRows : 1);
    const long long blocks = (threads + per_block - 1) / per_block;
    const long long rows = (long long)B * Hkv;
    const dim3 grid((unsigned)blocks, (unsigned)(rows < 65535 ? rows : 65535));
    cudaStream_t cs = (cudaStream_t)stream;
    before_launch(SAF_KERNEL_KV_READ, cs);
    const cudaError_t err =
        launch_ex(dt == SAF_BF16 ? (many ? read_kernel<Eight, kManyRows> : read_kernel<Eight, 1>)
                                 : (many ? read_kernel<Four, kManyRows> : read_kernel<Four, 1>),
                  grid, dim3(kThreads), 0, cs, true, 1, p);
    after_launch(SAF_KERNEL_KV_READ, cs);
    return launch_status(err);
}
