// Keys and values of new tokens into a paged cache, with the rotary position rotation of
// k (and of q, for the attention that follows) on the way.
//
// Token t of sequence b goes to slot x = ctx[b] + t of the sequence: row x mod page of page
// table[b][x / page]. Pair c of a row's first `rope_dim` elements is turned by the angle
// pos * f_c with pos = pos_base + x:
//     (y0, y1) = (x0 cos - x1 sin, x0 sin + x1 cos),
// in fp32, rounded once to the cache's type. Angles of far positions keep their digits: the
// host turns f_c into F_c = (f_c / 2 pi mod 1) 2^64, and pos * F_c in 64-bit integers is the
// angle in turns, modulo one, to 2^-64 of a turn per position.
//
// Bound by memory: every element is read once and written once; the angles cost one
// sincospif per pair and token for several heads. Thread = 16 elements of a row (8 pairs) of
// `per` heads of a token, so that neighbouring threads read whole rows.
#include <math.h>
#include <string.h>

#include "saf_internal.h"

namespace saf {
namespace {

constexpr int kThreads = 128;

struct AppendArgs {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    const int32_t *ctx, *n_new, *table;
    uint32_t* status;
    long long sq[3], sk[3], sv[3];   // element strides (sequence, head, token)
    long long pos_base;
    int B, H, Hkv, T, d, max_pages, num_pages, page_log2;
    int rope, interleaved;
    int units;                       // d / 16
    int nq, nk, slots;               // heads of q, of k, and all with v's that are moved
    int per, groups;                 // slots of a thread; ceil(slots / per)
    uint64_t freq[64];               // F_c
    uint8_t heads[2 * SAF_MAX_HEADS];   // nq query heads, then nk key heads
};

template <typename E>
struct Vec;   // 8 elements
template <>
struct Vec<float> {
    float x[8];
    __device__ void load(const float* p) {
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(p);
        *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ void store(float* p) const {
        *reinterpret_cast<float4*>(p) = *reinterpret_cast<const float4*>(x);
        *reinterpret_cast<float4*>(p + 4) = *reinterpret_cast<const float4*>(x + 4);
    }
};
template <>
struct Vec<__nv_bfloat16> {
    float x[8];
    __device__ void load(const __nv_bfloat16* p) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    __device__ void store(__nv_bfloat16* p) const {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename E>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs p) {
    grid_dep_wait();
    grid_dep_launch();
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int u = (int)(id % p.units);
    long long rest = id / p.units;
    const int group = (int)(rest % p.groups);
    rest /= p.groups;
    const int t = (int)(rest % p.T), b = (int)(rest / p.T);
    if (b >= p.B) return;
    const int c = p.ctx[b];
    const int n = p.n_new ? p.n_new[b] : p.T;
    const long long room = (long long)p.max_pages << p.page_log2;
    if (c < 0 || n < 0 || n > p.T || c + (long long)n > room) {
        if (t == 0 && group == 0 && u == 0 && p.status) atomicOr(p.status, kStatusPage);
        if (c < 0) return;
    }
    if (t >= n) return;
    const long long slot = (long long)c + t;
    int page = slot < room ? p.table[(size_t)b * p.max_pages + (slot >> p.page_log2)] : -1;
    if (slot < room && (page < 0 || page >= p.num_pages)) {
        if (group == 0 && u == 0 && p.status) atomicOr(p.status, kStatusPage);
        page = -1;
    }
    const size_t page_row = (size_t)(slot & ((1 << p.page_log2) - 1));

    // my 16 elements: two runs of 8, for a rotated row's pairs (8u + e, rope / 2 + 8u + e) when
    // the pairs are halves apart
    const bool turn = 16 * u < p.rope;
    const int c0 = turn && !p.interleaved ? 8 * u : 16 * u;
    const int c1 = turn && !p.interleaved ? (p.rope >> 1) + 8 * u : 16 * u + 8;
    float cs[8], sn[8];
    const int s0 = group * p.per, s1 = min(s0 + p.per, p.slots);
    if (turn && s0 < p.nq + p.nk) {
        const uint64_t pos = (uint64_t)(p.pos_base + slot);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // the angle in half turns, in [-1, 1)
            const int32_t x = (int32_t)((pos * p.freq[8 * u + e]) >> 32);
            sincospif((float)x * 4.656612873077393e-10f, &sn[e], &cs[e]);   // 2^-31
        }
    }
    for (int s = s0; s < s1; ++s) {
        const bool is_q = s < p.nq, is_v = s >= p.nq + p.nk;
        const int h = is_v ? s - p.nq - p.nk : p.heads[s];
        const E* src;
        E* dst;
        if (is_q) {
            src = (const E*)p.q + b * p.sq[0] + h * p.sq[1] + t * p.sq[2];
            dst = (E*)p.q_out + (((size_t)b * p.H + h) * p.T + t) * p.d;
        } else {
            if (page < 0) continue;
            const long long* st = is_v ? p.sv : p.sk;
            src = (const E*)(is_v ? p.v : p.k) + b * st[0] + h * st[1] + t * st[2];
            dst = (E*)(is_v ? p.v_cache : p.k_cache) +
                  ((((size_t)page * p.Hkv + h) << p.page_log2) + page_row) * p.d;
        }
        const int o0 = is_v ? 16 * u : c0, o1 = is_v ? 16 * u + 8 : c1;
        Vec<E> x, y;
        x.load(src + o0);
        y.load(src + o1);
        if (turn && !is_v) {
            if (!p.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = x.x[e], z = y.x[e];
                    x.x[e] = a * cs[e] - z * sn[e];
                    y.x[e] = a * sn[e] + z * cs[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a = x.x[2 * e], z = x.x[2 * e + 1];
                    x.x[2 * e] = a * cs[e] - z * sn[e];
                    x.x[2 * e + 1] = a * sn[e] + z * cs[e];
                    a = y.x[2 * e], z = y.x[2 * e + 1];
                    y.x[2 * e] = a * cs[4 + e] - z * sn[4 + e];
                    y.x[2 * e + 1] = a * sn[4 + e] + z * cs[4 + e];
                }
            }
        }
        x.store(dst + o0);
        y.store(dst + o1);
    }
}

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace
}  // namespace saf

using namespace saf;

extern "C" int saf_kv_append(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* ctx,
                             const int32_t* n_new, const int32_t* page_table, int max_pages, const double* inv_freq,
                             int rope_dim, int interleaved, int64_t pos_base, const uint8_t* frozen, int B, int H,
                             int Hkv, int T, int d, int num_pages, int page_size, saf_dtype_t dt, void* q_out,
                             void* k_cache, void* v_cache, uint32_t* status, void* stream) {
    if (B < 0 || H <= 0 || T < 0 || H > SAF_MAX_HEADS || Hkv <= 0 || H % Hkv != 0) return SAF_EINVAL;
    if (dt != SAF_BF16 && dt != SAF_FP32) return SAF_EINVAL;
    if (!head_dim_supported(d, dt)) return SAF_EUNSUPPORTED;
    if (rope_dim < 0 || rope_dim > d || rope_dim % 16 != 0 || (rope_dim > 0 && !inv_freq)) return SAF_EINVAL;
    if (interleaved != 0 && interleaved != 1) return SAF_EINVAL;
    if (pos_base < 0 || (long long)B * T > (1ll << 30)) return SAF_EINVAL;
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
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(ctx, 4) || !aligned(n_new, 4) || !aligned(page_table, 4) ||
        !aligned(status, 4))
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
        const double turns = inv_freq[c] * 0.15915494309189533577;   // 1 / (2 pi)
        const double frac = turns - floor(turns);                    // in [0, 1]
        p.freq[c] = frac < 1.0 ? (uint64_t)(frac * 18446744073709551616.0) : 0;
    }
    int s = check_device();
    if (s != SAF_OK) return s;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
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
    p.slots = p.nq + p.nk + Hkv;
    p.per = 1;
    p.groups = p.slots;
    const long long threads = (long long)B * T * p.groups * p.units;
    const long long blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffll) return SAF_EINVAL;
    cudaStream_t cs = (cudaStream_t)stream;
    before_launch(SAF_KERNEL_KV_APPEND, cs);
    const cudaError_t err =
        dt == SAF_BF16 ? launch_ex(append_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(kThreads), 0, cs, true, 1, p)
                       : launch_ex(append_kernel<float>, dim3((unsigned)blocks), dim3(kThreads), 0, cs, true, 1, p);
    after_launch(SAF_KERNEL_KV_APPEND, cs);
    return launch_status(err);
}
