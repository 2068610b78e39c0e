// Host side of attention over a paged cache (saf_attn_paged, saf_attn_paged_shared):
// argument checks, the split of the keys over work items, the workspace, and the kernel
// that joins the items of a row.
#include <string.h>

#include "paged.h"

namespace saf {
namespace {

constexpr int kSms = 152;   // GB300
constexpr float kLn2 = 0.6931471805599453f;

// Items that run at the same time, and the most rounds of them that a call is split into.
constexpr int kSlotsSimt = kSms * 3, kSlotsTc = kSms * 2;
constexpr int kRounds = 8;
// What an item costs beside its tiles (the rows' counts, the first pages, the output, its share of
// the join), in tiles. Measured: 32 sequences of 4K to 16K tokens, 8 key/value heads, d 128 take
// 237, 211, 210, 218, 215 us with 2, 3, 5, 8, 12 items per sequence and head.
constexpr int kSetUp = 10;
// What the joining kernel costs, in tiles, where a call could do without one: one new token of
// one sequence (12 heads, d 64) takes 6.1 and 7.1 us with 1 and 2 items for 256 keys, 7.6 with 1
// and 4 for 512, 10.5 and 8.5 for 1024.
constexpr int kJoin = 3;

// Joins the items of a row. kWarps warps share a row (a block of four warps holds 4 / kWarps
// rows): with few items a warp each, with many the four warps of a block, whose loads are
// then all in flight together.
template <typename E, int D, int kWarps>
__global__ void __launch_bounds__(128) join_kernel(const float2* __restrict__ ml, const float* __restrict__ po,
                                                   E* __restrict__ o, float* __restrict__ lse, long long rows,
                                                   int nsplit) {
    __shared__ float4 part[4][32];
    __shared__ float part_l[4];
    grid_dep_wait();   // the items are done
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp % kWarps;
    const long long row = (long long)blockIdx.x * (4 / kWarps) + warp / kWarps;
    constexpr int kLanes = D / 4;             // lanes of one item's row
    constexpr int kSide = kLanes <= 16 ? 2 : 1;   // items next to each other in a warp
    const int side = kSide == 2 ? lane >> 4 : 0, c = kSide == 2 ? lane & 15 : lane;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) {
        const float2* r = ml + row * nsplit;
        for (int s = lane; s < nsplit; s += 32) M = fmaxf(M, r[s].x);
        for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        const float base = M == -INFINITY ? 0.f : M;   // a row that sees no key
#pragma unroll 4
        for (int s = mine * kSide + side; s < nsplit; s += kWarps * kSide) {
            const float2 e = r[s];
            const float w = exp2f(e.x - base);
            l += w * e.y;   // (a NaN sum stays one, whatever its weight)
            // an item whose keys the row does not see wrote no output
            if (w > 0.f && c < kLanes) {
                const float4 x = *reinterpret_cast<const float4*>(po + (row * nsplit + s) * D + 4 * c);
                acc.x = fmaf(w, x.x, acc.x);
                acc.y = fmaf(w, x.y, acc.y);
                acc.z = fmaf(w, x.z, acc.z);
                acc.w = fmaf(w, x.w, acc.w);
            }
        }
    }
    if (kSide == 2) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
    }
    if (kWarps > 1) {
        part[warp][lane] = acc;
        if (lane == 0) part_l[warp] = l;
        __syncthreads();
        if (mine != 0) return;
#pragma unroll
        for (int x = 1; x < kWarps; ++x) {
            const float4 y = part[warp + x][lane];
            acc.x += y.x;
            acc.y += y.y;
            acc.z += y.z;
            acc.w += y.w;
            l += part_l[warp + x];
        }
    }
    if (row >= rows) return;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    if (side == 0 && c < kLanes) {
        E* dst = o + row * D + 4 * c;
        from_f(dst, acc.x * inv);
        from_f(dst + 1, acc.y * inv);
        from_f(dst + 2, acc.z * inv);
        from_f(dst + 3, acc.w * inv);
    }
    if (lane == 0) lse[row] = l != 0.f ? (M + log2f(l)) * kLn2 : -INFINITY;
}

template <typename E, int D>
cudaError_t launch_join_d(const PagedArgs& p, cudaStream_t s) {
    const long long rows = (long long)p.B * p.H * p.T;
    if (p.nsplit > 8)
        return launch_ex(join_kernel<E, D, 4>, dim3((unsigned)rows), dim3(128), 0, s, true, 1, (const float2*)p.ml,
                         (const float*)p.po, (E*)p.o, p.lse, rows, p.nsplit);
    return launch_ex(join_kernel<E, D, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, true, 1,
                     (const float2*)p.ml, (const float*)p.po, (E*)p.o, p.lse, rows, p.nsplit);
}

template <typename E>
cudaError_t launch_join(const PagedArgs& p, cudaStream_t s) {
    switch (p.d) {
        case 96: return launch_join_d<E, 96>(p, s);
        case 128: return launch_join_d<E, 128>(p, s);
        default: return launch_join_d<E, 64>(p, s);
    }
}

long long ceil_div(long long x, long long y) { return (x + y - 1) / y; }

struct Plan {
    int tile[2], rows[2];
    int nrb[2], head_blocks[2];
    long long units[2];    // (sequence, key/value head, row block) triples
    long long tiles[2];    // key tiles of one of them, at most, without a window
    long long slots;       // items that run at the same time
    long long max_split;   // items of a row, at most, whatever the window
};

// Items along the keys of a part, at most: kRounds rounds of items over all units.
long long most_chunks(const Plan& x, int part, long long tiles) {
    const long long c = ceil_div(x.slots * kRounds, x.units[part]);
    return c < tiles ? c : tiles;
}

Plan make_plan(int B, int H, int Hkv, int T, int d, int max_len, int P, bool bf16) {
    Plan x;
    x.slots = bf16 ? kSlotsTc : kSlotsSimt;
    const long long G = H / Hkv;
    const long long n[2] = {P > 0 ? G * B * T : 0, G * T};
    const int keys[2] = {P, max_len};
    x.max_split = 0;
    for (int i = 0; i < 2; ++i) {
        // tensor cores: copies of the rows fill the 128 of a tile (paged_tc.cu)
        x.rows[i] = !bf16 ? kSimtRows : n[i] <= 32 ? 32 : n[i] <= 64 ? 64 : 128;
        x.tile[i] = bf16 ? paged_tc_tile(d, x.rows[i]) : kSimtTile;
        // several blocks to a head: each head begins its own
        const long long per_head = n[i] / G;
        x.head_blocks[i] = per_head >= 4 * x.rows[i] ? (int)ceil_div(per_head, x.rows[i]) : 0;
        x.nrb[i] = (int)(x.head_blocks[i] ? G * x.head_blocks[i] : ceil_div(n[i], x.rows[i]));
        x.units[i] = (long long)x.nrb[i] * Hkv * (i ? B : 1);
        x.tiles[i] = ceil_div(keys[i], x.tile[i]);
        if (x.units[i]) x.max_split += most_chunks(x, i, x.tiles[i]);
    }
    return x;
}

// Items along the keys for `units` units of `nt` tiles each: the number that makes the part
// shortest, with `slots` items at a time. even: the units have the same length, so that rounds
// end together; else their lengths differ, and the last items run alone for a while.
// Candidates: one, the most items that fit in 1, 2, ... rounds, and the minimum over c of
// (units c / slots) (kSetUp + nt / c) + nt / c, the work and the tail of c items per unit.
long long pick_chunks(long long units, long long nt, long long most, long long slots, bool even, bool joins_anyway) {
    long long best = 1;
    double best_cost = 1e300;
    for (int r = -1; r <= kRounds; ++r) {
        long long c = r < 0 ? 1 : r ? slots * r / units
                        : (long long)sqrt((double)nt * (double)slots / ((double)units * (double)kSetUp));
        c = c < 1 ? 1 : c > most ? most : c;
        const long long per = ceil_div(nt, c);
        const double rounds = (double)(units * ceil_div(nt, per)) / (double)slots;
        const double cost =
            (even ? ceil(rounds) : rounds + 1.0) * (double)(kSetUp + per) + (c > 1 && !joins_anyway ? kJoin : 0);
        if (cost < best_cost || (cost == best_cost && c < best)) {
            best_cost = cost;
            best = c;
        }
    }
    return best;
}

void set_items(PagedArgs& p, const Plan& x, int nfrozen) {
    long long nt[2] = {x.tiles[0], x.tiles[1]};
    const bool windowed = p.window > 0 && nfrozen == 0;
    unsigned items[2];
    long long slots = x.slots;
    for (int i = 1; i >= 0; --i) {
        p.nrb[i] = x.nrb[i];
        p.head_blocks[i] = x.head_blocks[i];
        p.rows[i] = x.rows[i];
        p.tile[i] = x.tile[i];
        p.chunks[i] = p.per_chunk[i] = 0;
        items[i] = 0;
        if (x.units[i] == 0) continue;
        if (windowed) {
            // a block's rows stand within T positions (or as many as it has rows) in part 1 and past
            // the prefix in part 0: the tiles that hold that many keys more than the window less
            // one, and those of the sinks
            const long long spread = i == 0 ? 1 : x.head_blocks[1] ? x.rows[1] : p.T;
            const long long span = p.window + spread - 1;
            const long long off = i ? p.P : 0;
            const long long sinks = p.sinks > off ? p.sinks - off : 0;
            const long long n = ceil_div(span, x.tile[i]) + 1 + ceil_div(sinks, x.tile[i]);
            if (n < nt[i]) nt[i] = n;
        }
        // (a prefix's units have the same length, and so have windows)
        const long long c = pick_chunks(x.units[i], nt[i], most_chunks(x, i, nt[i]), slots, i == 0 || windowed,
                                        p.P > 0);
        p.per_chunk[i] = (int)ceil_div(nt[i], c);
        p.chunks[i] = (int)ceil_div(nt[i], p.per_chunk[i]);
        items[i] = (unsigned)(x.units[i] * p.chunks[i]);
        // Few own items run beside the prefix's, in the same round. (Half of the slots for the
        // prefix beside many own items was slower: 176 against 111 us for 64 sequences after 32K.)
        if (items[i] < slots / 2) slots -= items[i];
    }
    p.nsplit = p.chunks[0] + p.chunks[1];
    p.items0 = items[0];
    p.items = items[0] + items[1];
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t workspace_bytes(const Plan& x, int B, int H, int T, int d, size_t* po_off) {
    const size_t rows = (size_t)B * H * T;
    const size_t ml = align256(rows * (size_t)x.max_split * sizeof(float2));
    if (po_off) *po_off = kStatusBytes + ml;
    if (x.max_split <= 1) return kStatusBytes;
    return kStatusBytes + ml + align256(rows * (size_t)x.max_split * d * sizeof(float));
}

bool power_of_two(int n) { return n > 0 && (n & (n - 1)) == 0; }
bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Sizes, in the order of the workspace query and of both calls.
int check_sizes(int B, int H, int Hkv, int T, int d, int max_len, int prefix_len, saf_dtype_t dt) {
    if (B < 0 || H <= 0 || T < 0 || H > SAF_MAX_HEADS || Hkv <= 0 || H % Hkv != 0) return SAF_EINVAL;
    if (dt != SAF_BF16 && dt != SAF_FP32) return SAF_EINVAL;
    if (!head_dim_supported(d, dt)) return SAF_EUNSUPPORTED;
    if (max_len < 1 || prefix_len < 0 || (long long)max_len + prefix_len > (1ll << 30)) return SAF_EINVAL;
    if ((long long)B * H * T > (1ll << 29)) return SAF_EINVAL;   // (items are counted in 32 bits)
    return SAF_OK;
}

int paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* prefix_pages, int prefix_len,
          const int32_t* page_table, int max_pages, const int32_t* ctx, const int32_t* n_new, const float* a,
          const float* r, int ld_prior, const uint8_t* frozen, int window, int sinks, int B, int H, int Hkv, int T,
          int d, int max_len, int num_pages, int page_size, saf_dtype_t dt, void* o, float* lse, void* workspace,
          size_t ws_bytes, void* stream) {
    int st = check_sizes(B, H, Hkv, T, d, max_len, prefix_len, dt);
    if (st != SAF_OK) return st;
    if (window < 0 || sinks < 0) return SAF_EINVAL;
    if (B == 0 || T == 0) return SAF_OK;
    if (!power_of_two(page_size) || page_size < 8 || page_size > 1024) return SAF_EINVAL;
    if (num_pages < 1 || max_pages < 1 || (long long)num_pages * Hkv > 0x7fffffffll) return SAF_EINVAL;
    if (max_len > (long long)max_pages * page_size) return SAF_EINVAL;
    PagedArgs p;
    memset(&p, 0, sizeof(p));
    const int G = H / Hkv;
    int nfrozen = 0;
    for (int hk = 0; hk < Hkv; ++hk) {   // a group's ordinary query heads first
        int n = 0;
        for (int pass = 0; pass < 2; ++pass)
            for (int gi = 0; gi < G; ++gi) {
                const int h = hk * G + gi;
                if ((frozen && frozen[h]) == (pass == 1)) p.gheads[hk * G + n++] = (uint8_t)h;
            }
        int f = 0;
        for (int gi = 0; gi < G; ++gi)
            if (frozen && frozen[hk * G + gi]) {
                p.mask.w[(hk * G + gi) >> 6] |= 1ull << ((hk * G + gi) & 63);
                ++f;
            }
        p.gord[hk] = (uint16_t)(G - f);
        nfrozen += f;
    }
    if (!v_cache || !page_table || !ctx || !o || !lse || (prefix_len > 0 && !prefix_pages)) return SAF_EINVAL;
    if (nfrozen < H && (!q || !k_cache)) return SAF_EINVAL;
    if (nfrozen > 0 && (!a || !r || ld_prior < prefix_len + max_len)) return SAF_EINVAL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(a, 4) || !aligned(r, 4) || !aligned(page_table, 4) || !aligned(prefix_pages, 4) ||
        !aligned(ctx, 4) || !aligned(n_new, 4))
        return SAF_EALIGN;
    if (!workspace) return SAF_EWORKSPACE;
    if (!aligned(workspace, 256)) return SAF_EALIGN;
    const Plan plan = make_plan(B, H, Hkv, T, d, max_len, prefix_len, dt == SAF_BF16);
    size_t po_off;
    if (ws_bytes < workspace_bytes(plan, B, H, T, d, &po_off)) return SAF_EWORKSPACE;
    if ((st = check_device()) != SAF_OK) return st;

    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.prefix_pages = prefix_pages;
    p.page_table = page_table;
    p.ctx = ctx;
    p.n_new = n_new;
    p.a = a;
    p.r = r;
    p.o = o;
    p.lse = lse;
    p.status = (uint32_t*)workspace;
    p.ml = (float2*)((char*)workspace + kStatusBytes);
    p.po = (float*)((char*)workspace + po_off);
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.G = G;
    p.T = T;
    p.d = d;
    p.ld = ld_prior;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    while ((1 << p.page_log2) < page_size) ++p.page_log2;
    p.P = prefix_len;
    p.max_len = max_len;
    p.window = window >= prefix_len + max_len ? 0 : window;   // a window that reaches every key is none
    p.sinks = sinks < prefix_len + max_len ? sinks : prefix_len + max_len;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)d);
    set_items(p, plan, nfrozen);

    cudaStream_t s = (cudaStream_t)stream;
    const bool bf16 = dt == SAF_BF16;
    before_launch(SAF_KERNEL_PAGED, s);
    cudaError_t e = bf16 ? launch_paged_tc(p, s) : launch_paged_simt(p, s);
    if (e == cudaSuccess && p.nsplit > 1) {
        note_launch();
        e = bf16 ? launch_join<__nv_bfloat16>(p, s) : launch_join<float>(p, s);
    }
    after_launch(SAF_KERNEL_PAGED, s);
    return launch_status(e);
}

}  // namespace
}  // namespace saf

using namespace saf;

extern "C" {

size_t saf_attn_paged_workspace_bytes(int B, int H, int Hkv, int T, int d, int max_len, int prefix_len,
                                      saf_dtype_t dt) {
    if (check_sizes(B, H, Hkv, T, d, max_len, prefix_len, dt) != SAF_OK) return 0;
    if (B == 0 || T == 0) return kStatusBytes;
    return workspace_bytes(make_plan(B, H, Hkv, T, d, max_len, prefix_len, dt == SAF_BF16), B, H, T, d, nullptr);
}

int saf_attn_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table, int max_pages,
                   const int32_t* ctx, const int32_t* n_new, const float* a, const float* r, int ld_prior,
                   const uint8_t* frozen, int window, int sinks, int B, int H, int Hkv, int T, int d, int max_len,
                   int num_pages, int page_size, saf_dtype_t dt, void* o, float* lse, void* workspace,
                   size_t ws_bytes, void* stream) {
    return paged(q, k_cache, v_cache, nullptr, 0, page_table, max_pages, ctx, n_new, a, r, ld_prior, frozen, window,
                 sinks, B, H, Hkv, T, d, max_len, num_pages, page_size, dt, o, lse, workspace, ws_bytes, stream);
}

int saf_attn_paged_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* prefix_pages,
                          int prefix_len, const int32_t* page_table, int max_pages, const int32_t* ctx,
                          const int32_t* n_new, const float* a, const float* r, int ld_prior, const uint8_t* frozen,
                          int window, int sinks, int B, int H, int Hkv, int T, int d, int max_len, int num_pages,
                          int page_size, saf_dtype_t dt, void* o, float* lse, void* workspace, size_t ws_bytes,
                          void* stream) {
    return paged(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, max_pages, ctx, n_new, a, r, ld_prior,
                 frozen, window, sinks, B, H, Hkv, T, d, max_len, num_pages, page_size, dt, o, lse, workspace,
                 ws_bytes, stream);
}

}  // extern "C"
