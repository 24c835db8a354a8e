// sas_append_paged, sas_append_paged_q8: new tokens into the pages of a paged
// KV cache, with the head norm and the position rotation of q and k on the way.
//
//   k' = R(pos) (k r w_k), v' = v into page page_table[n, pos / 64], row pos % 64;
//   q' = R(pos) (q r w_q) to q_out.
// 8-bit pages hold code = e4m3(x / s) with one fp32 scale s for each (page, KV
// head): the least power of two with max|x| <= 448 s over the rows written so
// far. A power of two keeps the codes' full precision (e4m3 is a floating
// type), and lets older rows be expressed in a grown scale exactly, down to the
// codes' subnormals. Norm, rotation and the division are in fp32; each value
// is rounded once.
//
// One launch: the first CTAs take the query heads (four heads of a token for
// each row slot, head_row.cuh), the others one (sequence, block, KV head) of
// K or of V each, so that the rows of a page that is new to this call are read
// and written once, its amax needs no second pass, and no two CTAs share a
// scale. Bound by HBM for prompts, by the launch for single tokens.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "head_row.cuh"
#include "launch.h"
#include "page_rows.h"

namespace sas {
namespace {

constexpr int kThreads = 128;

using bf16 = __nv_bfloat16;

__device__ __forceinline__ SeqNew load_seq(const AppendArgs& a, int n) {
    const bool cu = a.cu_new != nullptr;
    return seq_new(cu, cu ? __ldg(a.cu_new + n) : 0, cu ? __ldg(a.cu_new + n + 1) : 0, n, a.T, a.max_new,
                   __ldg(a.kv_len + n), a.max_pages, a.max_pos);
}

// Sequence that owns token row t, or -1.
__device__ __forceinline__ int seq_of_row(const AppendArgs& a, long long t) {
    if (a.cu_new == nullptr) return (int)t;
    int lo = 0, hi = a.N;                        // the last n with cu[n] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu_new + mid) <= t) lo = mid; else hi = mid;
    }
    return __ldg(a.cu_new + lo) <= t && t < __ldg(a.cu_new + lo + 1) ? lo : -1;
}

constexpr int kHeads = 4;       // query heads of one token that a row slot takes

template <int D>
__device__ __forceinline__ void append_q(const AppendArgs& a, uint32_t cta) {
    constexpr int kSlots = kThreads / HeadRow<D>::kLanes;
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    const uint32_t parts = ((uint32_t)a.Hq + kHeads - 1) / kHeads;
    const uint32_t u = cta * kSlots + threadIdx.x / HeadRow<D>::kLanes, t = u / parts, h0 = u - t * parts;
    // the rows' loads are on their way before the token's sequence is looked for
    const bf16* src = static_cast<const bf16*>(a.q) + (t < a.T ? t * a.ld_q : 0) + 8 * l;
    uint4 lo[kHeads][1], hi[kHeads][1];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = (int)(h0 + i * parts);
        lo[i][0] = hi[i][0] = make_uint4(0u, 0u, 0u, 0u);
        if (t < a.T && h < a.Hq) {
            lo[i][0] = ld_stream(src + h * D);
            hi[i][0] = ld_stream(src + h * D + D / 2);
        }
    }
    const bf16* weight = static_cast<const bf16*>(a.q_weight);
    const Row w = load_weight<bf16, D>(weight, l);
    // -1: a padding entry, whose row is zero; rows of no sequence, or of one that is skipped, stay as they are
    int pos = -1;
    bool live = t < a.T;
    if (live) {
        const int n = seq_of_row(a, t);
        live = n >= 0;
        if (live) {
            const SeqNew s = load_seq(a, n);
            live = !s.bad;
            if (s.count > 0) pos = s.first + (int)(t - s.row0);
        }
    }
    const Turn turn(load_angles<bf16, D>(a.table, live ? max(pos, 0) : 0, l), w);
    bf16* dst = static_cast<bf16*>(a.q_out) + (long long)t * a.Hq * D;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = (int)(h0 + i * parts);
        Row x;
        x.a = Raw8<bf16>::get(lo[i]);
        x.b = Raw8<bf16>::get(hi[i]);
        Row y = turn(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);
        if (pos < 0) y.a = y.b = Half{};
        if (live && h < a.Hq) {
            store_row<D>(dst + h * D, l, y);
        }
    }
}

// Eight e4m3 codes (8 bytes) from eight values times inv, and back.
__device__ __forceinline__ uint2 to_codes(const Half& x, float inv) {
    const f2 ii = f2_pack(inv, inv);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __nv_cvt_float2_to_fp8x2(f2_unpack(f2_mul(x.v[i], ii)), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
__device__ __forceinline__ Half from_codes(uint2 c) {
    const uint32_t w[2] = {c.x, c.y};
    Half h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
        h.v[i] = f2_pack(f.x, f.y);
    }
    return h;
}
__device__ __forceinline__ void add(Half& s, const Half& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s.v[i] = f2_add(s.v[i], x.v[i]);
}
// An infinity has no code: it is kept as NaN. Returns the largest finite magnitude so far.
__device__ __forceinline__ float finite_max(Half& x, float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = f2_unpack(x.v[i]);
        if (!(fabsf(f.x) <= 3.402823466e38f)) f.x = __int_as_float(0x7fffffff);
        if (!(fabsf(f.y) <= 3.402823466e38f)) f.y = __int_as_float(0x7fffffff);
        m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
        x.v[i] = f2_pack(f.x, f.y);
    }
    return m;
}

template <int D, bool kQ8>
__device__ __forceinline__ void append_kv(const AppendArgs& a, long long item) {
    constexpr int kLanes = HeadRow<D>::kLanes, kSlots = kThreads / kLanes, kRows = kPageRows / kSlots;
    __shared__ __align__(16) float red[kSlots][D];
    __shared__ float wmax[kThreads / 32];
    const int tiles = max_tiles(a.max_new);
    const int h = (int)(item % a.Hkv);
    const bool is_v = (item / a.Hkv) & 1;
    const long long nt = item / (2 * a.Hkv);
    const int n = (int)(nt / tiles);
    const int l = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
    const SeqNew s = load_seq(a, n);
    if (s.bad) {
        if (threadIdx.x == 0) flag_status(a.status, kStatusBadData);
        return;
    }
    bf16* k_out = static_cast<bf16*>(a.k_out);
    if (s.count == 0 && a.cu_new == nullptr && k_out != nullptr && !is_v && slot == 0) {   // a padding entry
        store_row<D>(k_out + ((long long)n * a.Hkv + h) * D, l, Row{});
    }
    const PageTile t = page_tile(s, (int)(nt % tiles));
    if (t.hi <= t.lo) return;
    const int page = __ldg(a.page_table + (long long)n * a.max_pages + t.block);    // block < max_pages by kv_len's check
    const bool page_ok = page >= 0 && page < a.num_pages;
    if (!page_ok) {
        if (threadIdx.x == 0) flag_status(a.status, kStatusBadData);
        if (is_v || k_out == nullptr) return;
    }

    // the new rows, one for each of kRows steps of a slot
    const bf16* src = (is_v ? static_cast<const bf16*>(a.v) : static_cast<const bf16*>(a.k)) + h * D + 8 * l;
    const long long ld = is_v ? a.ld_v : a.ld_k;
    uint4 lo[kRows][1], hi[kRows][1];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = slot + i * kSlots;
        lo[i][0] = hi[i][0] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= t.lo && r < t.hi) {
            const bf16* p = src + (t.row + r - t.lo) * ld;
            lo[i][0] = ld_stream(p);
            hi[i][0] = ld_stream(p + D / 2);
        }
    }
    const bf16* weight = static_cast<const bf16*>(a.k_weight);
    Row w;
    if (!is_v) w = load_weight<bf16, D>(weight, l);
    Row x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        x[i].a = Raw8<bf16>::get(lo[i]);
        x[i].b = Raw8<bf16>::get(hi[i]);
        if (is_v) continue;
        const int r = slot + i * kSlots;
        const float rr = weight != nullptr ? row_rrms<D>(x[i], a.eps) : 1.f;
        if (r >= t.lo && r < t.hi) {
            x[i] = Turn(load_angles<bf16, D>(a.table, t.block * kPageRows + r, l), w)(x[i], rr);
            if (k_out != nullptr) store_row<D>(k_out + ((t.row + r - t.lo) * a.Hkv + h) * D, l, x[i]);
        }
    }
    if (!page_ok) return;
    const long long tile0 = ((long long)page * a.Hkv + h) * kPageRows;      // row of the cache
    const bool pool = a.kpool != nullptr && !is_v && t.hi == kPageRows;
    Row sum{};
    float unit = 1.f;               // what a pooled value is in

    if constexpr (kQ8) {
        uint8_t* cache = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + tile0 * D + 8 * l;
        float* scale = (is_v ? a.v_scale : a.k_scale) + (long long)page * a.Hkv + h;
        const float old = t.lo > 0 ? *scale : 0.f;
        float m = 0.f;              // rows that are not new are zero here
#pragma unroll
        for (int i = 0; i < kRows; ++i) m = finite_max(x[i].b, finite_max(x[i].a, m));
        m = warp_max(m);
        if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
        __syncthreads();            // (and every thread has read the old scale)
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, wmax[i]);
        if (t.lo > 0 && !scale_ok(old)) {       // the rows already there have no value
            if (threadIdx.x == 0) flag_status(a.status, kStatusBadData);
            return;
        }
        const bool keep = t.lo > 0 && m <= 448.f * old;
        const float sn = keep ? old : __int_as_float((scale_exp(__float_as_uint(m)) + 127) << 23);
        const float inv = 1.f / sn, ratio = old * inv;
        if (threadIdx.x == 0 && !keep) *scale = sn;
        unit = sn;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = slot + i * kSlots;
            if (r >= t.hi || (r < t.lo && keep && !pool)) continue;
            uint2* p = reinterpret_cast<uint2*>(cache + r * D);
            uint2* p2 = reinterpret_cast<uint2*>(cache + r * D + D / 2);
            uint2 c, c2;
            if (r >= t.lo) {
                *p = c = to_codes(x[i].a, inv);
                *p2 = c2 = to_codes(x[i].b, inv);
            } else {
                c = *p;
                c2 = *p2;
                if (!keep) {
                    *p = c = to_codes(from_codes(c), ratio);
                    *p2 = c2 = to_codes(from_codes(c2), ratio);
                }
            }
            if (pool) {
                add(sum.a, from_codes(c));
                add(sum.b, from_codes(c2));
            }
        }
    } else {
        bf16* cache = static_cast<bf16*>(is_v ? a.v_cache : a.k_cache) + tile0 * D;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = slot + i * kSlots;
            if (r >= t.lo && r < t.hi) store_row<D>(cache + r * D, l, x[i]);
            if (pool) {             // what this thread has stored, or an older row
                const bf16* p = cache + r * D + 8 * l;
                const uint4 u[1] = {*reinterpret_cast<const uint4*>(p)}, v[1] = {*reinterpret_cast<const uint4*>(p + D / 2)};
                add(sum.a, Raw8<bf16>::get(u));
                add(sum.b, Raw8<bf16>::get(v));
            }
        }
    }
    if (!pool) return;
    // the filled page's mean key: the slots' sums in slot order
    *reinterpret_cast<ulonglong2*>(&red[slot][8 * l]) = make_ulonglong2(sum.a.v[0], sum.a.v[1]);
    *reinterpret_cast<ulonglong2*>(&red[slot][8 * l + 4]) = make_ulonglong2(sum.a.v[2], sum.a.v[3]);
    *reinterpret_cast<ulonglong2*>(&red[slot][D / 2 + 8 * l]) = make_ulonglong2(sum.b.v[0], sum.b.v[1]);
    *reinterpret_cast<ulonglong2*>(&red[slot][D / 2 + 8 * l + 4]) = make_ulonglong2(sum.b.v[2], sum.b.v[3]);
    __syncthreads();
    if (threadIdx.x < D) {
        float m = 0.f;
        for (int i = 0; i < kSlots; ++i) m += red[i][threadIdx.x];
        a.kpool[((long long)page * a.Hkv + h) * D + threadIdx.x] = m * unit * (1.f / kPageRows);
    }
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a, long long q_ctas) {
    if (blockIdx.x < q_ctas)
        append_q<D>(a, blockIdx.x);
    else
        append_kv<D, kQ8>(a, blockIdx.x - q_ctas);
}

template <int D, bool kQ8>
cudaError_t go(const AppendArgs& a, cudaStream_t st) {
    constexpr int kSlots = kThreads / HeadRow<D>::kLanes;
    const long long q_ctas = a.q != nullptr ? (a.T * ((a.Hq + kHeads - 1) / kHeads) + kSlots - 1) / kSlots : 0;
    append_kernel<D, kQ8><<<(unsigned)(q_ctas + append_kv_ctas(a)), kThreads, 0, st>>>(a, q_ctas);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

long long append_kv_ctas(const AppendArgs& a) { return (long long)a.N * max_tiles(a.max_new) * a.Hkv * 2; }

cudaError_t launch_append(const AppendArgs& a, int D, cudaStream_t st) {
    if (a.k_scale != nullptr) return D == 128 ? go<128, true>(a, st) : go<64, true>(a, st);
    return D == 128 ? go<128, false>(a, st) : go<64, false>(a, st);
}

}  // namespace sas
