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

template <int D>
__device__ __forceinline__ void append_q(const AppendArgs& a, long long cta) {
    constexpr int kSlots = kThreads / HeadRow<D>::kLanes;
    const int l = threadIdx.x % HeadRow<D>::kLanes, parts = unit_parts(a.Hq);
    const long long u = cta * kSlots + threadIdx.x / HeadRow<D>::kLanes;
    const long long t = u / parts;
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
    norm_rope_unit<bf16, D>(static_cast<const bf16*>(a.q) + (live ? t * a.ld_q : 0),
                            static_cast<bf16*>(a.q_out) + t * a.Hq * D, a.Hq, (int)(u % parts),
                            static_cast<const bf16*>(a.q_weight), a.table, a.eps, l, live, [&] { return pos; });
}

// Eight e4m3 codes (8 bytes) from eight values, and back.
__device__ __forceinline__ uint2 to_codes(const float* x, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void from_codes(uint2 c, float* x) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <int D, bool kQ8>
__device__ __forceinline__ void append_kv(const AppendArgs& a, long long item) {
    constexpr int kLanes = HeadRow<D>::kLanes, kSlots = kThreads / kLanes, kRows = kPageRows / kSlots;
    __shared__ float red[kSlots][D];
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
        const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        store8(k_out + ((long long)n * a.Hkv + h) * D + 8 * l, zero);
        store8(k_out + ((long long)n * a.Hkv + h) * D + D / 2 + 8 * l, zero);
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
    const bf16* src = is_v ? static_cast<const bf16*>(a.v) + h * D : static_cast<const bf16*>(a.k) + h * D;
    const long long ld = is_v ? a.ld_v : a.ld_k;
    Raw8<bf16> lo[kRows], hi[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = slot + i * kSlots;
        lo[i].zero();
        hi[i].zero();
        if (r >= t.lo && r < t.hi) {
            const bf16* p = src + (t.row + r - t.lo) * ld + 8 * l;
            lo[i].load(p);
            hi[i].load(p + D / 2);
        }
    }
    float x[kRows][16];
    const bf16* weight = static_cast<const bf16*>(a.k_weight);
    float w[16];
    if (!is_v && weight != nullptr) load_weight<bf16, D>(weight, l, w);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        lo[i].get(x[i]);
        hi[i].get(x[i] + 8);
        if (is_v) continue;
        const int r = slot + i * kSlots;
        if (weight != nullptr) {
            const float rr = row_rrms<D>(x[i], a.eps);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[i][e] = x[i][e] * rr * w[e];
        }
        if (r >= t.lo && r < t.hi) {
            Angles ang;
            ang.load<D>(a.table, t.block * kPageRows + r, l);
            ang.turn(x[i]);
            if (k_out != nullptr) {
                bf16* p = k_out + ((t.row + r - t.lo) * a.Hkv + h) * D + 8 * l;
                store8(p, x[i]);
                store8(p + D / 2, x[i] + 8);
            }
        }
    }
    if (!page_ok) return;
    const long long tile0 = ((long long)page * a.Hkv + h) * kPageRows;      // row of the cache
    const bool pool = a.kpool != nullptr && !is_v && t.hi == kPageRows;
    float sum[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] = 0.f;
    float unit = 1.f;               // what a pooled value is in

    if constexpr (kQ8) {
        uint8_t* cache = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + tile0 * D;
        float* scale = (is_v ? a.v_scale : a.k_scale) + (long long)page * a.Hkv + h;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                // an infinity has no code: it is kept as NaN, and no scale follows it
                if (!(fabsf(x[i][e]) <= 3.402823466e38f)) x[i][e] = __int_as_float(0x7fffffff);
                const int r = slot + i * kSlots;
                if (r >= t.lo && r < t.hi) m = fmaxf(m, fabsf(x[i][e]));
            }
        m = warp_max(m);
        if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
        const float old = t.lo > 0 ? *scale : 0.f;
        __syncthreads();
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
            if (r >= t.hi) continue;
            uint2* p = reinterpret_cast<uint2*>(cache + r * D + 8 * l);
            uint2* p2 = reinterpret_cast<uint2*>(cache + r * D + D / 2 + 8 * l);
            uint2 c, c2;
            if (r >= t.lo) {
                c = to_codes(x[i], inv);
                c2 = to_codes(x[i] + 8, inv);
                *p = c;
                *p2 = c2;
            } else {
                if (keep && !pool) continue;
                c = *p;
                c2 = *p2;
                if (!keep) {
                    float y[16];
                    from_codes(c, y);
                    from_codes(c2, y + 8);
                    c = to_codes(y, ratio);
                    c2 = to_codes(y + 8, ratio);
                    *p = c;
                    *p2 = c2;
                }
            }
            if (pool) {
                float y[16];
                from_codes(c, y);
                from_codes(c2, y + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[e] += y[e];
            }
        }
    } else {
        bf16* cache = static_cast<bf16*>(is_v ? a.v_cache : a.k_cache) + tile0 * D;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = slot + i * kSlots;
            bf16* p = cache + r * D + 8 * l;
            if (r >= t.lo && r < t.hi) {
                store8(p, x[i]);
                store8(p + D / 2, x[i] + 8);
            }
            if (pool) {
                float y[16];
                if (r < t.lo) {
                    Raw8<bf16> u, v;
                    u.w = *reinterpret_cast<const uint4*>(p);
                    v.w = *reinterpret_cast<const uint4*>(p + D / 2);
                    u.get(y);
                    v.get(y + 8);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = __bfloat162float(__float2bfloat16_rn(x[i][e]));
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[e] += y[e];
            }
        }
    }
    if (!pool) return;
    // the filled page's mean key: the slots' sums in slot order
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        red[slot][8 * l + e] = sum[e];
        red[slot][D / 2 + 8 * l + e] = sum[e + 8];
    }
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
    const long long q_ctas = a.q != nullptr ? (a.T * unit_parts(a.Hq) + kSlots - 1) / kSlots : 0;
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
