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
// Single tokens (max_new = 1) are bound by latency: a row slot (the D / 16 lanes of
// a row, head_row.cuh) takes one query head, a warp the new row of one (sequence, KV
// head) of K or of V. Prompts are bound by HBM. Into bf16 pages, persistent CTAs take
// units of four heads of one token of q, k or v, which share the token's angles.
// Into 8-bit pages a scale needs all new rows of a page: there the units of k and v
// are (sequence, block, KV head) tiles, so that new rows are read and written
// once, their amax needs no second pass and no two CTAs share a scale. Each
// thread prefetches its pieces of the next unit or tile with cp.async.
//
// Measured on one B200 (32/8 heads of 128): one token of one sequence 3.8 us (8.3
// with a CTA's 64-row tile for it), of 64 sequences into 8-bit pages 7.4 us, two
// of which fill a page, of 256 sequences 9.2 (22.5); prompts of 8k and 32k tokens
// into bf16 pages 43 and 147 us (74 and 86% of the copy rate; 45 and 170 with one
// CTA for each tile and four heads' loads in registers), 8k into 8-bit pages 43.8.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dependent.cuh"
#include "head_row.cuh"
#include "launch.h"
#include "page_rows.h"

namespace sas {
namespace {

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

// Position of token row t: -1 for a padding entry, whose rows are zero; -2 for rows
// of no sequence, or of one that is skipped, which stay as they are.
__device__ __forceinline__ int append_pos(const AppendArgs& a, long long t) {
    const int n = seq_of_row(a, t);
    if (n < 0) return -2;
    const SeqNew s = load_seq(a, n);
    return s.bad ? -2 : s.count > 0 ? s.first + (int)(t - s.row0) : -1;
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
// Largest magnitude of a row's values (NaN ignored) and m.
__device__ __forceinline__ float row_max(const Row& x, float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = f2_unpack(x.a.v[i]), g = f2_unpack(x.b.v[i]);
        m = sm100::max3(m, fabsf(f.x), fabsf(f.y));
        m = sm100::max3(m, fabsf(g.x), fabsf(g.y));
    }
    return m;
}
// An infinity has no code: it is kept as NaN.
__device__ __forceinline__ void drop_infinities(Half& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = f2_unpack(x.v[i]);
        if (fabsf(f.x) == INFINITY) f.x = __int_as_float(0x7fffffff);
        if (fabsf(f.y) == INFINITY) f.y = __int_as_float(0x7fffffff);
        x.v[i] = f2_pack(f.x, f.y);
    }
}

// A row slot's fp32 sums to a row of shared memory.
template <int D>
__device__ __forceinline__ void store_sum(float* p, int l, const Row& x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<ulonglong2*>(p + 8 * l + 4 * i) = make_ulonglong2(x.a.v[2 * i], x.a.v[2 * i + 1]);
        *reinterpret_cast<ulonglong2*>(p + D / 2 + 8 * l + 4 * i) = make_ulonglong2(x.b.v[2 * i], x.b.v[2 * i + 1]);
    }
}

// The scale of a page and head with new rows of magnitude up to m: the old one
// (`lo` rows are there already) where it holds them.
struct PageScale {
    bool ok, keep;
    float s;
};
__device__ __forceinline__ PageScale page_scale(int lo, float old, float m) {
    PageScale p;
    p.ok = lo == 0 || scale_ok(old);        // else the rows already there have no value
    p.keep = lo > 0 && m <= 448.f * old;
    p.s = p.keep ? old : __int_as_float((scale_exp(__float_as_uint(m)) + 127) << 23);
    return p;
}

// The mean key of a filled page is summed in one order by both kernels: the
// rows j, j + kSumRows, ... for each j, then these sums by j.
template <int D>
constexpr int kSumRows = D == 128 ? 16 : 32;

// The rare work on the rows of a page and head, by one warp: the codes of the
// first `grown` rows times `ratio`, and with `pool` the mean of the page's 64 keys
// (times their scale `unit`). Rows from `rows` on are not looked at. `red`: the
// warp's [kSumRows][D] floats.
template <int D, bool kQ8>
__device__ __forceinline__ void page_rows(const AppendArgs& a, bool is_v, int page, int h, int rows, int grown, float ratio,
                                          float unit, bool pool, float (*red)[D]) {
    constexpr int kLanes = HeadRow<D>::kLanes, kPerWarp = HeadRow<D>::kPerWarp;
    const int lane = threadIdx.x & 31, l = lane % kLanes, grp = lane / kLanes;
    const long long head = (long long)page * a.Hkv + h, tile0 = head * kPageRows;
#pragma unroll
    for (int k = 0; k < kSumRows<D> / kPerWarp; ++k) {
        Row sum{};
#pragma unroll
        for (int i = 0; i < kPageRows / kSumRows<D>; ++i) {
            const int r = grp + kPerWarp * k + kSumRows<D> * i;
            if (r >= rows) continue;
            if (kQ8) {
                uint8_t* row = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (tile0 + r) * D + 8 * l;
                uint2 c = *reinterpret_cast<const uint2*>(row), c2 = *reinterpret_cast<const uint2*>(row + D / 2);
                if (r < grown) {
                    *reinterpret_cast<uint2*>(row) = c = to_codes(from_codes(c), ratio);
                    *reinterpret_cast<uint2*>(row + D / 2) = c2 = to_codes(from_codes(c2), ratio);
                }
                if (pool) {
                    add(sum.a, from_codes(c));
                    add(sum.b, from_codes(c2));
                }
            } else {
                const bf16* row = static_cast<const bf16*>(a.k_cache) + (tile0 + r) * D + 8 * l;
                const uint4 c[1] = {*reinterpret_cast<const uint4*>(row)}, c2[1] = {*reinterpret_cast<const uint4*>(row + D / 2)};
                add(sum.a, Raw8<bf16>::get(c));
                add(sum.b, Raw8<bf16>::get(c2));
            }
        }
        if (pool) store_sum<D>(red[grp + kPerWarp * k], l, sum);
    }
    if (!pool) return;
    __syncwarp();
    for (int d = lane; d < D; d += 32) {
        float m = 0.f;
#pragma unroll 16
        for (int i = 0; i < kSumRows<D>; ++i) m += red[i][d];
        a.kpool[head * D + d] = m * unit * (1.f / kPageRows);
    }
}

// ------------------------------------------------------------------ single tokens
constexpr int kTokenThreads = 128;

template <int D>
__device__ __forceinline__ void token_q(const AppendArgs& a, uint32_t u) {
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    const uint32_t t = u / (uint32_t)a.Hq, h = u - t * a.Hq;
    const bool in = t < a.T;
    // the row's loads are on their way before the token's sequence is looked for
    const bf16* src = static_cast<const bf16*>(a.q) + (in ? t * a.ld_q + h * D : 0) + 8 * l;
    uint4 lo[1] = {make_uint4(0u, 0u, 0u, 0u)}, hi[1] = {lo[0]};
    if (in) lo[0] = ld_stream(src), hi[0] = ld_stream(src + D / 2);
    const bf16* weight = static_cast<const bf16*>(a.q_weight);
    const Row w = load_weight<bf16, D>(weight, l);
    const int pos = in ? append_pos(a, t) : -2;
    const Turn turn(load_angles<bf16, D>(a.table, max(pos, 0), l), w);
    const Row x = {Raw8<bf16>::get(lo), Raw8<bf16>::get(hi)};
    Row y = turn(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);
    if (pos < 0) y = Row{};
    if (pos > -2) store_row<D>(static_cast<bf16*>(a.q_out) + (long long)u * D, l, y);
}

// The new row of one (sequence, KV head) of K or of V, by one warp: its first
// D / 16 lanes hold the row, the whole warp does the rare work on the page's
// older rows. `red`: the warp's [kSumRows][D] floats.
template <int D, bool kQ8>
__device__ __forceinline__ void token_kv(const AppendArgs& a, uint32_t u, float (*red)[D]) {
    constexpr int kLanes = HeadRow<D>::kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes, grp = lane / kLanes;
    if (u >= 2u * a.N * a.Hkv) return;
    const uint32_t n = u / (2u * a.Hkv), rest = u - n * 2u * a.Hkv;
    const bool is_v = rest >= (uint32_t)a.Hkv;
    const int h = (int)(is_v ? rest - a.Hkv : rest);
    const SeqNew s = load_seq(a, (int)n);
    bf16* k_out = is_v ? nullptr : static_cast<bf16*>(a.k_out);
    if (s.bad) {
        if (lane == 0) flag_status(a.status, kStatusBadData);
        return;
    }
    if (s.count == 0) {
        if (a.cu_new == nullptr && k_out != nullptr && grp == 0)       // a padding entry
            store_row<D>(k_out + ((long long)n * a.Hkv + h) * D, l, Row{});
        return;
    }
    const PageTile t = page_tile(s, 0);             // the one new row is t.lo
    const int page = __ldg(a.page_table + (long long)n * a.max_pages + t.block);   // block < max_pages by kv_len's check
    const bf16* src = (is_v ? static_cast<const bf16*>(a.v) + t.row * a.ld_v : static_cast<const bf16*>(a.k) + t.row * a.ld_k) +
                      h * D + 8 * l;
    const uint4 lo[1] = {ld_stream(src)}, hi[1] = {ld_stream(src + D / 2)};
    const bf16* weight = static_cast<const bf16*>(a.k_weight);
    const Row w = load_weight<bf16, D>(weight, l);
    const Angles ang = load_angles<bf16, D>(a.table, s.first, l);
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && lane == 0) flag_status(a.status, kStatusBadData);
    const long long tile0 = ok ? ((long long)page * a.Hkv + h) * kPageRows : 0;     // row of the cache
    float* scale = kQ8 ? (is_v ? a.v_scale : a.k_scale) + (ok ? (long long)page * a.Hkv + h : 0) : nullptr;
    const float old = kQ8 && ok && t.lo > 0 ? *scale : 0.f;

    Row x = {Raw8<bf16>::get(lo), Raw8<bf16>::get(hi)};
    if (!is_v) {
        // the products in the order of the prompts' kernels: both store the same bits
        const float r = weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f;
        x = kQ8 ? norm_turn(x, w, r, ang) : Turn(ang, w)(x, r);
        if (k_out != nullptr && grp == 0) store_row<D>(k_out + (t.row * a.Hkv + h) * D, l, x);
    }
    if (!ok) return;

    PageScale ps{true, true, 1.f};
    if constexpr (kQ8) {
        float m = warp_max(row_max(x, 0.f));        // (behind the shuffles every lane has read the old scale)
        if (m == INFINITY) {
            drop_infinities(x.a);
            drop_infinities(x.b);
            m = warp_max(row_max(x, 0.f));
        }
        ps = page_scale(t.lo, old, m);
        if (!ps.ok) {
            if (lane == 0) flag_status(a.status, kStatusBadData);
            return;
        }
        if (grp == 0) {
            uint8_t* row = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (tile0 + t.lo) * D;
            *reinterpret_cast<uint2*>(row + 8 * l) = to_codes(x.a, 1.f / ps.s);
            *reinterpret_cast<uint2*>(row + D / 2 + 8 * l) = to_codes(x.b, 1.f / ps.s);
        }
        if (lane == 0 && !ps.keep) *scale = ps.s;
    } else if (grp == 0) {
        store_row<D>(static_cast<bf16*>(is_v ? a.v_cache : a.k_cache) + (tile0 + t.lo) * D, l, x);
    }

    const bool grown = kQ8 && t.lo > 0 && !ps.keep, pool = !is_v && a.kpool != nullptr && t.lo == kPageRows - 1;
    if (!grown && !pool) return;
    __syncwarp();                                   // the new row is written
    page_rows<D, kQ8>(a, is_v, page, h, t.lo + pool, grown ? t.lo : 0, old * (1.f / ps.s), ps.s, pool, red);
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kTokenThreads) append_token_kernel(const AppendArgs a, uint32_t q_ctas) {
    constexpr int kSlots = kTokenThreads / HeadRow<D>::kLanes, kCtaWarps = kTokenThreads / 32;
    __shared__ __align__(16) float red[kCtaWarps][kSumRows<D>][D];
    after_previous();
    if (blockIdx.x < q_ctas)
        token_q<D>(a, blockIdx.x * kSlots + threadIdx.x / HeadRow<D>::kLanes);
    else
        token_kv<D, kQ8>(a, (blockIdx.x - q_ctas) * kCtaWarps + threadIdx.x / 32, red[threadIdx.x / 32]);
}

// ------------------------------------------------------------------ prompts into 8-bit pages
constexpr int kThreads = 128;
constexpr int kHeads = 4;                   // query heads of a unit
constexpr int kCtas = 4;                    // resident CTAs of an SM
constexpr int kStages = 2;                  // pieces of work in flight
constexpr int kStageBytes = 2 * kHeads * kThreads * 16;    // a thread's pieces of a unit, or of its rows of a tile

// A piece of work of a CTA: a (sequence, block, KV head) tile of K or of V with new
// rows, or a query unit for each of its row slots, in few registers: one waits while
// the other is worked on.
struct Work {
    enum : uint32_t { kNone, kUnit, kK, kV };
    uint32_t kind;          // bits 0-1; of a tile: rows lo (bits 8-15) to hi (bits 16-23)
    int at;                 // a unit: its number; a tile: the token row of its first new row
    int pos;                // a unit: its position (append_pos); a tile: its block
    int h, page;            // a tile's KV head and page
    __device__ __forceinline__ bool is(uint32_t k) const { return (kind & 3) == k; }
    __device__ __forceinline__ bool tile() const { return kind & 2; }
    __device__ __forceinline__ int lo() const { return kind >> 8 & 255; }
    __device__ __forceinline__ int hi() const { return kind >> 16; }
};
// The sequence that a thread's last piece of work belonged to. The next one mostly
// belongs to it too, and then no load stands in front of its copies.
struct SeqAt {
    int n = -1;                 // -1: none yet
    int row0 = 0, count = 0, first = 0;
    uint32_t tile0 = 0, tile1 = 0;      // its tile indices (seq_tile_base)
    bool bad = false;
    __device__ __forceinline__ void load(const AppendArgs& a, int at) {
        const SeqNew s = load_seq(a, at);
        n = at;
        row0 = (int)s.row0;
        count = s.count;
        first = s.first;
        bad = s.bad;
        tile0 = seq_tile_base(__ldg(a.cu_new + at), at);
        tile1 = seq_tile_base(__ldg(a.cu_new + at + 1), at + 1);
    }
    __device__ __forceinline__ bool holds(int t) const { return n >= 0 && !bad && t >= row0 && t - row0 < count; }
    // Goes to the sequence of token row t; false for a row of none, or of one that is skipped.
    __device__ __forceinline__ bool find(const AppendArgs& a, int t) {
        if (holds(t)) return true;
        int at = seq_of_row(a, t);
        if (at < 0) return false;
        load(a, at);
        // a sequence that is skipped may overlap another, where cu_new decreases
        for (at = 0; bad && at < a.N; ++at) {
            load(a, at);
            bad = !holds(t);
        }
        return holds(t);
    }
};
__device__ __forceinline__ Work kv_work(const AppendArgs& a, SeqAt& s, uint32_t v, uint32_t rest) {
    Work k{};
    const bool is_v = rest >= (uint32_t)a.Hkv;
    if (s.n < 0 || v < s.tile0 || v >= s.tile1) {       // the last n with its tile base <= v
        int lo = 0, hi = a.N;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seq_tile_base(__ldg(a.cu_new + mid), mid) <= v) lo = mid; else hi = mid;
        }
        s.load(a, lo);
    }
    if (s.bad || v < s.tile0 || v - s.tile0 >= (uint32_t)max_tiles(a.max_new)) return k;
    const PageTile t = page_tile(SeqNew{s.row0, s.first, s.count, false}, (int)(v - s.tile0));
    if (t.hi <= t.lo) return k;
    k.kind = (is_v ? Work::kV : Work::kK) | (uint32_t)t.lo << 8 | (uint32_t)t.hi << 16;
    k.at = (int)t.row;
    k.pos = t.block;
    k.h = (int)(is_v ? rest - a.Hkv : rest);
    k.page = __ldg(a.page_table + (long long)s.n * a.max_pages + t.block);     // block < max_pages by kv_len's check
    return k;
}
template <int D>
__device__ __forceinline__ Work q_work(const AppendArgs& a, SeqAt& s, uint32_t batch, uint32_t q_units) {
    Work k{};
    k.kind = Work::kUnit;
    k.pos = -2;
    const uint32_t u = batch * (kThreads / HeadRow<D>::kLanes) + threadIdx.x / HeadRow<D>::kLanes;
    if (u < q_units) {
        const int t = (int)(u / parts_of(a.Hq, kHeads));
        k.at = (int)u;
        if (s.find(a, t)) k.pos = s.first + (t - s.row0);
    }
    return k;
}

// Flags every sequence that breaks the call's terms, also those that no token row
// or tile index leads to (by the first CTA).
__device__ __forceinline__ void flag_sequences(const AppendArgs& a) {
    if (blockIdx.x != 0) return;
    for (int n = threadIdx.x; n < a.N; n += kThreads)
        if (load_seq(a, n).bad || __ldg(a.cu_new + n + 1) < __ldg(a.cu_new + n)) flag_status(a.status, kStatusBadData);
}

// Starts the copies of a piece of work into a stage.
template <int D>
__device__ __forceinline__ void issue(const AppendArgs& a, const Work& k, uint32_t at) {
    constexpr int kLanes = HeadRow<D>::kLanes, kSlots = kThreads / kLanes, kRows = kPageRows / kSlots;
    const int l = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
    if (k.tile()) {
        const bool is_v = k.is(Work::kV);
        const bf16* src = (is_v ? static_cast<const bf16*>(a.v) : static_cast<const bf16*>(a.k)) + k.h * D;
        const long long ld = is_v ? a.ld_v : a.ld_k;
        const int lo = k.lo(), hi = k.hi();
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = slot + i * kSlots;        // rows that are not new: zeroes, copied from nowhere
            copy_row<bf16, D, kThreads>(at + 2 * i * kThreads * 16, src + (k.at + min(max(r, lo), hi - 1) - lo) * ld, l,
                                        r >= lo && r < hi);
        }
    } else if (k.is(Work::kUnit) && k.pos > -2) {
        const uint32_t parts = parts_of(a.Hq, kHeads), t = k.at / parts;
        const bf16* src = static_cast<const bf16*>(a.q) + (long long)t * a.ld_q;
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = (int)(k.at - t * parts + i * parts);
            copy_row<bf16, D, kThreads>(at + 2 * i * kThreads * 16, src + (h < a.Hq ? h : 0) * D, l, h < a.Hq);
        }
    }
    copy_commit();
}

template <int D>
__device__ __forceinline__ void store_unit(const AppendArgs& a, const Work& k, uint32_t at) {
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    const bf16* weight = static_cast<const bf16*>(a.q_weight);
    const uint32_t parts = parts_of(a.Hq, kHeads), t = k.at / parts;
    const Turn turn(load_angles<bf16, D>(a.table, max(k.pos, 0), l), load_weight<bf16, D>(weight, l));
    bf16* dst = static_cast<bf16*>(a.q_out) + (long long)t * a.Hq * D;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = (int)(k.at - t * parts + i * parts);
        const Row x = read_row<bf16, kThreads>(at + 2 * i * kThreads * 16);
        Row y = turn(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);
        if (k.pos < 0) y = Row{};
        if (k.pos > -2 && h < a.Hq) store_row<D>(dst + h * D, l, y);
    }
}

// `stage`: the CTA's whole stage of this tile, `at` this thread's pieces of it.
template <int D>
__device__ __forceinline__ void store_tile(const AppendArgs& a, const Work& k, uint32_t at, uint8_t* stage, float* wmax) {
    constexpr int kLanes = HeadRow<D>::kLanes, kSlots = kThreads / kLanes, kRows = kPageRows / kSlots;
    const int l = threadIdx.x % kLanes, slot = threadIdx.x / kLanes, lo = k.lo(), hi = k.hi();
    const bool is_v = k.is(Work::kV), page_ok = k.page >= 0 && k.page < a.num_pages;
    bf16* k_out = is_v ? nullptr : static_cast<bf16*>(a.k_out);
    if (!page_ok) {
        if (threadIdx.x == 0) flag_status(a.status, kStatusBadData);
        if (k_out == nullptr) return;
    }
    const long long tile0 = page_ok ? ((long long)k.page * a.Hkv + k.h) * kPageRows : 0;      // row of the cache
    float* scale = (is_v ? a.v_scale : a.k_scale) + (page_ok ? (long long)k.page * a.Hkv + k.h : 0);
    const float old = page_ok && lo > 0 ? *scale : 0.f;
    const bf16* weight = static_cast<const bf16*>(a.k_weight);
    Row x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = slot + i * kSlots;
        x[i] = read_row<bf16, kThreads>(at + 2 * i * kThreads * 16);
        if (is_v) continue;
        const float rr = weight != nullptr ? row_rrms<D>(x[i], a.eps) : 1.f;
        x[i] = norm_turn(x[i], load_weight<bf16, D>(weight, l), rr,
                         load_angles<bf16, D>(a.table, k.pos * kPageRows + min(max(r, lo), hi - 1), l));
        if (r < lo || r >= hi)
            x[i] = Row{};               // not a new row: nothing of it counts
        else if (k_out != nullptr)
            store_row<D>(k_out + ((long long)(k.at + r - lo) * a.Hkv + k.h) * D, l, x[i]);
    }
    if (!page_ok) return;
    const bool pool = a.kpool != nullptr && !is_v && hi == kPageRows;
    Row sum{};
    uint8_t* cache = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + tile0 * D + 8 * l;
    auto tile_max = [&] {
        float m = 0.f;              // rows that are not new are zero here
#pragma unroll
        for (int i = 0; i < kRows; ++i) m = row_max(x[i], m);
        m = warp_max(m);
        __syncthreads();            // the last maxima have been read
        if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
        __syncthreads();            // (and every thread has read the old scale)
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, wmax[i]);
        return m;
    };
    float m = tile_max();
    if (m == INFINITY) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            drop_infinities(x[i].a);
            drop_infinities(x[i].b);
        }
        m = tile_max();
    }
    const PageScale ps = page_scale(lo, old, m);
    if (!ps.ok) {
        if (threadIdx.x == 0) flag_status(a.status, kStatusBadData);
        return;
    }
    const float inv = 1.f / ps.s, ratio = old * inv;
    if (threadIdx.x == 0 && !ps.keep) *scale = ps.s;
    #pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = slot + i * kSlots;
        if (r >= hi || (r < lo && ps.keep && !pool)) continue;
        uint2* p = reinterpret_cast<uint2*>(cache + r * D);
        uint2* p2 = reinterpret_cast<uint2*>(cache + r * D + D / 2);
        uint2 c, c2;
        if (r >= lo) {
            *p = c = to_codes(x[i].a, inv);
            *p2 = c2 = to_codes(x[i].b, inv);
        } else {
            c = *p;
            c2 = *p2;
            if (!ps.keep) {
                *p = c = to_codes(from_codes(c), ratio);
                *p2 = c2 = to_codes(from_codes(c2), ratio);
            }
        }
        if (pool) {
            add(sum.a, from_codes(c));
            add(sum.b, from_codes(c2));
        }
    }
    if (!pool) return;
    // the filled page's mean key: the slots' sums in slot order, where the rows were
    static_assert(kSlots == kSumRows<D> && kSlots * D * 4 <= kStageBytes, "sums of a tile");
    float(*red)[D] = reinterpret_cast<float(*)[D]>(stage);
    __syncthreads();                // every thread has its rows
    store_sum<D>(red[slot], l, sum);
    __syncthreads();
    if (threadIdx.x < D) {
        float m = 0.f;
#pragma unroll 16
        for (int i = 0; i < kSlots; ++i) m += red[i][threadIdx.x];
        a.kpool[((long long)k.page * a.Hkv + k.h) * D + threadIdx.x] = m * ps.s * (1.f / kPageRows);
    }
    __syncthreads();                // read before the stage's next copies
}

// A CTA's share: batches of query units (kSlots units each) and tiles, contiguous
// runs of both (neighbouring tiles are the heads of one block, whose table rows
// are then L1 hits; every gridDim-th tile instead takes 2 to 10% longer). It starts with a
// batch of units, whose copies wait for no lookup.
template <int D>
__global__ void __launch_bounds__(kThreads, kCtas)
append_tiles_kernel(const AppendArgs a, uint32_t q_units, uint32_t batches, uint32_t items) {
    constexpr int kSlots = kThreads / HeadRow<D>::kLanes;
    __shared__ __align__(16) uint8_t ring_s[kStages * kStageBytes];
    __shared__ float wmax[kThreads / 32];
    after_previous();
    const uint32_t ring = sm100::smem_u32(ring_s) + threadIdx.x * 16;
    // both kinds in proportion, their sum to within one: where a CTA has a batch at least, all shares are >= 0
    const uint32_t c = blockIdx.x;
    auto share = [&](unsigned long long n, uint32_t c) { return (uint32_t)(n * c / gridDim.x); };
    const unsigned long long all = (unsigned long long)batches + items;
    uint32_t kv0 = share(items, c), kv1 = share(items, c + 1), q0 = share(all, c) - kv0, q1 = share(all, c + 1) - kv1;
    if (batches < gridDim.x) {          // few batches: one list, the batches first
        const uint32_t b0 = share(all, c), b1 = share(all, c + 1);
        q0 = min(b0, batches), q1 = min(b1, batches);
        kv0 = max(b0, batches) - batches, kv1 = max(b1, batches) - batches;
    }
    const uint32_t lead = q1 > q0 ? 1 : 0, tiles = kv1 - kv0, count = q1 - q0 + tiles;
    static_assert(kStages == 2, "one piece of work waits");
    SeqAt seq;
    uint32_t v = kv0 / (2u * a.Hkv), rest = kv0 - v * 2u * a.Hkv;       // the next tile: its index, and head of K or of V
    auto work_at = [&](uint32_t j) {
        if (j >= lead && j < lead + tiles) {
            const Work k = kv_work(a, seq, v, rest);
            if (++rest == 2u * a.Hkv) rest = 0, ++v;
            return k;
        }
        return q_work<D>(a, seq, q0 + (j < lead ? j : j - tiles), j < count ? q_units : 0);
    };
    Work cur = work_at(0);
    issue<D>(a, cur, ring);
    uint32_t st = 0;
    for (uint32_t j = 0; j < count; ++j) {
        const Work next = work_at(j + 1);
        issue<D>(a, next, ring + (st ^ 1) * kStageBytes);
        copy_wait<kStages - 1>();
        if (cur.tile())
            store_tile<D>(a, cur, ring + st * kStageBytes, ring_s + st * kStageBytes, wmax);
        else if (cur.is(Work::kUnit))
            store_unit<D>(a, cur, ring + st * kStageBytes);
        cur = next;
        st ^= 1;
    }
    copy_wait<0>();
    flag_sequences(a);
}

// ------------------------------------------------------------------ prompts into bf16 pages
// Units of four heads of one token: queries, keys, and values, which are copied as they are.
template <int D>
__global__ void __launch_bounds__(kThreads, kCtas) append_rows_kernel(const AppendArgs a, uint32_t q_parts, uint32_t units) {
    constexpr int kSlots = kThreads / HeadRow<D>::kLanes, kRow = 2 * kThreads * 16;
    __shared__ __align__(16) uint8_t ring_s[kStages * kStageBytes];
    after_previous();
    const uint32_t ring = sm100::smem_u32(ring_s) + threadIdx.x * 16;
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    const uint32_t kv_parts = parts_of(a.Hkv, kHeads), per = q_parts + 2 * kv_parts;
    const uint32_t first = blockIdx.x * kSlots + threadIdx.x / HeadRow<D>::kLanes, step = gridDim.x * kSlots;

    enum { kNone, kQ, kK, kV };
    struct Unit {
        int kind, t, part, pos, page;
    };
    SeqAt seq;
    auto unit_at = [&](uint32_t u) {
        Unit r{kNone, 0, 0, 0, 0};
        if (u >= units) return r;
        const uint32_t t = u / per, j = u - t * per;
        if (!seq.find(a, (int)t)) return r;             // a row of no sequence, or of one that is skipped
        r.t = (int)t;
        r.pos = seq.first + (int)t - seq.row0;
        r.kind = j < q_parts ? kQ : j < q_parts + kv_parts ? kK : kV;
        r.part = (int)(j < q_parts ? j : j < q_parts + kv_parts ? j - q_parts : j - q_parts - kv_parts);
        if (r.kind != kQ) r.page = __ldg(a.page_table + (long long)seq.n * a.max_pages + r.pos / kPageRows);    // in range by kv_len's check
        return r;
    };
    auto issue = [&](const Unit& r, uint32_t at) {
        if (r.kind != kNone) {
            const bf16* src = r.kind == kQ   ? static_cast<const bf16*>(a.q) + r.t * a.ld_q
                              : r.kind == kK ? static_cast<const bf16*>(a.k) + r.t * a.ld_k
                                             : static_cast<const bf16*>(a.v) + r.t * a.ld_v;
            const int H = r.kind == kQ ? a.Hq : a.Hkv, parts = (int)(r.kind == kQ ? q_parts : kv_parts);
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int h = r.part + i * parts;
                copy_row<bf16, D, kThreads>(at + i * kRow, src + (h < H ? h : 0) * D, l, h < H);
            }
        }
        copy_commit();
    };

    Unit cur = unit_at(first);
    issue(cur, ring);
    uint32_t st = 0;
    for (uint32_t base = blockIdx.x * kSlots, u = first; base < units; base += step, u += step) {
        const Unit next = unit_at(u + step);
        issue(next, ring + (st ^ 1) * kStageBytes);
        const bool is_q = cur.kind == kQ, is_v = cur.kind == kV;
        const bf16* weight = static_cast<const bf16*>(is_q ? a.q_weight : a.k_weight);
        const Turn turn(load_angles<bf16, D>(a.table, cur.pos, l), load_weight<bf16, D>(weight, l));
        const int H = is_q ? a.Hq : a.Hkv, parts = (int)(is_q ? q_parts : kv_parts);
        const bool page_ok = cur.page >= 0 && cur.page < a.num_pages, live = cur.kind != kNone;
        if (live && !page_ok && l == 0) flag_status(a.status, kStatusBadData);
        // queries go to their row of q_out, keys and values to row pos % 64 of the page's tile of their head
        bf16* dst = is_q ? static_cast<bf16*>(a.q_out) + (long long)cur.t * a.Hq * D
                         : static_cast<bf16*>(is_v ? a.v_cache : a.k_cache) +
                               ((long long)(page_ok ? cur.page : 0) * a.Hkv * kPageRows + cur.pos % kPageRows) * D;
        const int stride = is_q ? D : kPageRows * D;
        bf16* k_out = cur.kind == kK ? static_cast<bf16*>(a.k_out) : nullptr;
        copy_wait<kStages - 1>();
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = cur.part + i * parts;
            const uint32_t at = ring + st * kStageBytes + i * kRow;
            const Row x = read_row<bf16, kThreads>(at);
            const Row y = turn(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);
            if (!live || h >= H) continue;
            if (k_out != nullptr) store_row<D>(k_out + ((long long)cur.t * a.Hkv + h) * D, l, y);
            if (!page_ok) continue;
            bf16* p = dst + (long long)h * stride;
            if (is_v) {
                *reinterpret_cast<uint4*>(p + 8 * l) = ld_shared16(at);
                *reinterpret_cast<uint4*>(p + D / 2 + 8 * l) = ld_shared16(at + kThreads * 16);
            } else {
                store_row<D>(p, l, y);
            }
        }
        cur = next;
        st ^= 1;
    }
    copy_wait<0>();
    flag_sequences(a);
}

// The mean key of every page that the call has filled: a warp for each (block, KV head).
template <int D>
__global__ void __launch_bounds__(kThreads) pool_filled_kernel(const AppendArgs a, uint32_t items) {
    constexpr int kCtaWarps = kThreads / 32;
    __shared__ __align__(16) float red[kCtaWarps][kSumRows<D>][D];
    after_previous();
    const uint32_t it = blockIdx.x * kCtaWarps + threadIdx.x / 32;
    if (it >= items) return;
    SeqAt seq;
    const Work k = kv_work(a, seq, it / a.Hkv, it % a.Hkv);
    if (!k.is(Work::kK) || k.hi() != kPageRows || k.page < 0 || k.page >= a.num_pages) return;
    page_rows<D, false>(a, false, k.page, k.h, kPageRows, 0, 1.f, 1.f, true, red[threadIdx.x / 32]);
}

template <int D, bool kQ8>
cudaError_t go(const AppendArgs& a, cudaStream_t st) {
    constexpr long long kSlots = kThreads / HeadRow<D>::kLanes;
    const long long items = append_items(a);
    cudaError_t e;
    if (a.max_new == 1) {
        constexpr long long kTokenSlots = kTokenThreads / HeadRow<D>::kLanes, kCtaWarps = kTokenThreads / 32;
        const long long q_ctas = a.q != nullptr ? (a.T * a.Hq + kTokenSlots - 1) / kTokenSlots : 0;
        e = launch_dependent(append_token_kernel<D, kQ8>, dim3((unsigned)(q_ctas + (items + kCtaWarps - 1) / kCtaWarps)),
                             kTokenThreads, 0, st, a, (uint32_t)q_ctas);
        if (e == cudaSuccess) count_launches(1);
        return e;
    }
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    const long long q_parts = a.q != nullptr ? parts_of(a.Hq, kHeads) : 0, most = (long long)kCtas * sms;
    if constexpr (kQ8) {
        const long long q_units = a.T * q_parts, batches = (q_units + kSlots - 1) / kSlots;
        e = launch_dependent(append_tiles_kernel<D>, dim3((unsigned)std::min(batches + items, most)), kThreads, 0, st, a,
                             (uint32_t)q_units, (uint32_t)batches, (uint32_t)items);
    } else {
        const long long units = a.T * (q_parts + 2 * parts_of(a.Hkv, kHeads));
        e = launch_dependent(append_rows_kernel<D>, dim3((unsigned)std::min((units + kSlots - 1) / kSlots, most)), kThreads, 0,
                             st, a, (uint32_t)q_parts, (uint32_t)units);
        if (e == cudaSuccess && a.kpool != nullptr) {
            count_launches(1);
            constexpr int kCtaWarps = kThreads / 32;
            const long long heads = items / 2;
            e = launch_dependent(pool_filled_kernel<D>, dim3((unsigned)((heads + kCtaWarps - 1) / kCtaWarps)), kThreads, 0, st, a,
                                 (uint32_t)heads);
        }
    }
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

long long append_items(const AppendArgs& a) {
    return (a.max_new == 1 ? (long long)a.N : (long long)seq_tile_base((int)a.T, a.N) + 1) * a.Hkv * 2;
}

cudaError_t launch_append(const AppendArgs& a, int D, cudaStream_t st) {
    if (a.k_scale != nullptr) return D == 128 ? go<128, true>(a, st) : go<64, true>(a, st);
    return D == 128 ? go<128, false>(a, st) : go<64, false>(a, st);
}

}  // namespace sas
