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
// of one (sequence, block, two heads of k or four of v) go to one CTA, so that new rows
// are read and written once, their amax needs no second pass and no two CTAs share a scale.
// Each thread prefetches its pieces of the next unit with cp.async.
//
// Measured on one B200 (32/8 heads of 128): one token of one sequence 3.4 us, of 64
// sequences into 8-bit pages 4.0, two of which fill a page, of 256 sequences 5.8
// (22.5 with a CTA for each row; 6.9 and 8.8 where the filled pages' rows met in
// shared memory instead of by shuffles, without their loads in flight together);
// prompts of 8k and 32k tokens into bf16 pages 36.7 and 127.5 us (87 and 100% of the
// copy rate; as 64-row tiles of one head 42.5 and 147; 42 and 142 with the pages'
// mean keys), into 8-bit pages 40.2 and 144 (73 and 81%; 44.5 and 160 with mean keys):
// the blocks' barrier leaves the latencies of one CTA's 16 warps in a row. (Reading the
// rows twice instead of holding them in registers, for two or three CTAs an SM: 46.8
// and 75 us at 8k.)
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "dependent.cuh"
#include "head_row.cuh"
#include "launch.h"
#include "page_rows.h"

namespace sas {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ SeqNew load_seq(const AppendArgs& a, int n) {
    const bool cu = a.cu_new != nullptr;
    return seq_new(cu, cu ? a.cu_new[n] : 0, cu ? a.cu_new[n + 1] : 0, n, a.T, a.max_new,
                   a.kv_len[n], a.max_pages, a.max_pos);
}

// Sequence that owns token row t, or -1.
__device__ __forceinline__ int seq_of_row(const AppendArgs& a, long long t) {
    if (a.cu_new == nullptr) return (int)t;
    int lo = 0, hi = a.N;                        // the last n with cu[n] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_new[mid] <= t) lo = mid; else hi = mid;
    }
    return a.cu_new[lo] <= t && t < a.cu_new[lo + 1] ? lo : -1;
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
// Largest of the warp's magnitudes: without a sign the bits order like the values.
__device__ __forceinline__ float warp_max_abs(float m) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
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

// The mean key of a filled page is summed in one order by all kernels. A warp's row
// slots take kPerWarp neighbouring rows a round, kRounds rounds a page. For each slot
// the rounds of each of four groups are added, these sums by group, and the results
// over the slots (sum_slots).
constexpr int kGroups = 4;
template <int D>
struct Rounds {
    static constexpr int kPerWarp = HeadRow<D>::kPerWarp, kRounds = kPageRows / kPerWarp, kOfGroup = kRounds / kGroups;
};

// Sums of a row over the warp's row slots. Each step halves what a lane keeps: it
// ends with kKept pairs of neighbouring dimensions, from sum_dim on.
template <int D>
struct SlotSum {
    static constexpr int kSteps = D == 128 ? 2 : 3, kKept = 8 >> kSteps;
    f2 v[kKept];
};
template <int D>
__device__ __forceinline__ int sum_dim(int lane) {
    const int l = lane % HeadRow<D>::kLanes, grp = lane / HeadRow<D>::kLanes;
    return (grp & 1) * (D / 2) + 8 * l + (grp >> 1 & 1) * 4 + (D == 64 ? (grp >> 2) * 2 : 0);
}
template <int D>
__device__ __forceinline__ SlotSum<D> sum_slots(int lane, const Row& r) {
    f2 v[8] = {r.a.v[0], r.a.v[1], r.a.v[2], r.a.v[3], r.b.v[0], r.b.v[1], r.b.v[2], r.b.v[3]};
#pragma unroll
    for (int k = 0; k < SlotSum<D>::kSteps; ++k) {
        const int o = HeadRow<D>::kLanes << k;
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < (4 >> k); ++i) {
            const f2 keep = up ? v[i + (4 >> k)] : v[i], give = up ? v[i] : v[i + (4 >> k)];
            v[i] = f2_add(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    SlotSum<D> s;
#pragma unroll
    for (int i = 0; i < SlotSum<D>::kKept; ++i) s.v[i] = v[i];
    return s;
}

// The rare work on the rows of a page and head, by one warp: the codes of the
// first `grown` rows times `ratio`, and with `pool` the mean of the page's 64 keys
// (times their scale `unit`). Rows from `rows` on are not looked at.
template <int D, bool kQ8>
__device__ __forceinline__ void page_rows(const AppendArgs& a, bool is_v, int page, int h, int rows, int grown, float ratio,
                                          float unit, bool pool) {
    constexpr int kLanes = HeadRow<D>::kLanes, kPerWarp = Rounds<D>::kPerWarp, kAt = Rounds<D>::kOfGroup;
    const int lane = threadIdx.x & 31, l = lane % kLanes, grp = lane / kLanes;
    const long long head = (long long)page * a.Hkv + h, tile0 = head * kPageRows;
    Row sum{};
    // two groups of rounds at a time: their loads are in flight together
#pragma unroll 1
    for (int g0 = 0; g0 < kGroups; g0 += 2) {
        using Piece = typename std::conditional<kQ8, uint2, uint4>::type;
        Piece c[2 * kAt][2];
        auto ptr = [&](int r) {
            return static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + ((tile0 + r) * D + 8 * l) * (kQ8 ? 1 : 2);
        };
        constexpr int kHalf = D / 2 * (kQ8 ? 1 : 2);            // bytes
#pragma unroll
        for (int k = 0; k < 2 * kAt; ++k) {
            const int r = (g0 * kAt + k) * kPerWarp + grp;
            c[k][0] = c[k][1] = Piece{};
            if (r < rows) {
                c[k][0] = *reinterpret_cast<const Piece*>(ptr(r));
                c[k][1] = *reinterpret_cast<const Piece*>(ptr(r) + kHalf);
            }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            Row group{};
#pragma unroll
            for (int k = g * kAt; k < (g + 1) * kAt; ++k) {
                if constexpr (kQ8) {
                    const int r = (g0 * kAt + k) * kPerWarp + grp;
                    if (r < grown) {
                        *reinterpret_cast<uint2*>(ptr(r)) = c[k][0] = to_codes(from_codes(c[k][0]), ratio);
                        *reinterpret_cast<uint2*>(ptr(r) + kHalf) = c[k][1] = to_codes(from_codes(c[k][1]), ratio);
                    }
                    add(group.a, from_codes(c[k][0]));
                    add(group.b, from_codes(c[k][1]));
                } else {
                    const uint4 lo[1] = {c[k][0]}, hi[1] = {c[k][1]};
                    add(group.a, Raw8<bf16>::get(lo));
                    add(group.b, Raw8<bf16>::get(hi));
                }
            }
            add(sum.a, group.a);
            add(sum.b, group.b);
        }
    }
    if (!pool) return;
    const SlotSum<D> mean = sum_slots<D>(lane, sum);
    const f2 u = f2_pack(unit, unit), n = f2_pack(1.f / kPageRows, 1.f / kPageRows);
    f2* out = reinterpret_cast<f2*>(a.kpool + head * D + sum_dim<D>(lane));
#pragma unroll
    for (int i = 0; i < SlotSum<D>::kKept; ++i) out[i] = f2_mul(f2_mul(mean.v[i], n), u);    // (64 keys times a scale of 2^120 have no fp32 sum)
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
// older rows.
template <int D, bool kQ8>
__device__ __forceinline__ void token_kv(const AppendArgs& a, uint32_t u) {
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
    const int page = a.page_table[(long long)n * a.max_pages + t.block];   // block < max_pages by kv_len's check
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
        x = Turn(ang, w)(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);     // as the prompts' kernels: the same bits
        if (k_out != nullptr && grp == 0) store_row<D>(k_out + (t.row * a.Hkv + h) * D, l, x);
    }
    if (!ok) return;

    PageScale ps{true, true, 1.f};
    if constexpr (kQ8) {
        float m = warp_max_abs(row_max(x, 0.f));        // (behind the shuffles every lane has read the old scale)
        if (m == INFINITY) {
            drop_infinities(x.a);
            drop_infinities(x.b);
            m = warp_max_abs(row_max(x, 0.f));
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
    page_rows<D, kQ8>(a, is_v, page, h, t.lo + pool, grown ? t.lo : 0, old * (1.f / ps.s), ps.s, pool);
}

template <int D, bool kQ8>
__global__ void __launch_bounds__(kTokenThreads) append_token_kernel(const AppendArgs a, uint32_t q_ctas) {
    constexpr int kCtaSlots = kTokenThreads / HeadRow<D>::kLanes, kCtaWarps = kTokenThreads / 32;
    after_previous();
    if (blockIdx.x < q_ctas)
        token_q<D>(a, blockIdx.x * kCtaSlots + threadIdx.x / HeadRow<D>::kLanes);
    else
        token_kv<D, kQ8>(a, (blockIdx.x - q_ctas) * kCtaWarps + threadIdx.x / 32);
}

// ------------------------------------------------------------------ prompts
constexpr int kHeads = 4;                   // heads of a unit, which is of one token
constexpr int kStages = 2;                  // units in flight

// The sequence of a thread's last unit. The next one mostly belongs to it too, and
// then no load stands in front of its copies.
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
        tile0 = seq_tile_base(a.cu_new[at], at);
        tile1 = seq_tile_base(a.cu_new[at + 1], at + 1);
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
    // Goes to the sequence of tile index v, and says which of its new rows the tile has (none: empty).
    __device__ __forceinline__ PageTile find_tile(const AppendArgs& a, uint32_t v) {
        if (n < 0 || v < tile0 || v >= tile1) {         // the last n with its tile base <= v
            int lo = 0, hi = a.N;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (seq_tile_base(a.cu_new[mid], mid) <= v) lo = mid; else hi = mid;
            }
            load(a, lo);
        }
        if (bad || v < tile0 || v - tile0 >= (uint32_t)max_tiles(a.max_new)) return PageTile{0, 0, 0, 0};
        return page_tile(SeqNew{row0, first, count, false}, (int)(v - tile0));
    }
    __device__ __forceinline__ int page(const AppendArgs& a, int block) const {     // block < max_pages by kv_len's check
        return a.page_table[(long long)n * a.max_pages + block];
    }
};
// Flags every sequence that breaks the call's terms, also those that no token row
// or tile index leads to (by the first CTA).
__device__ __forceinline__ void flag_sequences(const AppendArgs& a) {
    if (blockIdx.x != 0) return;
    for (int n = threadIdx.x; n < a.N; n += blockDim.x)
        if (load_seq(a, n).bad || a.cu_new[n + 1] < a.cu_new[n]) flag_status(a.status, kStatusBadData);
}

enum UnitKind { kNone, kQ, kK, kV };
// A row slot's unit: heads part, part + parts, ... of a token's row of q, k or v.
struct Unit {
    int kind, t, part, pos, page;
};
// Starts the copies of a unit (row pieces of kThreads threads each) into a stage.
template <int D, int kThreads, int kKHeads, int kVHeads>
__device__ __forceinline__ void issue(const AppendArgs& a, const Unit& r, uint32_t at) {
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    if (r.kind != kNone) {
        const bf16* src = r.kind == kQ   ? static_cast<const bf16*>(a.q) + r.t * a.ld_q
                          : r.kind == kK ? static_cast<const bf16*>(a.k) + r.t * a.ld_k
                                         : static_cast<const bf16*>(a.v) + r.t * a.ld_v;
        const int H = r.kind == kQ ? a.Hq : a.Hkv, heads = r.kind == kQ ? kHeads : r.kind == kK ? kKHeads : kVHeads, parts = (int)parts_of(H, heads);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (i >= heads) break;
            const int h = r.part + i * parts;
            copy_row<bf16, D, kThreads>(at + 2 * i * kThreads * 16, src + (h < H ? h : 0) * D, l, h < H);
        }
    }
    copy_commit();
}

// ------------------------------------------------------------------ prompts into bf16 pages
constexpr int kThreads = 128;
constexpr int kCtas = 4;                    // resident CTAs of an SM
constexpr int kStageBytes = 2 * kHeads * kThreads * 16;

// Units of queries, keys, and values, which are copied as they are.
template <int D>
__global__ void __launch_bounds__(kThreads, kCtas) append_rows_kernel(const AppendArgs a, uint32_t q_parts, uint32_t units) {
    constexpr int kCtaSlots = kThreads / HeadRow<D>::kLanes, kRow = 2 * kThreads * 16;
    __shared__ __align__(16) uint8_t ring_s[kStages * kStageBytes];
    after_previous();
    const uint32_t ring = sm100::smem_u32(ring_s) + threadIdx.x * 16;
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    const uint32_t kv_parts = parts_of(a.Hkv, kHeads), per = q_parts + 2 * kv_parts;
    const uint32_t first = blockIdx.x * kCtaSlots + threadIdx.x / HeadRow<D>::kLanes, step = gridDim.x * kCtaSlots;

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
        if (r.kind != kQ) r.page = seq.page(a, r.pos / kPageRows);
        return r;
    };
    Unit cur = unit_at(first);
    issue<D, kThreads, kHeads, kHeads>(a, cur, ring);
    uint32_t st = 0;
    for (uint32_t base = blockIdx.x * kCtaSlots, u = first; base < units; base += step, u += step) {
        const Unit next = unit_at(u + step);
        issue<D, kThreads, kHeads, kHeads>(a, next, ring + (st ^ 1) * kStageBytes);
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

// The mean key of every page that the call has filled, in the order of page_rows: a CTA
// for each (block, KV head), each warp with its share of the rounds, so that the
// tile's loads are all in flight together.
template <int D>
__global__ void __launch_bounds__(kThreads) pool_filled_kernel(const AppendArgs a) {
    constexpr int kLanes = HeadRow<D>::kLanes, kPerWarp = Rounds<D>::kPerWarp, kAt = Rounds<D>::kOfGroup;
    static_assert(kThreads / 32 == kGroups, "a warp for each group of rounds");
    __shared__ __align__(16) float red[kGroups][kPerWarp][D];
    after_previous();
    SeqAt seq;
    const PageTile t = seq.find_tile(a, blockIdx.x / a.Hkv);
    if (t.hi != kPageRows || t.hi <= t.lo) return;
    const int page = seq.page(a, t.block);
    if (page < 0 || page >= a.num_pages) return;
    const int lane = threadIdx.x & 31, l = lane % kLanes, grp = lane / kLanes, warp = threadIdx.x / 32;
    const long long head = (long long)page * a.Hkv + blockIdx.x % a.Hkv;
    const bf16* rows = static_cast<const bf16*>(a.k_cache) + (head * kPageRows + warp * kAt * kPerWarp + grp) * D + 8 * l;
    uint4 c[kAt][2][1];
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
        c[k][0][0] = *reinterpret_cast<const uint4*>(rows + k * kPerWarp * D);
        c[k][1][0] = *reinterpret_cast<const uint4*>(rows + k * kPerWarp * D + D / 2);
    }
    Row group{};
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
        add(group.a, Raw8<bf16>::get(c[k][0]));
        add(group.b, Raw8<bf16>::get(c[k][1]));
    }
    store_sum<D>(red[warp][grp], l, group);
    __syncthreads();
    if (threadIdx.x >= D) return;
    float part[kPerWarp];
#pragma unroll
    for (int r = 0; r < kPerWarp; ++r) {
        part[r] = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) part[r] += red[g][r][threadIdx.x];
    }
#pragma unroll
    for (int n = 1; n < kPerWarp; n *= 2)
#pragma unroll
        for (int r = 0; r < kPerWarp; r += 2 * n) part[r] += part[r + n];
    a.kpool[head * D + threadIdx.x] = part[0] * (1.f / kPageRows);
}

// ------------------------------------------------------------------ prompts into 8-bit pages
// A CTA with a row slot for each row of a page. Its work: 64 units of queries, or of
// keys (values) those of the new rows of one (sequence, block, group of heads), whose
// scales the CTA finds in shared memory while the values wait in registers.
template <int D>
struct Blocks {
    static constexpr int kThreads = kPageRows * HeadRow<D>::kLanes, kCtas = 512 / kThreads;     // CTAs of an SM
    static constexpr int kWarps = kThreads / 32;
    // heads of a work: as many as the registers hold between the largest magnitude and the
    // codes (keys: with their rotation. V of two heads: 40.7 and 151 us at 8k and 32k
    // instead of 40.2 and 144; K of four: spills, 46.0 and 163)
    static constexpr int kKHeads = 2, kVHeads = 4;
    static constexpr int kStageBytes = 2 * kHeads * kThreads * 16;
    static constexpr int kRing = kStages * kStageBytes;
    // fp32 rows of a page and the work's heads of keys, for their mean; padded so that a
    // warp's row slots meet no bank twice
    static constexpr int kStride = D + 32 / HeadRow<D>::kPerWarp;
    static constexpr int kRed = kKHeads * kPageRows * kStride * 4;
};
template <int D>
__global__ void __launch_bounds__(Blocks<D>::kThreads, Blocks<D>::kCtas)
append_blocks_kernel(const AppendArgs a, uint32_t kv_works, uint32_t q_units, uint32_t works) {
    using B = Blocks<D>;
    extern __shared__ __align__(16) uint8_t ring_s[];
    __shared__ float wmax[2][B::kVHeads][B::kWarps];
    after_previous();
    const uint32_t ring = sm100::smem_u32(ring_s) + threadIdx.x * 16;
    float(*red)[kPageRows][B::kStride] = reinterpret_cast<float(*)[kPageRows][B::kStride]>(ring_s + B::kRing);   // with kpool
    const int l = threadIdx.x % HeadRow<D>::kLanes, slot = threadIdx.x / HeadRow<D>::kLanes;
    const int q_parts = (int)parts_of(a.Hq, kHeads), k_parts = (int)parts_of(a.Hkv, B::kKHeads), v_parts = (int)parts_of(a.Hkv, B::kVHeads);

    // the unit, and of a block of keys or values its rows lo .. hi - 1 that are new (all slots: `rows`, 0: none)
    struct Work {
        Unit u;
        int rows;
        __device__ __forceinline__ int lo() const { return rows & 255; }
        __device__ __forceinline__ int hi() const { return rows >> 8; }
    };
    SeqAt seq;
    auto work_at = [&](uint32_t w) {
        Work k{{kNone, 0, 0, 0, 0}, 0};
        if (w >= works) return k;
        if (w >= kv_works) {
            const uint32_t u = (w - kv_works) * kPageRows + slot, t = u / q_parts;
            if (u >= q_units || !seq.find(a, (int)t)) return k;
            k.u = {kQ, (int)t, (int)(u - t * q_parts), seq.first + (int)t - seq.row0, 0};
            return k;
        }
        const uint32_t per = k_parts + v_parts, v = w / per, rest = w - v * per;
        const PageTile t = seq.find_tile(a, v);
        if (t.hi <= t.lo) return k;
        k.rows = t.lo | t.hi << 8;
        const bool is_v = rest >= (uint32_t)k_parts;
        k.u.part = (int)(is_v ? rest - k_parts : rest);
        k.u.pos = t.block * kPageRows + slot;
        k.u.page = seq.page(a, t.block);
        k.u.t = (int)t.row + slot - t.lo;
        k.u.kind = is_v ? kV : kK;
        return k;
    };
    // copies of the rows that there are: the others' slots have nothing to copy
    auto issue_work = [&](const Work& k, uint32_t at) {
        Unit u = k.u;
        if (k.rows != 0 && (slot < k.lo() || slot >= k.hi())) u.kind = kNone;
        issue<D, B::kThreads, B::kKHeads, B::kVHeads>(a, u, at);
    };
    constexpr int kRow = 2 * B::kThreads * 16;

    Work cur = work_at(blockIdx.x);
    issue_work(cur, ring);
    uint32_t st = 0, buf = 0;
    for (uint32_t w = blockIdx.x; w < works; w += gridDim.x) {
        const Work next = work_at(w + gridDim.x);
        issue_work(next, ring + (st ^ 1) * B::kStageBytes);
        copy_wait<kStages - 1>();
        const uint32_t at = ring + st * B::kStageBytes;
        st ^= 1;
        const Unit& u = cur.u;
        if (cur.rows == 0) {
            // queries
            const bf16* weight = static_cast<const bf16*>(a.q_weight);
            const Turn turn(load_angles<bf16, D>(a.table, u.pos, l), load_weight<bf16, D>(weight, l));
            bf16* dst = static_cast<bf16*>(a.q_out) + (long long)u.t * a.Hq * D;
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int h = u.part + i * q_parts;
                const Row x = read_row<bf16, B::kThreads>(at + i * kRow);
                const Row y = turn(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);
                if (u.kind == kQ && h < a.Hq) store_row<D>(dst + h * D, l, y);
            }
            cur = next;
            continue;
        }
        // keys or values (uniform over the CTA up to the slot's row)
        auto block = [&](auto values) {
            constexpr bool is_v = decltype(values)::value;
            constexpr int kN = is_v ? B::kVHeads : B::kKHeads;
            const int parts = is_v ? v_parts : k_parts;
            const int lo = cur.lo(), hi = cur.hi();
            const bool fresh = slot >= lo && slot < hi, page_ok = u.page >= 0 && u.page < a.num_pages;
            if (!page_ok && threadIdx.x == 0) flag_status(a.status, kStatusBadData);
            bf16* k_out = is_v ? nullptr : static_cast<bf16*>(a.k_out);
            const long long head0 = (long long)(page_ok ? u.page : 0) * a.Hkv;
            float* scale = (is_v ? a.v_scale : a.k_scale) + head0;
            float old[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int h = u.part + i * parts;
                old[i] = page_ok && lo > 0 && h < a.Hkv ? scale[h] : 0.f;
            }
            Row y[kN];
            if constexpr (is_v) {
#pragma unroll
                for (int i = 0; i < kN; ++i) y[i] = read_row<bf16, B::kThreads>(at + i * kRow);
            } else {
                const bf16* weight = static_cast<const bf16*>(a.k_weight);
                const int pos = min(max(u.pos, u.pos - slot + lo), u.pos - slot + hi - 1);
                const Turn turn(load_angles<bf16, D>(a.table, pos, l), load_weight<bf16, D>(weight, l));
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const int h = u.part + i * parts;
                    const Row x = read_row<bf16, B::kThreads>(at + i * kRow);
                    y[i] = turn(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);
                    if (k_out != nullptr && fresh && h < a.Hkv) store_row<D>(k_out + ((long long)u.t * a.Hkv + h) * D, l, y[i]);
                }
            }
            float m[kN];
            auto block_max = [&] {
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const float r = warp_max_abs(fresh ? row_max(y[i], 0.f) : 0.f);
                    if ((threadIdx.x & 31) == 0) wmax[buf][i][threadIdx.x >> 5] = r;
                }
                __syncthreads();        // (and every thread has read the old scales, and its rows of this stage)
#pragma unroll
                for (int i = 0; i < kN; ++i) m[i] = warp_max_abs(wmax[buf][i][(threadIdx.x & 31) % B::kWarps]);
                buf ^= 1;               // the next maxima go elsewhere: these may still be read
            };
            block_max();
            float top = m[0];
#pragma unroll
            for (int i = 1; i < kN; ++i) top = fmaxf(top, m[i]);
            if (top == INFINITY) {
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    drop_infinities(y[i].a);
                    drop_infinities(y[i].b);
                }
                block_max();
            }
            const bool pool = a.kpool != nullptr && !is_v && hi == kPageRows && page_ok;
            float unit[kN];             // scales of the heads whose mean key is wanted
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int h = u.part + i * parts;
                unit[i] = 0.f;
                if (!page_ok || h >= a.Hkv) continue;
                const PageScale ps = page_scale(lo, old[i], m[i]);
                if (!ps.ok) {
                    if (threadIdx.x == 0) flag_status(a.status, kStatusBadData);
                    continue;
                }
                if (threadIdx.x == 0 && !ps.keep) scale[h] = ps.s;
                uint8_t* row = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + ((head0 + h) * kPageRows + slot) * D + 8 * l;
                uint2 c = make_uint2(0u, 0u), c2 = c;
                if (fresh) {
                    c = to_codes(y[i].a, 1.f / ps.s);
                    c2 = to_codes(y[i].b, 1.f / ps.s);
                } else if (slot < lo && (!ps.keep || pool)) {
                    c = *reinterpret_cast<const uint2*>(row);
                    c2 = *reinterpret_cast<const uint2*>(row + D / 2);
                    if (!ps.keep) {
                        c = to_codes(from_codes(c), old[i] * (1.f / ps.s));
                        c2 = to_codes(from_codes(c2), old[i] * (1.f / ps.s));
                    }
                }
                if (fresh || (slot < lo && !ps.keep)) {
                    *reinterpret_cast<uint2*>(row) = c;
                    *reinterpret_cast<uint2*>(row + D / 2) = c2;
                }
                if (pool) {
                    store_sum<D>(red[i][slot], l, Row{from_codes(c), from_codes(c2)});
                    unit[i] = ps.s;
                }
            }
            if (pool) {
                // the mean keys of the filled page, in the order of page_rows: a thread for each
                // row slot of a warp and dimension. (The next block's maxima meet at a barrier
                // before `red` is written again.)
                constexpr int kPerWarp = Rounds<D>::kPerWarp, kAt = Rounds<D>::kOfGroup;
                static_assert(B::kThreads % (kPerWarp * kPerWarp) == 0, "whole warps");
                __syncthreads();
#pragma unroll
                for (int e = threadIdx.x; e < kN * kPerWarp * D; e += B::kThreads) {
                    const int i = e / (kPerWarp * D), r = e % kPerWarp, d = e / kPerWarp % D;
                    float total = 0.f;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        float group = 0.f;
#pragma unroll
                        for (int k = 0; k < kAt; ++k) group += red[i][(g * kAt + k) * kPerWarp + r][d];
                        total += group;
                    }
#pragma unroll
                    for (int n = 1; n < kPerWarp; n *= 2) total += __shfl_xor_sync(0xffffffffu, total, n);
                    const float s = unit[i];
                    if (r == 0 && s > 0.f) a.kpool[(head0 + u.part + i * parts) * D + d] = total * (1.f / kPageRows) * s;
                }
            }
        };
        if (u.kind == kV)
            block(std::true_type());
        else
            block(std::false_type());
        cur = next;
    }
    copy_wait<0>();
    flag_sequences(a);
}

template <int D, bool kQ8>
cudaError_t go(const AppendArgs& a, cudaStream_t st) {
    cudaError_t e;
    if (a.max_new == 1) {
        constexpr long long kTokenSlots = kTokenThreads / HeadRow<D>::kLanes, kCtaWarps = kTokenThreads / 32;
        const long long q_ctas = a.q != nullptr ? (a.T * a.Hq + kTokenSlots - 1) / kTokenSlots : 0;
        const long long items = 2LL * a.N * a.Hkv;
        e = launch_dependent(append_token_kernel<D, kQ8>, dim3((unsigned)(q_ctas + (items + kCtaWarps - 1) / kCtaWarps)),
                             kTokenThreads, 0, st, a, (uint32_t)q_ctas);
        if (e == cudaSuccess) count_launches(1);
        return e;
    }
    const long long blocks = (long long)seq_tile_base((int)a.T, a.N) + 1;       // tile indices
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    const long long q_parts = a.q != nullptr ? parts_of(a.Hq, kHeads) : 0;
    if constexpr (kQ8) {
        using B = Blocks<D>;
        const int smem = B::kRing + (a.kpool != nullptr ? B::kRed : 0);
        e = cudaFuncSetAttribute(append_blocks_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, B::kRing + B::kRed);
        if (e != cudaSuccess) return e;
        const long long kv_works = blocks * (parts_of(a.Hkv, B::kKHeads) + parts_of(a.Hkv, B::kVHeads)), q_units = a.T * q_parts;
        const long long works = kv_works + (q_units + kPageRows - 1) / kPageRows;
        e = launch_dependent(append_blocks_kernel<D>, dim3((unsigned)std::min(works, (long long)B::kCtas * sms)), B::kThreads,
                             smem, st, a, (uint32_t)kv_works, (uint32_t)q_units, (uint32_t)works);
    } else {
        constexpr long long kCtaSlots = kThreads / HeadRow<D>::kLanes;
        const long long units = a.T * (q_parts + 2 * parts_of(a.Hkv, kHeads));
        e = launch_dependent<false>(append_rows_kernel<D>, dim3((unsigned)std::min((units + kCtaSlots - 1) / kCtaSlots, (long long)kCtas * sms)), kThreads, 0,
                             st, a, (uint32_t)q_parts, (uint32_t)units);
        if (e == cudaSuccess && a.kpool != nullptr) {
            count_launches(1);
            e = launch_dependent(pool_filled_kernel<D>, dim3((unsigned)(blocks * a.Hkv)), kThreads, 0, st, a);
        }
    }
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int D, cudaStream_t st) {
    if (a.k_scale != nullptr) return D == 128 ? go<128, true>(a, st) : go<64, true>(a, st);
    return D == 128 ? go<128, false>(a, st) : go<64, false>(a, st);
}

}  // namespace sas
