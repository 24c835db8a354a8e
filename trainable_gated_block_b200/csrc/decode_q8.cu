// sas_decode_paged_q8: the gated decode step of decode.cu over 8-bit pages.
//
// Pages hold e4m3 codes with one scale for K and one for V for each (page, KV
// head): key = ks kc, value = vs vc. With gate g of a kept block (0 for the
// current one) and x = sm_scale ks (q . kc) + g,
//   o = sum_j e^(x_j - m) vs_j vc_j / sum_j e^(x_j - m),  lse = m + log(sum_j e^(x_j - m)).
// With y = x log2(e) and m the running maximum of y, w = 2^(y - m + 15): the largest
// weight is 2^15, near the top of fp16, so that weights keep all bits down to
// 2^-29 of it, and some down to 2^-39. A block's product of weights and value codes
// has accumulators of its own, which times vs are added to those of the range:
// neither the weights nor the sum depend on the scales, however far apart they lie.
// (Sums of codes times 2^128, the largest that vs and 16-bit values allow, stay in
// range for 2^20 tokens: they are kept times 2^-36.)
// Codes are exact in fp16, the queries are scaled by a power of two (their
// largest element to 2^13 .. 2^14, what falls out of fp16 below is under 2^-30 of
// it), a weight is the sum of two fp16 numbers (2^-21 relative; one alone, 2^-11 off,
// made outputs differ by 4 to 6 parts in 10^4 of their norm); logits, sums and
// accumulators are fp32. Where up to four heads share a KV head the second numbers take
// the columns that these leave empty, which costs 64 x 33 slots of 8 KV heads 48.9 ->
// 49.3 us and 8 x 1025 165.7 -> 167.3; a product of their own, as beyond four, 49.3 and 171.9.
//
// HBM-bound design. Each (sequence, KV head) item has K + 1 slots: its kept blocks and
// the current one. The warps of a cluster of one to eight CTAs cut an item's slots
// into contiguous ranges; a warp streams its range on its own: its lanes resolve 32
// slots at a time (selection entry, page, gate, scales), lane 0 copies a (page, head)
// tile, 8 KiB of K and 8 KiB of V, by TMA into the warp's stage, and the warp does
// the block on mma.sync m16n8k16 with keys (or value dimensions) as the 16 rows
// and the up to 8 query heads of the group as the 8 columns:
//   S^T = K Q^T : A from ldmatrix over byte pairs. A lane gets four neighbouring
//       dimensions of a key; the first two serve as the lane's low k pair, the
//       others as its high pair, and Q is loaded in the same order.
//   O^T = V^T P^T : A from ldmatrix.trans over byte pairs, which are two
//       neighbouring dimensions of a key: the even ones become rows 0..7 of the
//       tile, the odd ones rows 8..15. P^T comes from S^T by movmatrix.
// No warp waits for another until its range is done. Then its state (m, l, o) is in
// its shared memory, and the cluster joins its warps' states over distributed shared
// memory: one launch, and nothing but the output is written. Twelve warps an SM, of
// twelve other blocks, hide each other's copies and math.
// Where clusters do not fill the device (few items with many slots, odd waves) all
// items' slots lie end to end instead, cut into a range for each warp of the device;
// a warp that leaves an item writes its state to the workspace, and a combine kernel
// joins them.
//
// Measured on one B200 (32/8 heads): eight 64k sequences with all history 164 us, 6.57
// TB/s of codes (by ranges 186); 64 sequences at 8k-64k, K = 32: 50.8 us, 5.4 TB/s (by
// ranges 55.0); one sequence at 8k, K = 16: 7.0 us (9.6), the latency of a launch, the
// chain selection entry -> page -> tile, one block's math and the join. A
// variant with a producer warp, consumers that meet at each item's end and
// one exp2f for each logit took 237 and 81.6 us: its math did not keep up.
#include <cuda_fp16.h>

#include <type_traits>

#include "byte_map.h"
#include "common.cuh"
#include "dependent.cuh"
#include "launch.h"
#include "page_rows.h"
#include "sm100.cuh"

namespace sas {
namespace {

using namespace sm100;

constexpr int kD = 128;
constexpr uint32_t kTileBytes = 64 * 128;          // one (page, head) tile of K or V: 64 rows of 128 codes
constexpr int kShortRows = 8;                      // short box (one 128-byte swizzle period) for a partial block
constexpr uint32_t kShortBytes = kShortRows * 128;
constexpr uint32_t kStageBytes = 2 * kTileBytes;
struct Block {              // a resolved block of a warp's stream
    int row0;               // first cache row of its tile
    int tokens;             // rows to copy; 0: nothing to read
    int item;
    int nvalid;             // rows to attend: tokens, or 0 when a scale is out of range
    float bias;             // gate, log2 units
    float ks, vs;           // vs times kUnit
    int pad;
};
constexpr float kUnit = 1.f / (1LL << 36);          // of the accumulators

// What a weight's exponent is taken against, with m the largest of the exponents: 15 below m.
// (Beyond 2^24 that difference would be rounded by more than fp16 has room for. Exponents
// are whole numbers there, and the weights stay at 1 or below.)
__device__ __forceinline__ float weight_ref(float m) { return fabsf(m) < 16777216.f ? m - 15.f : m; }
constexpr int kList = 64;                           // two batches of a warp

// A cluster of kCtas CTAs of kWarps warps with one stage each has one item: twelve
// warps an SM (their rings are its shared memory).
constexpr int kSmWarps = 12;
// Without clusters the slots of all items are one line, cut into a range for each
// warp of the device: a CTA of four warps with three stages each an SM, or, where their
// ranges would be longer than the 32 slots that a warp resolves at a time, of ten warps
// of one stage, which have more math under way. (Measured, four / ten: 1,032 slots
// 12.8 / 12.6 us, 8,200 slots 31.6 / 33.5, 16,400 slots 51.9 / 55.3, 19,800 slots
// 62.9 / 62.7, 24,024 slots 72.2 / 71.3, 39,000 slots 111.9 / 109.2, 77,400 slots 217 / 202;
// of five heads a KV head 16,400 slots 51.4 / 56.7, 77,400 slots 230 / 209.)
constexpr int kRangeWarps = 4, kRangeStages = 3, kLongRangeWarps = 10, kLongRangeStages = 1;

// kWarps warps of a CTA, kDepth ring stages each, and their shared memory.
template <int kWarps, int kDepth>
struct Shape {
    static constexpr uint32_t kOffList = kWarps * kDepth * kStageBytes;
    static constexpr uint32_t kOffBar = kOffList + kWarps * kList * sizeof(Block);
    static constexpr uint32_t kOffAbort = kOffBar + kWarps * kDepth * 8;
    static constexpr uint32_t kOffMl = (kOffAbort + kWarps * 4 + 7) / 8 * 8;     // a warp's weight_ref and sum for each head
    static constexpr uint32_t kSmem = kOffMl + kWarps * 8 * sizeof(float2) + 1024;       // + alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

struct Params {
    const __nv_bfloat16* q;
    const float* k_scale;
    const float* v_scale;
    int num_pages;
    const int32_t* page_table;
    int max_pages;
    const int32_t* kv_len;
    int Hq, Hkv, G, K;
    const int32_t* idx;
    const int32_t* cnt;
    const float* log_gate;
    float qscale;           // sm_scale * log2(e)
    long long V;            // n_items * (K + 1) block slots
    int ranges;
    int nslot;              // partial slots per query head
    float* part_o;          // [N * Hq, nslot, D], times kUnit
    float* part_ml;         // [N * Hq, nslot, 2]
    __nv_bfloat16* o;       // [N, Hq, D]; lse [N, Hq] or null (clusters; else the combine writes them)
    float* lse;
    int* status;
};

// Range r owns block slots [r V / ranges, (r + 1) V / ranges); range_of is its inverse.
__host__ __device__ __forceinline__ long long range_begin(long long r, long long V, int ranges) { return r * V / ranges; }
__host__ __device__ __forceinline__ int range_of(long long s, long long V, int ranges) {
    return (int)(((s + 1) * ranges - 1) / V);
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Address of a cluster's CTA's counterpart of a shared memory address; loads from there.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int cta) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
    return r;
}
__device__ __forceinline__ float2 ld_cluster(uint32_t addr) {
    float2 x;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
    return x;
}
// Every thread of every CTA of the cluster; what they wrote before is visible behind it.
template <int kCtas>
__device__ __forceinline__ void cluster_sync() {
    if (kCtas == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// D (16x8 fp32) += A (16x16 fp16) * B (16x8 fp16)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 codes to two fp16 pairs (exact): codes 0, 1 and codes 2, 3.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The part of a weight that fp16's 11 bits hold.
__device__ __forceinline__ float upper(float w) { return __uint_as_float(__float_as_uint(w) & 0xffffe000u); }

// A block slot: whether it holds a kept or current block, that block's tile, and
// its gate (in log2 units) and scales (finish() comes after the tile's copy is under way).
struct Slot {
    bool use;
    int row0, tokens, item;
    float gate, ks, vs;
};
__device__ __forceinline__ Slot resolve(const Params& p, long long v) {
    Slot r;
    r.use = false;
    r.row0 = r.tokens = 0;
    r.gate = 0.f;
    r.ks = r.vs = 1.f;
    const int Kp1 = p.K + 1;
    const int t = (int)(v % Kp1);
    r.item = (int)(v / Kp1);
    const int n = r.item / p.Hkv, h = r.item % p.Hkv;
    // independent loads first: an entry that turns out not to be one is not used
    const int L = p.kv_len[n], cnt = p.cnt[r.item];
    const long long srow = (long long)r.item * p.K + t;
    int j = t < p.K ? p.idx[srow] : -1;
    const float gate = t < p.K ? p.log_gate[srow] : 0.f;
    if (L < 1 || L > (long long)p.max_pages * kBlock) {
        if (L != 0) flag_status(p.status, kStatusBadData);       // 0: a padding entry
        return r;
    }
    const int c = (L - 1) / kBlock;
    const int n_sel = max(0, min(cnt, min(p.K, c)));
    if (n_sel != cnt) flag_status(p.status, kStatusBadData);
    if (t > n_sel) return r;
    const bool cur = t == n_sel;
    if (cur) j = c;
    r.gate = cur ? 0.f : gate * kLog2e;
    if (r.gate == -INFINITY && j >= 0 && j < c) return r;        // a closed gate: nothing of the block is looked at
    r.use = true;
    int page = -1;
    if (j >= 0 && j < c + cur) page = p.page_table[(long long)n * p.max_pages + j];   // j <= c < max_pages
    if (page < 0 || page >= p.num_pages) {
        flag_status(p.status, kStatusBadData);
        return r;
    }
    r.row0 = (page * p.Hkv + h) * kBlock;                        // < 2^31 (checked on the host)
    r.tokens = cur ? L - c * kBlock : kBlock;
    r.ks = p.k_scale[(long long)page * p.Hkv + h];
    r.vs = p.v_scale[(long long)page * p.Hkv + h];
    return r;
}
__device__ __forceinline__ void finish(const Params& p, const Slot& r, Block& b) {
    const bool ok = scale_ok(r.ks) && scale_ok(r.vs);
    if (!ok) flag_status(p.status, kStatusBadData);
    b.bias = r.gate;
    b.nvalid = ok ? r.tokens : 0;
    b.ks = r.ks;
    b.vs = r.vs * kUnit;
}

// kCluster = 0: the ranges of the whole device, whose partials go to the workspace.
// Otherwise a cluster of kCluster CTAs for each item: its warps cut the item's K + 1
// slots, and their partials meet in the cluster's shared memory.
template <int kWarps, int kDepth, int kCluster>
__global__ void __launch_bounds__(kWarps * 32, kCluster == 0 ? 1 : kSmWarps / kWarps)
decode_q8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_k8, const __grid_constant__ CUtensorMap map_v8, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    after_previous();
    constexpr int kRanges = kWarps * kCluster;      // of an item
    const int cta = (int)blockIdx.x % max(kCluster, 1);
    const int range = kCluster == 0 ? warp * (int)gridDim.x + (int)blockIdx.x : warp * kCluster + cta;
    if (kCluster == 0 && range >= p.ranges) return;

    uint8_t* ring = smem + warp * kDepth * kStageBytes;
    Block* list = reinterpret_cast<Block*>(smem + Shape<kWarps, kDepth>::kOffList) + warp * kList;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Shape<kWarps, kDepth>::kOffBar) + warp * kDepth;
    volatile int* abort = reinterpret_cast<int*>(smem + Shape<kWarps, kDepth>::kOffAbort) + warp;
    if (lane == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        for (int s = 0; s < kDepth; ++s) mbar_init(&full[s], 1);
        *abort = 0;
        fence_barrier_init();
    }
    __syncwarp();

    const int Kp1 = p.K + 1;
    const int own_item = (int)(blockIdx.x / max(kCluster, 1));
    long long v, v1;            // next slot to resolve, end of the range
    if constexpr (kCluster == 0) {
        v = range_begin(range, p.V, p.ranges);
        v1 = range_begin(range + 1, p.V, p.ranges);
    } else {
        v = (long long)own_item * Kp1 + range_begin(range, Kp1, kRanges);
        v1 = (long long)own_item * Kp1 + range_begin(range + 1, Kp1, kRanges);
    }
    const int last_item = (int)((v1 - 1) / Kp1);
    int cur_item = kCluster == 0 ? (int)(v / Kp1) : own_item;

    const int grp = lane >> 2, tig = lane & 3;     // mma fragment coordinates
    const bool few_heads = p.G <= 4;               // columns 4..7 are the same heads as 0..3, for the weights' lower parts
    // ldmatrix: this lane's row within 16 keys; chunk c of that row is at lofs ^ (c << 4) (c even; the odd
    // chunk of the pair goes to the upper lanes)
    const uint32_t lofs = sw128_offset((lane & 7) + (lane & 8), lane >> 4);
    const uint32_t ring_s = smem_u32(ring) + lofs;
    uint32_t qb[8][2];          // Q^T as B fragments: 8 k-steps x (dims 4tig, +1 / +2, +3 of the step) of head grp
    float o[8][4];              // O^T times kUnit: tile mt, dims 16mt + 2grp (+1 in [2], [3]) x heads 2tig, 2tig + 1
    float m[2], mr[2], l[2];    // heads 2tig, 2tig + 1: max of y and its weight_ref; this lane's part of the sum
    float qm[2];                // sm_scale log2(e) over the query scale of those heads

    auto start = [&](int item) {
        const int n = item / p.Hkv, h = item % p.Hkv;
        const int g = few_heads ? grp & 3 : grp;
        const bool real = g < p.G;
        const uint2* qrow = reinterpret_cast<const uint2*>(p.q + ((long long)n * p.Hq + h * p.G + (real ? g : 0)) * kD);
        uint2 qr[8];
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) qr[kk] = real ? qrow[4 * kk + tig] : make_uint2(0u, 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const float2 a = bf16x2_to_f32(qr[kk].x), b = bf16x2_to_f32(qr[kk].y);
            top = fmaxf(top, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e with top 2^e in [2^13, 2^14), or at most 2^126 (rows below 2^-112, down to subnormals); 1 for an infinite row
        const int te = (int)(__float_as_uint(top) >> 23);           // biased exponent of top
        const int e = te == 255 ? 0 : min(13 + 127 - te, 126);
        const float qs = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const float2 a = bf16x2_to_f32(qr[kk].x), b = bf16x2_to_f32(qr[kk].y);
            qb[kk][0] = pack_f16x2(a.x * qs, a.y * qs);
            qb[kk][1] = pack_f16x2(b.x * qs, b.y * qs);
        }
        const float qi = p.qscale * __uint_as_float((uint32_t)(127 - e) << 23);
        qm[0] = __shfl_sync(0xffffffffu, qi, 8 * tig);
        qm[1] = __shfl_sync(0xffffffffu, qi, 8 * tig + 4);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m[0] = m[1] = mr[0] = mr[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    };
    // row of the item's first query head, at this range's partial slot
    auto part_row = [&](int item) {
        const int n = item / p.Hkv, h = item % p.Hkv;
        return ((long long)n * p.Hq + h * p.G) * p.nslot + (range - range_of((long long)item * Kp1, p.V, p.ranges));
    };
    auto write_empty = [&](int item) {
        if (lane < p.G) {
            float* ml = p.part_ml + (part_row(item) + (long long)lane * p.nslot) * 2;
            ml[0] = -INFINITY;
            ml[1] = 0.f;
        }
    };
    // row g's partial: weight_ref and sum to ml + g * stride, its accumulators to o_out + g * stride * D
    auto write_to = [&](float2* ml, float* o_out, int stride) {
        if (few_heads) {
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][e] += __shfl_xor_sync(0xffffffffu, o[mt][e], 2);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
            if (l[e] != l[e]) mr[e] = fmaxf(mr[e], -1e30f);   // only NaN logits: the row is not an empty one
            const int g = 2 * tig + e;
            if (g >= p.G) continue;
            if (grp == 0) ml[(long long)g * stride] = make_float2(mr[e], l[e]);
            float* dst = o_out + (long long)g * stride * kD + 2 * grp;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) *reinterpret_cast<float2*>(dst + 16 * mt) = make_float2(o[mt][e], o[mt][2 + e]);
        }
    };
    auto write = [&](int item) {
        const long long row = part_row(item);
        write_to(reinterpret_cast<float2*>(p.part_ml) + row, p.part_o + row * kD, p.nslot);
    };

    if (kCluster > 0 && v1 - v > 1) {
        // the item's pages are wanted behind its selection entries, its queries behind the
        // first tiles of all warps: they come to L2 meanwhile (24 sequences of 33 slots
        // 25.0 -> 24.5 us; with one slot a warp it costs 0.1)
        const int n = own_item / p.Hkv, h = own_item % p.Hkv;
        if (32 * lane < p.max_pages) prefetch_l2(p.page_table + (long long)n * p.max_pages + 32 * lane);
        if (lane < 2 * p.G) prefetch_l2(p.q + ((long long)n * p.Hq + h * p.G) * kD + 64 * lane);
    }
    uint32_t found = 0, issued = 0, done = 0;      // blocks resolved, copied, consumed
    bool started = false, alive = true;
    while (true) {
        // resolve a batch of slots when the ring has nothing more to copy
        Slot slot;
        slot.use = false;
        uint32_t at = 0;
        if (v < v1 && found == issued && found - done <= kList - 32) {
            if (v + lane < v1) slot = resolve(p, v + lane);
            const unsigned mask = __ballot_sync(0xffffffffu, slot.use);
            at = (found + __popc(mask & ((1u << lane) - 1u))) % kList;
            if (slot.use) {
                list[at].row0 = slot.row0;
                list[at].tokens = slot.tokens;
                list[at].item = slot.item;
            }
            found += __popc(mask);
            v += 32;
            __syncwarp();
        }
        while (issued < found && issued - done < kDepth) {
            if (lane == 0) {
                const Block& b = list[issued % kList];
                const uint32_t st = issued % kDepth;
                uint8_t* dst = ring + st * kStageBytes;
                if (b.tokens == kBlock) {
                    mbar_expect_tx(&full[st], kStageBytes);
                    tma_load_3d(dst, &map_k, &full[st], 0, 0, b.row0);
                    tma_load_3d(dst + kTileBytes, &map_v, &full[st], 0, 0, b.row0);
                } else {
                    // partial block (the current one): only the 8-row groups holding tokens; none of a skipped one
                    const int ng = (b.tokens + kShortRows - 1) / kShortRows;
                    mbar_expect_tx(&full[st], (uint32_t)ng * 2 * kShortBytes);
                    for (int g8 = 0; g8 < ng; ++g8) {
                        tma_load_3d(dst + g8 * kShortBytes, &map_k8, &full[st], 0, 0, b.row0 + g8 * kShortRows);
                        tma_load_3d(dst + kTileBytes + g8 * kShortBytes, &map_v8, &full[st], 0, 0,
                                    b.row0 + g8 * kShortRows);
                    }
                }
            }
            ++issued;
        }
        if (slot.use) finish(p, slot, list[at]);
        __syncwarp();
        if (done == issued) {
            if (v < v1) continue;
            break;                                 // nothing left in this range
        }
        const Block b = list[done % kList];
        const uint32_t st = done % kDepth;
        if (!started || b.item != cur_item) {
            if (started) write(cur_item++);
            for (; cur_item < b.item; ++cur_item) write_empty(cur_item);
            start(b.item);
            started = true;
        }
        if (!mbar_wait_warp(&full[st], (done / kDepth) & 1, abort, p.status)) {
            alive = false;
            break;
        }
        if (b.nvalid > 0) {
            const uint32_t kt = ring_s + st * kStageBytes, vt = kt + kTileBytes;
            float s[4][4];      // S^T: keys 16mt + grp (+8 in [2], [3]) x heads 2tig, 2tig + 1
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 8; kk += 2) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    uint32_t r[4], a0, a1, a2, a3;
                    ldsm_x4((kt ^ (kk << 4)) + mt * 2048, r);
                    codes_f16(r[0], a0, a2);
                    codes_f16(r[1], a1, a3);
                    mma16816(s[mt], a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
                    codes_f16(r[2], a0, a2);
                    codes_f16(r[3], a1, a3);
                    mma16816(s[mt], a0, a1, a2, a3, qb[kk + 1][0], qb[kk + 1][1]);
                }
            }
            const float f[2] = {qm[0] * b.ks, qm[1] * b.ks};
            float bm[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][e] = fmaf(s[mt][e], f[e & 1], b.bias);
            if (b.nvalid < kBlock) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (16 * mt + grp + 8 * (e >> 1) >= b.nvalid) s[mt][e] = -INFINITY;
                // rows past the sequence end are zeroed: their weight is 0, but whatever
                // the page holds there must not reach O as 0 * NaN
                uint8_t* vrow = ring + st * kStageBytes + kTileBytes;
                for (int e = b.nvalid * 8 + lane; e < kBlock * 8; e += 32)
                    *reinterpret_cast<uint4*>(vrow + sw128_offset(e >> 3, e & 7)) = make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) bm[e] = max3(bm[e], s[mt][e], s[mt][e + 2]);
            float sc[2], mu[2], ls[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) bm[e] = fmaxf(bm[e], __shfl_xor_sync(0xffffffffu, bm[e], x));
                m[e] = fmaxf(m[e], bm[e]);
                const float ref = weight_ref(m[e]);
                mu[e] = ref == -INFINITY ? 0.f : ref;            // no finite logit yet: 2^(-inf - 0) = 0
                sc[e] = fast_exp2(mr[e] - mu[e]);
                mr[e] = ref;
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[mt][e] = fast_exp2(s[mt][e] - mu[e & 1]);
                    ls[e & 1] += s[mt][e];
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) l[e] = fmaf(l[e], sc[e], ls[e]);
            if (__any_sync(0xffffffffu, sc[0] != 1.f || sc[1] != 1.f)) {     // a maximum grew
#pragma unroll
                for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][e] *= sc[e & 1];
            }
            // O^T of this block. P^T as B fragments: the weights' upper parts and what is left
            // of them, in the columns of the heads and those behind or one after the other
            auto product = [&](auto side_by_side) {
                constexpr int kParts = decltype(side_by_side)::value ? 1 : 2;
                uint32_t pb[kParts][4][2];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float w0 = s[mt][2 * e], w1 = s[mt][2 * e + 1], u0 = upper(w0), u1 = upper(w1);
                        if (kParts == 1) {
                            pb[0][mt][e] = transpose8x8(tig < 2 ? pack_f16x2(u0, u1) : pack_f16x2(w0 - u0, w1 - u1));
                        } else {
                            pb[0][mt][e] = transpose8x8(pack_f16x2(u0, u1));
                            pb[kParts - 1][mt][e] = transpose8x8(pack_f16x2(w0 - u0, w1 - u1));
                        }
                    }
#pragma unroll
                for (int mt = 0; mt < 8; mt += 2) {
                    float pv[2][4];     // in codes
#pragma unroll
                    for (int e = 0; e < 4; ++e) pv[0][e] = pv[1][e] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        uint32_t r[4], a0, a1, a2, a3;
                        ldsm_x4_t((vt ^ (mt << 4)) + kk * 2048, r);
                        codes_f16(__byte_perm(r[0], 0u, 0x3120), a0, a1);
                        codes_f16(__byte_perm(r[1], 0u, 0x3120), a2, a3);
#pragma unroll
                        for (int i = 0; i < kParts; ++i) mma16816(pv[0], a0, a1, a2, a3, pb[i][kk][0], pb[i][kk][1]);
                        codes_f16(__byte_perm(r[2], 0u, 0x3120), a0, a1);
                        codes_f16(__byte_perm(r[3], 0u, 0x3120), a2, a3);
#pragma unroll
                        for (int i = 0; i < kParts; ++i) mma16816(pv[1], a0, a1, a2, a3, pb[i][kk][0], pb[i][kk][1]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[mt][e] = fmaf(pv[0][e], b.vs, o[mt][e]);
                        o[mt + 1][e] = fmaf(pv[1][e], b.vs, o[mt + 1][e]);
                    }
                }
            };
            if (few_heads)
                product(std::true_type());
            else
                product(std::false_type());
        }
        fence_proxy_async_smem();     // this stage's reads and zeroes before its next copy
        __syncwarp();
        ++done;
    }
    if (!alive) {                     // let the copies in flight land before the CTA exits
        volatile int no_abort = 0;
        for (uint32_t k = done; k < issued; ++k) mbar_wait(&full[k % kDepth], (k / kDepth) & 1, &no_abort, nullptr);
    }
    if constexpr (kCluster == 0) {
        if (started) write(cur_item++);
        for (; cur_item <= last_item; ++cur_item) write_empty(cur_item);
    } else {
        // the warp's partial into its ring, which is done with
        static_assert(kRanges <= 32, "a lane for each partial");
        float2* ml = reinterpret_cast<float2*>(smem + Shape<kWarps, kDepth>::kOffMl);
        if (started)
            write_to(ml + warp * 8, reinterpret_cast<float*>(ring), 1);
        else if (lane < p.G)
            ml[warp * 8 + lane] = make_float2(-INFINITY, 0.f);
        cluster_sync<kCluster>();
        const int n = cur_item / p.Hkv, h = cur_item % p.Hkv;
        // the halves of the heads' rows, two dimensions a lane, over all warps of the cluster
        for (int u = warp * kCluster + cta; u < 2 * p.G; u += kRanges) {
            const int g = u >> 1, d = (u & 1) * 64 + 2 * lane;
            float wm = -INFINITY, wl = 0.f;
            if (lane < kRanges) {
                const float2 w = ld_cluster(cluster_addr(smem_u32(ml + lane / kCluster * 8 + g), lane % kCluster));
                wm = w.x, wl = w.y;
            }
            const float M = warp_max(wm);
            const float f = wm == -INFINITY ? 0.f : exp2f(wm - M);
            const unsigned some = __ballot_sync(0xffffffffu, wm != -INFINITY);
            float L = wm == -INFINITY ? 0.f : wl * f;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll 8
            for (int i = 0; i < kRanges; ++i) {
                // (an empty partial's place is read all the same, and not used)
                const float2 x = ld_cluster(cluster_addr(
                    smem_u32(smem + i / kCluster * kDepth * kStageBytes) + (g * kD + d) * (int)sizeof(float), i % kCluster));
                const float fi = __shfl_sync(0xffffffffu, f, i);
                if (some >> i & 1) {
                    acc.x = fmaf(x.x, fi, acc.x);
                    acc.y = fmaf(x.y, fi, acc.y);
                }
            }
            const bool none = M == -INFINITY;
            const long long row = (long long)n * p.Hq + h * p.G + g;
            const float inv = (1.f / kUnit) / L;
            *reinterpret_cast<__nv_bfloat162*>(p.o + row * kD + d) =
                none ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
            if (p.lse != nullptr && d == 0) p.lse[row] = none ? M : (M + log2f(L)) * kLn2;
        }
        cluster_sync<kCluster>();   // nobody leaves while its partials are read
    }
}

// Joins the partials of one (sequence, query head): kGroups groups of threads
// take every kGroups-th partial, one thread of a group for each output
// dimension, and meet in shared memory. Latency is what counts here: a thread
// has the loads of eight partials in flight. A row without a readable block
// gets 0 and an lse of -inf.
template <int kGroups>
__global__ void __launch_bounds__(kD* kGroups)
decode_q8_combine_kernel(const float* part_o, const float* part_ml, int nslot, int Hq, int Hkv,
                         int G, int K, long long V, int ranges, __nv_bfloat16* o, float* lse) {
    __shared__ float acc_s[kGroups][kD];
    __shared__ float2 ml_s[kGroups];
    after_previous();
    const long long row = blockIdx.x;          // n * Hq + hq
    const int d = threadIdx.x % kD, grp = threadIdx.x / kD;
    const long long s0 = (row / Hq * Hkv + row % Hq / G) * (K + 1);
    const int n = range_of(s0 + K, V, ranges) - range_of(s0, V, ranges) + 1;
    const float2* ml = reinterpret_cast<const float2*>(part_ml) + row * nslot;
    const float* po = part_o + row * nslot * kD + d;
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int base = grp; base < n; base += 8 * kGroups) {
        float2 w[8];
        float x[8];
        float mx = M;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = base + i * kGroups;
            w[i] = s < n ? ml[s] : make_float2(-INFINITY, 0.f);
            x[i] = s < n ? po[(long long)s * kD] : 0.f;    // not written for an empty partial: not used then
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, w[i].x);
        if (mx == -INFINITY) continue;
        const float f0 = exp2f(M - mx);
        L *= f0;
        acc *= f0;
        M = mx;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (w[i].x == -INFINITY) continue;
            const float f = exp2f(w[i].x - M);
            L = fmaf(w[i].y, f, L);
            acc = fmaf(x[i], f, acc);
        }
    }
    if (kGroups > 1) {
        acc_s[grp][d] = acc;
        if (d == 0) ml_s[grp] = make_float2(M, L);
        __syncthreads();
        if (grp) return;
        float mx = M;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) mx = fmaxf(mx, ml_s[i].x);
        if (mx != -INFINITY) {
            const float f0 = exp2f(M - mx);
            L *= f0;
            acc *= f0;
            M = mx;
#pragma unroll
            for (int i = 1; i < kGroups; ++i) {
                if (ml_s[i].x == -INFINITY) continue;
                const float f = exp2f(ml_s[i].x - M);
                L = fmaf(ml_s[i].y, f, L);
                acc = fmaf(acc_s[i][d], f, acc);
            }
        }
    }
    const bool none = M == -INFINITY;
    o[row * kD + d] = __float2bfloat16_rn(none ? 0.f : acc * ((1.f / kUnit) / L));
    if (lse != nullptr && d == 0) lse[row] = none ? M : (M + log2f(L)) * kLn2;
}

struct Layout {
    long long V;
    int warps, ctas;            // of a CTA, of a cluster; ctas 0: ranges
    int grid, ranges, nslot;
};
constexpr struct {
    int warps, ctas;
} kClusters[] = {{4, 8}, {3, 8}, {4, 4}, {3, 4}, {4, 2}, {3, 2}, {4, 1}, {3, 1}};        // most warps first

// The clusters that go through their items' slots in the fewest rounds (of one slot a
// warp): as many warps as still have all clusters resident together, or, with single
// CTAs, waves of which the last is at least half full. (Clusters stay within a GPC, so
// that not all places can be had: an eighth is left out.) Where one round does, the
// fewest warps; else the most. Left to the ranges: few items with many slots (the
// clusters' warps would be under half of what the device holds), and odd waves.
// Measured (us, clusters / ranges and combine; items x slots, an item being a sequence
// and KV head; eight items are one sequence of 8 KV heads, or eight of one):
//   8 x 17 7.0 / 9.6, 32 x 17 8.8 / 8.8, 64 x 17 10.3 / 14.2, 128 x 17 13.3 / 16.3,
//   64 x 33 14.2 / 17.1, 128 x 33 18.2 / 21.0, 192 x 33 24.4 / 27.8, 384 x 33 39.3 / 44.4,
//   512 x 33 49.7 / 55.0, 576 x 33 54.6 / 61.5, 1024 x 33 91.9 / 100.1, 32 x 65 15.3 / 15.6,
//   64 x 65 18.1 / 22.6, 192 x 65 39.5 / 43.4, 512 x 65 89.3 / 96.7, 64 x 1025 169 / 186;
// left to the ranges:
//   8 x 33 9.1 / 8.9, 16 x 33 10.2 / 9.1, 24 x 33 11.4 / 10.8, 8 x 65 11.4 / 9.7,
//   16 x 65 13.0 / 11.8, 24 x 65 14.2 / 13.7, 8 x 129 15.9 / 13.1, 16 x 129 17.3 / 16.3, and
//   with a last wave of a third 600 x 33 66.0 / 62.9, 640 x 33 66.9 / 66.2, 600 x 65 120 / 112.
// At 32 x 33 (two rounds of 32 warps for one slot more than they have) the rule takes the
// slower: 12.2 / 11.3.
bool choose_clusters(long long items, int slots, int sms, int& cta_warps, int& ctas) {
    long long best = 0;
    for (const auto& c : kClusters) {
        const long long most = (long long)(kSmWarps / c.warps) * sms * (c.ctas > 1 ? 7 : 8) / 8, need = items * c.ctas;
        const long long waves = (need + most - 1) / most;
        if (waves > 1 && (c.ctas > 1 || 2 * (need - (waves - 1) * most) < most)) continue;
        const int warps = c.warps * c.ctas;
        const long long rounds = waves * ((slots + warps - 1) / warps);
        if (best && (rounds > best || (rounds == best && best > 1))) continue;
        best = rounds;
        cta_warps = c.warps;
        ctas = c.ctas;
    }
    return best == 1 || (best > 1 && 2 * items * kClusters[0].warps * kClusters[0].ctas >= (long long)kSmWarps * sms);
}

Layout layout(int N, int Hkv, int K) {
    Layout r;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    r.V = (long long)N * Hkv * (K + 1);
    if (choose_clusters((long long)N * Hkv, K + 1, sms, r.warps, r.ctas)) {
        r.grid = N * Hkv * r.ctas;
        r.ranges = r.nslot = 0;
        return r;
    }
    r.ctas = 0;
    r.warps = r.V > 32LL * kRangeWarps * sms ? kLongRangeWarps : kRangeWarps;
    r.grid = (int)(r.V < sms ? r.V : sms);
    const long long most = (long long)sms * r.warps;
    r.ranges = (int)(r.V < most ? r.V : most);
    const long long mn = r.V / r.ranges;                     // shortest range
    const long long span = (K + 1 + mn - 1) / mn + 1;        // ranges one item's slots can touch
    r.nslot = (int)(span < r.ranges ? span : r.ranges);
    return r;
}

template <int kWarps, int kDepth, int kCluster = 0>
cudaError_t launch(const Layout& lay, const CUtensorMap (&map)[4], const Params& p, cudaStream_t st) {
    constexpr int kSmem = (int)Shape<kWarps, kDepth>::kSmem;
    const auto kernel = decode_q8_kernel<kWarps, kDepth, kCluster>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent<true, kCluster>(kernel, dim3(lay.grid), kWarps * 32, kSmem, st, map[0], map[1], map[2], map[3], p);
}

}  // namespace

size_t decode_q8_workspace(int N, int Hq, int Hkv, int K) {
    const Layout lay = layout(N, Hkv, K);
    if (lay.ctas) return 256;       // nothing is kept there (ranges need more: 520 bytes for one partial)
    const size_t per = (size_t)N * Hq * lay.nslot;
    return sizeof(float) * (per * kD + per * 2);
}

cudaError_t launch_decode_q8(const DecodeArgs& a, const float* k_scale, const float* v_scale, void* workspace,
                             cudaStream_t st) {
    const long long cache_rows = (long long)a.num_pages * a.Hkv * kBlock;
    const Layout lay = layout(a.N, a.Hkv, a.K);
    float* part_o = static_cast<float*>(workspace);
    float* part_ml = part_o + (size_t)a.N * a.Hq * lay.nslot * kD;
    CUtensorMap map[4];
    if (!make_byte_map(&map[0], a.k_cache, cache_rows, kBlock) || !make_byte_map(&map[1], a.v_cache, cache_rows, kBlock) ||
        !make_byte_map(&map[2], a.k_cache, cache_rows, kShortRows) ||
        !make_byte_map(&map[3], a.v_cache, cache_rows, kShortRows))
        return cudaErrorInvalidValue;
    Params p;
    p.q = (const __nv_bfloat16*)a.q;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.num_pages = a.num_pages;
    p.page_table = a.page_table;
    p.max_pages = a.max_pages;
    p.kv_len = a.kv_len;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.K = a.K;
    p.idx = a.idx;
    p.cnt = a.cnt;
    p.log_gate = a.log_gate;
    p.qscale = a.sm_scale * kLog2e;
    p.V = lay.V;
    p.ranges = lay.ranges;
    p.nslot = lay.nslot;
    p.part_o = part_o;
    p.part_ml = part_ml;
    p.o = (__nv_bfloat16*)a.o;
    p.lse = a.lse;
    p.status = a.status;
    cudaError_t e;
    if (lay.ctas) {
        if (lay.warps == 4)
            e = lay.ctas == 8   ? launch<4, 1, 8>(lay, map, p, st)
                : lay.ctas == 4 ? launch<4, 1, 4>(lay, map, p, st)
                : lay.ctas == 2 ? launch<4, 1, 2>(lay, map, p, st)
                                : launch<4, 1, 1>(lay, map, p, st);
        else
            e = lay.ctas == 8   ? launch<3, 1, 8>(lay, map, p, st)
                : lay.ctas == 4 ? launch<3, 1, 4>(lay, map, p, st)
                : lay.ctas == 2 ? launch<3, 1, 2>(lay, map, p, st)
                                : launch<3, 1, 1>(lay, map, p, st);
        if (e == cudaSuccess) count_launches(1);
        return e;
    }
    e = lay.warps == kRangeWarps ? launch<kRangeWarps, kRangeStages>(lay, map, p, st)
                                 : launch<kLongRangeWarps, kLongRangeStages>(lay, map, p, st);
    if (e != cudaSuccess) return e;
    count_launches(1);
    // (501 partials of a row: 13.5 us with eight groups, 14.8 with four; 34 partials: 12.0, 11.5)
    const int groups = lay.nslot > 128 ? 8 : lay.nslot > 8 ? 4 : 1;
    const auto combine = groups == 8   ? decode_q8_combine_kernel<8>
                         : groups == 4 ? decode_q8_combine_kernel<4>
                                       : decode_q8_combine_kernel<1>;
    e = launch_dependent(combine, dim3((unsigned)(a.N * a.Hq)), groups * kD, 0, st, part_o, part_ml, lay.nslot, a.Hq, a.Hkv, p.G,
                         a.K, lay.V, lay.ranges, (__nv_bfloat16*)a.o, a.lse);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace sas
