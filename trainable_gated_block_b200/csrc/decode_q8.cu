// sas_decode_paged_q8: the gated decode step of decode.cu over 8-bit pages.
//
// Pages hold e4m3 codes with one scale for K and one for V for each (page, KV
// head): key = ks kc, value = vs vc. With gate g of a kept block (0 for the
// current one) and x = sm_scale ks (q . kc) + g,
//   o = sum_j e^(x_j - m) vs_j vc_j / sum_j e^(x_j - m),  lse = m + log(sum_j e^(x_j - m)).
// The value scale goes into the exponent: with y = x log2(e) + log2(vs) and m the
// running maximum of y, w = 2^(y - m) <= 1 is the weight of the code itself, so
// that the value codes need no multiplication, and the softmax sum takes w / vs.
// Codes are exact in fp16, the queries are scaled by a power of two (their
// largest element to 2^13 .. 2^14, what falls out of fp16 below is under 2^-30 of
// it), the weights are rounded to fp16 (2^-11 relative); logits, sums and
// accumulators are fp32.
//
// HBM-bound, split as in decode_split.cuh: one persistent CTA per SM streams
// its share of the kept (page, KV head) tiles, 8 KiB of K and 8 KiB of V, by
// TMA into a ring of twelve stages. Consumer warp w takes every fourth
// block and does it whole on mma.sync m16n8k16 with keys (or value dimensions) as
// the 16 rows and the up to 8 query heads of the group as the 8 columns:
//   S^T = K Q^T : A from ldmatrix over byte pairs. A lane gets four neighbouring
//       dimensions of a key; the first two serve as the lane's low k pair, the
//       others as its high pair, and Q is loaded in the same order.
//   O^T = V^T P^T : A from ldmatrix.trans over byte pairs, which are two
//       neighbouring dimensions of a key: the even ones become rows 0..7 of the
//       tile, the odd ones rows 8..15. P^T comes from S^T by movmatrix.
#include <cuda_fp16.h>

#include "byte_map.h"
#include "common.cuh"
#include "decode_split.cuh"
#include "launch.h"
#include "page_rows.h"
#include "sm100.cuh"

namespace sas {
namespace {

using namespace sm100;

constexpr int kWarps = 4;                          // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;        // + one producer warp
constexpr int kStages = 3 * kWarps;                // warp w owns stages w, w + kWarps, w + 2 kWarps
constexpr uint32_t kTileBytes = 64 * 128;          // one (page, head) tile of K or V: 64 rows of 128 codes
constexpr int kShortRows = 8;                      // short box (one 128-byte swizzle period) for a partial block
constexpr uint32_t kShortBytes = kShortRows * 128;
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kOffMo = kStages * kStageBytes;                 // merge scratch: o [warp][8][D]
constexpr uint32_t kOffMl = kOffMo + kWarps * 8 * kD * 4;          // merge scratch: m, l [warp][8][2]
constexpr uint32_t kOffMeta = kOffMl + kWarps * 8 * 2 * 4;         // per stage: bias, valid keys, ks, 1 / vs
constexpr uint32_t kOffBar = kOffMeta + kStages * 16;
constexpr uint32_t kSmem = kOffBar + 2 * kStages * 8 + 16 + 1024;  // + alignment slack
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");

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
    int grid;
    int nslot;              // partial slots per query head
    float* part_o;          // [N * Hq, nslot, D]
    float* part_ml;         // [N * Hq, nslot, 2]
    int* status;
};

struct ItemInfo {
    int n, h, L, c, n_sel;
    bool ok;
};
__device__ __forceinline__ ItemInfo item_info(const Params& p, int item, bool flag) {
    ItemInfo r;
    r.n = item / p.Hkv;
    r.h = item % p.Hkv;
    r.L = p.kv_len[r.n];
    r.ok = r.L >= 1 && r.L <= (long long)p.max_pages * kBlock;
    r.c = r.ok ? (r.L - 1) / kBlock : 0;
    r.n_sel = 0;
    if (!r.ok) {
        if (r.L != 0 && flag) flag_status(p.status, kStatusBadData);     // 0: a padding entry
        return r;
    }
    const int n_sel = p.cnt[item], hi = min(p.K, r.c);
    r.n_sel = max(0, min(n_sel, hi));
    if (r.n_sel != n_sel && flag) flag_status(p.status, kStatusBadData);
    return r;
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
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

__global__ void __launch_bounds__(kThreads, 1)
decode_q8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_k8, const __grid_constant__ CUtensorMap map_v8, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* mo = reinterpret_cast<float*>(smem + kOffMo);
    float* ml = reinterpret_cast<float*>(smem + kOffMl);
    float4* meta = reinterpret_cast<float4*>(smem + kOffMeta);   // bias (log2 units), valid keys, ks, 1 / vs
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* empty = full + kStages;
    int* abort_flag = reinterpret_cast<int*>(empty + kStages);
    volatile int* abort = abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();

    const long long v0 = slot_begin(blockIdx.x, p.V, p.grid), v1 = slot_begin(blockIdx.x + 1, p.V, p.grid);
    const int Kp1 = p.K + 1;
    // the combine kernel may be scheduled now (it waits for this grid to finish)
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");

    if (warp == kWarps) {
        // ----------------------------------------------------------- producer
        // The 32 lanes resolve 32 block slots at a time (selection entry, page,
        // gate, scales: dependent loads, done in parallel); lane 0 then issues
        // the copies of the kept ones in slot order. The next batch is resolved
        // once the ring is full, while its copies are in flight.
        if (lane == 0) {
            prefetch_tensormap(&map_k);
            prefetch_tensormap(&map_v);
            prefetch_tensormap(&map_k8);
            prefetch_tensormap(&map_v8);
        }
        struct Slot {
            bool use;
            int row0;
            float4 m;
        };
        auto resolve = [&](long long base) {
            const long long v = base + lane;
            Slot s{false, -1, make_float4(0.f, 0.f, 1.f, 1.f)};
            if (v < v1) {
                const int item = (int)(v / Kp1), t = (int)(v % Kp1);
                const ItemInfo inf = item_info(p, item, true);
                if (inf.ok && t <= inf.n_sel) {
                    s.use = true;
                    const bool cur = (t == inf.n_sel);
                    const long long srow = (long long)item * p.K + t;
                    const int j = cur ? inf.c : p.idx[srow];
                    int page = -1;
                    if (j >= 0 && (cur || j < inf.c))
                        page = p.page_table[(long long)inf.n * p.max_pages + j];   // j < max_pages by kv_len's check
                    bool ok = page >= 0 && page < p.num_pages;
                    if (ok) {
                        const float ks = __ldg(p.k_scale + (long long)page * p.Hkv + inf.h);
                        const float vs = __ldg(p.v_scale + (long long)page * p.Hkv + inf.h);
                        ok = scale_ok(ks) && scale_ok(vs);
                        s.m.x = (cur ? 0.f : p.log_gate[srow] * kLog2e) + log2f(vs);
                        s.m.z = ks;
                        s.m.w = 1.f / vs;
                    }
                    if (!ok) flag_status(p.status, kStatusBadData);
                    s.m.y = ok ? (float)(cur ? inf.L - inf.c * kBlock : kBlock) : 0.f;
                    s.row0 = ok ? (page * p.Hkv + inf.h) * kBlock : -1;   // < 2^31 (checked on the host)
                }
            }
            return s;
        };
        uint32_t it = 0;
        bool ok_run = true;
        Slot cur = resolve(v0);
        for (long long base = v0; base < v1 && ok_run; base += 32) {
            const bool more = base + 32 < v1;
            Slot nxt{false, -1, make_float4(0.f, 0.f, 1.f, 1.f)};
            bool resolved = !more;
            int issued = 0;
            unsigned todo = __ballot_sync(0xffffffffu, cur.use);
            while (todo) {
                const int b = __ffs(todo) - 1;
                todo &= todo - 1;
                const int rb = __shfl_sync(0xffffffffu, cur.row0, b);
                float4 mb;
                mb.x = __shfl_sync(0xffffffffu, cur.m.x, b);
                mb.y = __shfl_sync(0xffffffffu, cur.m.y, b);
                mb.z = __shfl_sync(0xffffffffu, cur.m.z, b);
                mb.w = __shfl_sync(0xffffffffu, cur.m.w, b);
                if (lane == 0) {
                    const int st = it % kStages;
                    if (!mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1, abort, p.status)) {
                        ok_run = false;
                    } else {
                        meta[st] = mb;
                        uint8_t* dst = smem + st * kStageBytes;
                        const int nv = (int)mb.y;
                        if (rb >= 0 && nv < kBlock) {
                            // partial block (the current one): only the 8-row groups holding tokens
                            const int ng = (nv + kShortRows - 1) / kShortRows;
                            mbar_expect_tx(&full[st], (uint32_t)ng * 2 * kShortBytes);
                            for (int g8 = 0; g8 < ng; ++g8) {
                                tma_load_3d(dst + g8 * kShortBytes, &map_k8, &full[st], 0, 0, rb + g8 * kShortRows);
                                tma_load_3d(dst + kTileBytes + g8 * kShortBytes, &map_v8, &full[st], 0, 0,
                                            rb + g8 * kShortRows);
                            }
                        } else if (rb >= 0) {
                            mbar_expect_tx(&full[st], kStageBytes);
                            tma_load_3d(dst, &map_k, &full[st], 0, 0, rb);
                            tma_load_3d(dst + kTileBytes, &map_v, &full[st], 0, 0, rb);
                        } else {
                            mbar_arrive(&full[st]);
                        }
                        ++it;
                    }
                }
                ok_run = __shfl_sync(0xffffffffu, ok_run, 0);
                if (!ok_run) break;
                if (!resolved && ++issued == kStages) {
                    nxt = resolve(base + 32);
                    resolved = true;
                }
            }
            if (!resolved) nxt = resolve(base + 32);
            cur = nxt;
        }
        if (lane == 0 && *abort) {       // let the copies in flight land before the CTA exits
            volatile int no_abort = 0;
            const uint32_t lo = it > (uint32_t)kStages ? it - kStages : 0;
            for (uint32_t k = lo; k < it; ++k) mbar_wait(&full[k % kStages], (k / kStages) & 1, &no_abort, nullptr);
        }
        return;   // the producer takes no part in the consumers' named barrier
    }

    // -------------------------------------------------------------- consumers
    const int grp = lane >> 2, tig = lane & 3;     // mma fragment coordinates
    const uint32_t s_base = smem_u32(smem);
    const int lrow = (lane & 7) + (lane & 8);      // ldmatrix: key of this lane's row within 16, and chunk of two
    const int lchk = lane >> 4;
    uint32_t qb[8][2];          // Q^T as B fragments: 8 k-steps x (dims 4tig, +1 / +2, +3 of the step) of head grp
    float o[8][4];              // O^T: tile mt, dims 16mt + 2grp (+1 in [2], [3]) x heads 2tig, 2tig + 1
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};     // heads 2tig, 2tig + 1: max of y; this lane's part of the sum
    float qm[2] = {0.f, 0.f};   // sm_scale log2(e) over the query scale of those heads
    uint32_t blk = 0;           // blocks of this CTA's stream seen so far
    int cur_item = -1;
    ItemInfo inf{};
    bool dead = false;

    auto flush = [&]() {
        // sum over the lanes that share a head, then every warp's state to shared memory
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
            if (l[e] != l[e]) m[e] = fmaxf(m[e], -1e30f);     // only NaN logits: the row is not an empty one
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2*>(mo + (warp * 8 + 2 * tig + e) * kD + 16 * mt + 2 * grp) =
                    make_float2(o[mt][e], o[mt][2 + e]);
        if (grp == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ml[(warp * 8 + 2 * tig + e) * 2] = m[e];
                ml[(warp * 8 + 2 * tig + e) * 2 + 1] = l[e];
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        const int slot = (int)blockIdx.x - cta_of((long long)cur_item * Kp1, p.V, p.grid);
        for (int e = threadIdx.x; e < p.G * kD; e += kWarps * 32) {
            const int g = e / kD, d = e % kD;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[(w * 8 + g) * 2]);
            float acc = 0.f, L = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float mw = ml[(w * 8 + g) * 2];
                    const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
                    acc = fmaf(mo[(w * 8 + g) * kD + d], f, acc);
                    L = fmaf(ml[(w * 8 + g) * 2 + 1], f, L);
                }
            }
            const long long row = ((long long)inf.n * p.Hq + inf.h * p.G + g) * p.nslot + slot;
            p.part_o[row * kD + d] = acc;
            if (d == 0) {
                p.part_ml[row * 2] = M;
                p.part_ml[row * 2 + 1] = L;
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    };

    for (long long v = v0; v < v1; ++v) {
        const int item = (int)(v / Kp1), t = (int)(v % Kp1);
        if (item != cur_item) {
            if (cur_item >= 0) flush();
            cur_item = item;
            inf = item_info(p, item, false);
            const bool real = grp < p.G;
            const uint2* qrow = reinterpret_cast<const uint2*>(
                p.q + ((long long)inf.n * p.Hq + inf.h * p.G + (real ? grp : 0)) * kD);
            uint2 qr[8];
            float top = 0.f;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                qr[kk] = real ? __ldg(qrow + 4 * kk + tig) : make_uint2(0u, 0u);
                const float2 a = bf16x2_to_f32(qr[kk].x), b = bf16x2_to_f32(qr[kk].y);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^e with top 2^e in [2^13, 2^14); 1 for a zero or infinite row
            const int te = (int)(__float_as_uint(top) >> 23);           // biased exponent of top
            const int e = te == 0 || te == 255 ? 0 : min(13 + 127 - te, 126);
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
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.f;
        }
        if (!inf.ok || t > inf.n_sel) continue;
        const uint32_t b = blk++;
        if (b % kWarps != (uint32_t)warp || dead) continue;      // another warp's block
        const int st = b % kStages;
        if (!mbar_wait_warp(&full[st], (b / kStages) & 1, abort, p.status)) {
            dead = true;              // keep walking the slots so the flush barriers still meet
            continue;
        }
        const float4 md = meta[st];
        const int nvalid = (int)md.y;
        if (nvalid > 0) {
            const uint32_t kt = s_base + st * kStageBytes, vt = kt + kTileBytes;
            float s[4][4];      // S^T: keys 16mt + grp (+8 in [2], [3]) x heads 2tig, 2tig + 1
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < 8; kk += 2) {
                    uint32_t r[4], a0, a1, a2, a3;
                    ldsm_x4(kt + sw128_offset(16 * mt + lrow, kk + lchk), r);
                    codes_f16(r[0], a0, a2);
                    codes_f16(r[1], a1, a3);
                    mma16816(s[mt], a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
                    codes_f16(r[2], a0, a2);
                    codes_f16(r[3], a1, a3);
                    mma16816(s[mt], a0, a1, a2, a3, qb[kk + 1][0], qb[kk + 1][1]);
                }
            }
            float bm[2] = {-INFINITY, -INFINITY};
            const float f[2] = {qm[0] * md.z, qm[1] * md.z};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 16 * mt + grp + 8 * (e >> 1);
                    const float y = key < nvalid ? fmaf(s[mt][e], f[e & 1], md.x) : -INFINITY;
                    s[mt][e] = y;
                    bm[e & 1] = fmaxf(bm[e & 1], y);
                }
            float sc[2], ls[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) bm[e] = fmaxf(bm[e], __shfl_xor_sync(0xffffffffu, bm[e], x));
                const float mn = fmaxf(m[e], bm[e]);
                sc[e] = mn == -INFINITY ? 1.f : exp2f(m[e] - mn);
                m[e] = mn;
            }
            uint32_t pb[4][2];          // P^T as B fragments
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[mt][e] = s[mt][e] == -INFINITY ? 0.f : exp2f(s[mt][e] - m[e & 1]);
                    ls[e & 1] += s[mt][e];
                }
                pb[mt][0] = transpose8x8(pack_f16x2(s[mt][0], s[mt][1]));
                pb[mt][1] = transpose8x8(pack_f16x2(s[mt][2], s[mt][3]));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) l[e] = fmaf(l[e], sc[e], ls[e] * md.w);
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][e] *= sc[e & 1];
            if (nvalid < kBlock) {
                // rows past the sequence end (the current block) are zeroed: their weight
                // is 0, but whatever the page holds there must not reach O as 0 * NaN
                uint8_t* vrow = smem + st * kStageBytes + kTileBytes;
                for (int e = nvalid * 8 + lane; e < kBlock * 8; e += 32)
                    *reinterpret_cast<uint4*>(vrow + sw128_offset(e >> 3, e & 7)) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();     // ordered before the stage's next TMA refill
                __syncwarp();
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int mt = 0; mt < 8; mt += 2) {
                    uint32_t r[4], a0, a1, a2, a3;
                    ldsm_x4_t(vt + sw128_offset(16 * kk + lrow, mt + lchk), r);
                    codes_f16(__byte_perm(r[0], 0u, 0x3120), a0, a1);
                    codes_f16(__byte_perm(r[1], 0u, 0x3120), a2, a3);
                    mma16816(o[mt], a0, a1, a2, a3, pb[kk][0], pb[kk][1]);
                    codes_f16(__byte_perm(r[2], 0u, 0x3120), a0, a1);
                    codes_f16(__byte_perm(r[3], 0u, 0x3120), a2, a3);
                    mma16816(o[mt + 1], a0, a1, a2, a3, pb[kk][0], pb[kk][1]);
                }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
    }
    if (cur_item >= 0) flush();
}

}  // namespace

size_t decode_q8_workspace(int N, int Hq, int Hkv, int K) {
    const Layout lay = layout(N, Hkv, K);
    const size_t per = (size_t)N * Hq * lay.nslot;
    return sizeof(float) * (per * kD + per * 2);
}

cudaError_t launch_decode_q8(const DecodeArgs& a, const float* k_scale, const float* v_scale, void* workspace,
                             cudaStream_t st) {
    const long long cache_rows = (long long)a.num_pages * a.Hkv * kBlock;
    const Layout lay = layout(a.N, a.Hkv, a.K);
    float* part_o = static_cast<float*>(workspace);
    float* part_ml = part_o + (size_t)a.N * a.Hq * lay.nslot * kD;
    CUtensorMap mk, mv, mk8, mv8;
    if (!make_byte_map(&mk, a.k_cache, cache_rows, kBlock) || !make_byte_map(&mv, a.v_cache, cache_rows, kBlock) ||
        !make_byte_map(&mk8, a.k_cache, cache_rows, kShortRows) || !make_byte_map(&mv8, a.v_cache, cache_rows, kShortRows))
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
    p.grid = lay.grid;
    p.nslot = lay.nslot;
    p.part_o = part_o;
    p.part_ml = part_ml;
    p.status = a.status;
    cudaError_t e = cudaFuncSetAttribute(decode_q8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    decode_q8_kernel<<<lay.grid, kThreads, kSmem, st>>>(mk, mv, mk8, mv8, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // programmatic dependent launch: the combine's blocks are placed while the decode grid drains
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.N * a.Hq));
    cfg.blockDim = dim3(kD);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, decode_combine_kernel, (const float*)part_o, (const float*)part_ml, lay.nslot, a.Hq,
                           a.Hkv, p.G, a.K, lay.V, lay.grid, (__nv_bfloat16*)a.o, a.lse, 0.f);
    if (e != cudaSuccess) return e;
    count_launches(2);
    return cudaGetLastError();
}

}  // namespace sas
