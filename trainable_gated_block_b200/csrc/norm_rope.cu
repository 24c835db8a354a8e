// sas_qk_norm_rope and its gradient: the per-head RMS norm of queries and keys
// with the position rotation in the same pass.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,  y = R(pos) n
//   R: (n_i, n_{i+D/2}) -> (n_i c_i - n_{i+D/2} s_i, n_{i+D/2} c_i + n_i s_i)
// and for an upstream gradient dy, with gn = R^T dy, g = gn w, h = x r:
//   dx = r (g - h mean(g h)),   dw = sum over tokens and heads of gn h
// (r is recomputed from x, so the forward saves nothing). All of it in fp32,
// rounded once to the tensors' type at the store.
//
// Both are bound by HBM: a row is read and written once. A row lives in D / 16
// lanes (head_row.cuh). A unit of work is a few heads of one token, which share
// the token's angles, for one row slot (the lanes of a row). CTAs are persistent
// and every thread prefetches its own 16-byte pieces of the next units into
// shared memory with cp.async.
//
// Measured on one B200 (heads of 128, bf16): forward of 8k and 32k tokens of 32/8 heads
// 29.9 and 107 us (89 and 99% of the copy rate), gradient of two 32k sequences of 40/8
// heads 386 us (97%).
#include <algorithm>

#include "dependent.cuh"
#include "head_row.cuh"
#include "launch.h"

namespace sas {
namespace {

// Position of token row t; -1 (flagged) outside the table.
__device__ __forceinline__ int token_pos(const NormRopeArgs& a, uint32_t t) {
    const int pos = a.positions != nullptr ? a.positions[t] : (int)(t % (uint32_t)a.S);
    if (pos < 0 || pos >= a.max_pos) {
        flag_status(a.status, kStatusBadData);
        return -1;
    }
    return pos;
}

// The same a unit ahead of its use where it has to be loaded, so that the angles' load
// does not wait for it (-1 behind the last unit; without positions any value).
template <typename Token>
__device__ __forceinline__ int pos_ahead(const NormRopeArgs& a, bool live, Token token) {
    return a.positions == nullptr ? 0 : live ? token_pos(a, token()) : -1;
}
__device__ __forceinline__ int unit_pos(const NormRopeArgs& a, bool live, uint32_t t, int ahead) {
    return a.positions != nullptr ? ahead : live ? token_pos(a, t) : -1;
}

// Shapes of the two kernels: threads, resident CTAs of an SM, units in flight,
// heads of a unit. fp32 rows are twice as long. (fp32 forward, 32k tokens of 32/8 heads
// of 128: 201 us, with six CTAs an SM and units of one head 232; bf16 106.8, with three
// CTAs 117.4, five and units of two heads 117.7.)
template <typename T, int D>
struct Fwd {
    static constexpr int kThreads = 128, kCtas = sizeof(T) == 2 ? 4 : 3, kStages = 2, kHeads = sizeof(T) == 2 ? 4 : 2;
    static constexpr int kSlots = kThreads / HeadRow<D>::kLanes;
    static constexpr int kPieces = kHeads * 2 * Raw8<T>::kPieces;      // 16-byte pieces of a thread and unit
    // so much that one more would not fit: CTAs that are placed while the kernel in front
    // still runs must not crowd on the SMs that are free first (8k tokens, one call after
    // the other: 30.5 us, without 32.5, without early launch 32.6)
    static constexpr int kSmem = 227 * 1024 / (kCtas + 1) / 16 * 16;
    static_assert(kSmem >= kStages * kPieces * kThreads * 16, "the ring");
};
template <typename T, int D>
struct Bwd {
    static constexpr int kThreads = sizeof(T) == 2 ? 256 : 128, kCtas = 2;
    static constexpr int kStages = 2, kHeads = 2;
    static constexpr int kSlots = kThreads / HeadRow<D>::kLanes;
    static constexpr int kPieces = kHeads * 4 * Raw8<T>::kPieces;      // of x and dy
    static constexpr int kRing = kStages * kPieces * kThreads * 16;
    static constexpr int kSmem = kRing > kSlots * D * 4 ? kRing : kSlots * D * 4;
};

// A token's units lie one after the other, its queries' and its keys', so that the
// CTAs that run together read whole rows of a fused projection (all queries' units
// first, then the keys': 112.3 instead of 106.7 us for 32k tokens).
template <typename T, int D>
__global__ void __launch_bounds__(Fwd<T, D>::kThreads, Fwd<T, D>::kCtas)
norm_rope_kernel(const NormRopeArgs a, uint32_t units, T* q_out, T* k_out) {
    using S = Fwd<T, D>;
    constexpr int kRow = 2 * Raw8<T>::kPieces * S::kThreads * 16, kStage = S::kHeads * kRow;    // bytes from row to row, stage to stage
    extern __shared__ __align__(16) uint8_t smem[];
    after_previous();
    const uint32_t ring = sm100::smem_u32(smem) + threadIdx.x * 16;
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    const uint32_t first = blockIdx.x * S::kSlots + threadIdx.x / HeadRow<D>::kLanes, step = gridDim.x * S::kSlots;
    const uint32_t parts_q = parts_of(a.Hq, S::kHeads), parts_k = parts_of(a.Hkv, S::kHeads), per = parts_q + parts_k;

    auto issue = [&](uint32_t u, uint32_t st) {
        if (u < units) {
            const uint32_t t = u / per, j = u - t * per;
            const bool is_k = j >= parts_q;
            const int H = is_k ? a.Hkv : a.Hq, parts = (int)(is_k ? parts_k : parts_q), h0 = (int)(is_k ? j - parts_q : j);
            const T* src = static_cast<const T*>(is_k ? a.k : a.q) + (long long)t * (is_k ? a.ld_k : a.ld_q);
#pragma unroll
            for (int i = 0; i < S::kHeads; ++i) {
                const int h = h0 + i * parts;
                copy_row<T, D, S::kThreads>(ring + st * kStage + i * kRow, src + (h < H ? h : 0) * D, l, h < H);
            }
        }
        copy_commit();
    };

    uint32_t next = first, st = 0;
#pragma unroll
    for (int s = 0; s < S::kStages; ++s, next += step) issue(next, s);
    int ahead = pos_ahead(a, first < units, [&] { return first / per; });
    // (no sum here passes 2^32: units is below 2^31)
    for (uint32_t base = blockIdx.x * S::kSlots, u = first; base < units; base += step, u += step) {
        const bool live = u < units;
        const uint32_t t = live ? u / per : 0, j = live ? u - t * per : 0;
        const bool is_k = j >= parts_q;
        const int H = is_k ? a.Hkv : a.Hq, parts = (int)(is_k ? parts_k : parts_q), h0 = (int)(is_k ? j - parts_q : j);
        const T* weight = static_cast<const T*>(is_k ? a.k_weight : a.q_weight);
        const int pos = unit_pos(a, live, t, ahead);
        const Turn turn(load_angles<T, D>(a.table, max(pos, 0), l), load_weight<T, D>(weight, l));
        ahead = pos_ahead(a, u + step < units, [&] { return (u + step) / per; });
        T* dst = (is_k ? k_out : q_out) + (long long)t * H * D;
        copy_wait<S::kStages - 1>();
#pragma unroll
        for (int i = 0; i < S::kHeads; ++i) {
            const int h = h0 + i * parts;
            const Row x = read_row<T, S::kThreads>(ring + st * kStage + i * kRow);
            Row y = turn(x, weight != nullptr ? row_rrms<D>(x, a.eps) : 1.f);
            if (pos < 0) y = Row{};
            if (live && h < H) store_row<D>(dst + h * D, l, y);
        }
        issue(next, st);        // behind the uses of what this stage held
        next = next < units ? next + step : next;
        st = st + 1 == S::kStages ? 0 : st + 1;
    }
}

// fp32 sums of a lane's 16 values, kept in T's layout, to a row of D.
template <typename T, int D>
__device__ __forceinline__ void store_sums(float* p, int l, const Row& r) {
    constexpr int kSecond = sizeof(T) == 2 ? 4 : D / 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Half& h = i ? r.b : r.a;
        float* q = p + i * (D / 2) + Raw8<T>::kStep * l;
        *reinterpret_cast<ulonglong2*>(q) = make_ulonglong2(h.v[0], h.v[1]);
        *reinterpret_cast<ulonglong2*>(q + kSecond) = make_ulonglong2(h.v[2], h.v[3]);
    }
}

// Gradient. With q_ctas the first q_ctas CTAs walk the query units, the others
// the key units; without, every CTA its share of the query units, then of the
// key units. The lane's 16 weight gradients stay in registers; a CTA's sums go
// to the workspace and norm_rope_dw_kernel adds them in CTA order, so that
// the result does not depend on timing.
template <typename T, int D>
__global__ void __launch_bounds__(Bwd<T, D>::kThreads, Bwd<T, D>::kCtas)
norm_rope_bwd_kernel(const NormRopeArgs a, const T* dq_out, const T* dk_out, T* dq, T* dk, float* part,
                     unsigned q_ctas) {
    using S = Bwd<T, D>;
    constexpr int kRow = 2 * Raw8<T>::kPieces * S::kThreads * 16;
    extern __shared__ __align__(16) uint8_t smem[];
    after_previous();
    const uint32_t ring = sm100::smem_u32(smem) + threadIdx.x * 16;
    const int l = threadIdx.x % HeadRow<D>::kLanes, slot = threadIdx.x / HeadRow<D>::kLanes;
    const bool both = q_ctas == 0;
    for (int which = !both && blockIdx.x >= q_ctas; which < 2; ++which) {
        const uint32_t cta = !both && which ? blockIdx.x - q_ctas : blockIdx.x;
        const uint32_t ctas = both ? gridDim.x : which ? gridDim.x - q_ctas : q_ctas;
        const uint32_t first = cta * S::kSlots + slot, step = ctas * S::kSlots;
        const int H = which ? a.Hkv : a.Hq;
        const uint32_t parts = parts_of(H, S::kHeads), units = (uint32_t)a.T * parts;
        const long long ld = which ? a.ld_k : a.ld_q;
        const T* src = static_cast<const T*>(which ? a.k : a.q);
        const T* up = which ? dk_out : dq_out;
        T* out = which ? dk : dq;
        const T* weight = static_cast<const T*>(which ? a.k_weight : a.q_weight);
        const Row w = load_weight<T, D>(weight, l);

        auto issue = [&](uint32_t u, uint32_t st) {
            if (u < units) {
                const uint32_t t = u / parts;
                const uint32_t at = ring + st * (S::kPieces * S::kThreads * 16);
#pragma unroll
                for (int i = 0; i < S::kHeads; ++i) {
                    const int h = (int)(u - t * parts + i * parts);
                    const int hs = h < H ? h : 0;
                    copy_row<T, D, S::kThreads>(at + 2 * i * kRow, src + (long long)t * ld + hs * D, l, h < H);
                    copy_row<T, D, S::kThreads>(at + (2 * i + 1) * kRow, up + ((long long)t * H + hs) * D, l, h < H);
                }
            }
            copy_commit();
        };

        Row dw{};
        uint32_t next = first, st = 0;
#pragma unroll
        for (int s = 0; s < S::kStages; ++s, next += step) issue(next, s);
        int ahead = pos_ahead(a, first < units, [&] { return first / parts; });
        for (uint32_t base = cta * S::kSlots, u = first; base < units; base += step, u += step) {
            const bool live = u < units;
            const uint32_t t = live ? u / parts : 0;
            const int pos = unit_pos(a, live, t, ahead);
            const Angles ang = load_angles<T, D>(a.table, max(pos, 0), l);
            ahead = pos_ahead(a, u + step < units, [&] { return (u + step) / parts; });
            copy_wait<S::kStages - 1>();
            const uint32_t at = ring + st * (S::kPieces * S::kThreads * 16);
            Row dwu{};          // this unit's part: few terms are added before the long sum
#pragma unroll
            for (int i = 0; i < S::kHeads; ++i) {
                const int h = (int)(u - t * parts + i * parts);
                Row x = read_row<T, S::kThreads>(at + 2 * i * kRow), g;
                const Row dy = read_row<T, S::kThreads>(at + (2 * i + 1) * kRow);
                const f2 neg = f2_pack(-1.f, -1.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g.a.v[e] = f2_fma(dy.a.v[e], ang.c.v[e], f2_mul(dy.b.v[e], ang.s.v[e]));
                    g.b.v[e] = f2_fma(dy.b.v[e], ang.c.v[e], f2_mul(f2_mul(dy.a.v[e], ang.s.v[e]), neg));
                }
                if (weight != nullptr) {
                    const float r = row_rrms<D>(x, a.eps);
                    const f2 rr = f2_pack(r, r);
                    const bool add = pos >= 0 && live && h < H;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x.a.v[e] = f2_mul(x.a.v[e], rr);
                        x.b.v[e] = f2_mul(x.b.v[e], rr);
                        if (add) {
                            dwu.a.v[e] = f2_fma(g.a.v[e], x.a.v[e], dwu.a.v[e]);
                            dwu.b.v[e] = f2_fma(g.b.v[e], x.b.v[e], dwu.b.v[e]);
                        }
                        g.a.v[e] = f2_mul(g.a.v[e], w.a.v[e]);
                        g.b.v[e] = f2_mul(g.b.v[e], w.b.v[e]);
                    }
                    const float m = -row_dot<D>(g, x) * (1.f / D);
                    const f2 mm = f2_pack(m, m);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g.a.v[e] = f2_mul(rr, f2_fma(x.a.v[e], mm, g.a.v[e]));
                        g.b.v[e] = f2_mul(rr, f2_fma(x.b.v[e], mm, g.b.v[e]));
                    }
                }
                if (pos < 0) g = Row{};
                if (live && h < H) store_row<D>(out + ((long long)t * H + h) * D, l, g);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dw.a.v[e] = f2_add(dw.a.v[e], dwu.a.v[e]);
                dw.b.v[e] = f2_add(dw.b.v[e], dwu.b.v[e]);
            }
            issue(next, st);    // behind the uses of what this stage held
            next = next < units ? next + step : next;
            st = st + 1 == S::kStages ? 0 : st + 1;
        }
        copy_wait<0>();
        if (weight != nullptr) {
            // the ring is empty: the slots' sums take its place
            float* acc = reinterpret_cast<float*>(smem);
            __syncthreads();
            store_sums<T, D>(acc + slot * D, l, dw);
            __syncthreads();
            for (int d = threadIdx.x; d < D; d += S::kThreads) {
                float s = 0.f;
                for (int i = 0; i < S::kSlots; ++i) s += acc[i * D + d];
                part[((long long)(both ? which * gridDim.x : 0) + blockIdx.x) * D + d] = s;
            }
            __syncthreads();
        }
        if (!both) return;
    }
}

// dw[d] = sum of the CTAs' parts, in a fixed order: 32 columns for each CTA, whose
// 32 rows of threads take every 32nd part. The first D / 32 CTAs add the query parts.
template <int D>
__global__ void __launch_bounds__(1024)
norm_rope_dw_kernel(const float* part, int q_ctas, int ctas, float* dwq, float* dwk) {
    __shared__ float acc[32][32];
    after_previous();
    const bool is_k = blockIdx.x >= D / 32;
    const int d = (int)(blockIdx.x % (D / 32)) * 32 + threadIdx.x % 32, g = threadIdx.x / 32;
    const int lo = is_k ? q_ctas : 0, hi = is_k ? ctas : q_ctas;
    float s = 0.f;
#pragma unroll 4
    for (int i = lo + g; i < hi; i += 32) s += part[(long long)i * D + d];
    acc[g][threadIdx.x % 32] = s;
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) s += acc[i][threadIdx.x];
    (is_k ? dwk : dwq)[d] = s;
}

int sm_count() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    return sms;
}

// CTAs for `units` units: all of them, or as many as are resident together.
unsigned grid_for(long long units, int slots, int ctas) {
    const long long need = (units + slots - 1) / slots, most = (long long)ctas * sm_count();
    return (unsigned)(need < 1 ? 1 : need < most ? need : most);
}

template <typename T, int D>
cudaError_t fwd(const NormRopeArgs& a, void* q_out, void* k_out, cudaStream_t st) {
    using S = Fwd<T, D>;
    const uint32_t n = (uint32_t)a.T * (parts_of(a.Hq, S::kHeads) + parts_of(a.Hkv, S::kHeads));
    cudaError_t e = cudaFuncSetAttribute(norm_rope_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(norm_rope_kernel<T, D>, dim3(grid_for(n, S::kSlots, S::kCtas)), S::kThreads, S::kSmem, st, a, n,
                                static_cast<T*>(q_out), static_cast<T*>(k_out));
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// CTAs of the gradient kernel. Up to kSplitWaves units for each resident row slot,
// query and key units have CTAs of their own, in proportion, which saves the
// latency of one after the other; beyond, each CTA does first query, then key
// units. Measured, apart / together: 2,291 tokens of 8/2 heads of 64 in fp32 7.0 /
// 9.1 us; 2,000 tokens of 40/8 heads of 128 in bf16 (5 waves) 18.4 / 19.6;
// 8,000 (20 waves) 56.0 / 56.0; 65,536 (166 waves) 403 / 385.
constexpr int kSplitWaves = 8;

struct Split {
    unsigned q, grid, q_parts, parts;       // q: 0 where every CTA does both
};
template <typename T, int D>
Split bwd_split(long long tokens, int Hq, int Hkv) {
    using S = Bwd<T, D>;
    const long long uq = tokens * parts_of(Hq, S::kHeads), uk = tokens * parts_of(Hkv, S::kHeads);
    const long long nq = std::max(1LL, (uq + S::kSlots - 1) / S::kSlots), nk = std::max(1LL, (uk + S::kSlots - 1) / S::kSlots);
    const long long most = (long long)S::kCtas * sm_count();
    if (nq + nk > kSplitWaves * most) {
        const unsigned g = (unsigned)std::min(most, std::max(nq, nk));
        return {0, g, g, 2 * g};
    }
    long long q = nq, all = nq + nk;
    if (all > most) {
        q = most - std::min(most - 1, std::max(1LL, (most * uk + (uq + uk) / 2) / (uq + uk)));
        all = most;
    }
    return {(unsigned)q, (unsigned)all, (unsigned)q, (unsigned)all};
}

template <typename T, int D>
cudaError_t bwd(const NormRopeArgs& a, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq,
                float* dwk, void* workspace, cudaStream_t st) {
    using S = Bwd<T, D>;
    const Split grid = bwd_split<T, D>(a.T, a.Hq, a.Hkv);
    float* part = static_cast<float*>(workspace);
    cudaError_t e = cudaFuncSetAttribute(norm_rope_bwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_dependent<false>(norm_rope_bwd_kernel<T, D>, dim3(grid.grid), S::kThreads, S::kSmem, st, a, static_cast<const T*>(dq_out),
                         static_cast<const T*>(dk_out), static_cast<T*>(dq), static_cast<T*>(dk), part, grid.q);
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (dwq == nullptr) return cudaSuccess;
    e = launch_dependent(norm_rope_dw_kernel<D>, dim3(2 * (D / 32)), 1024, 0, st, part, (int)grid.q_parts, (int)grid.parts, dwq,
                         dwk);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

size_t norm_rope_bwd_workspace(long long T, int Hq, int Hkv, int D) {
    // the types' kernels have different units: the larger number of parts
    const unsigned g =
        D == 128 ? std::max(bwd_split<float, 128>(T, Hq, Hkv).parts, bwd_split<__nv_bfloat16, 128>(T, Hq, Hkv).parts)
                 : std::max(bwd_split<float, 64>(T, Hq, Hkv).parts, bwd_split<__nv_bfloat16, 64>(T, Hq, Hkv).parts);
    return sizeof(float) * (size_t)g * D;
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool bf16, int D, void* q_out, void* k_out, cudaStream_t st) {
    if (bf16) return D == 128 ? fwd<__nv_bfloat16, 128>(a, q_out, k_out, st) : fwd<__nv_bfloat16, 64>(a, q_out, k_out, st);
    return D == 128 ? fwd<float, 128>(a, q_out, k_out, st) : fwd<float, 64>(a, q_out, k_out, st);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, bool bf16, int D, const void* dq_out, const void* dk_out, void* dq,
                                 void* dk, float* dwq, float* dwk, void* workspace, cudaStream_t st) {
    if (bf16)
        return D == 128 ? bwd<__nv_bfloat16, 128>(a, dq_out, dk_out, dq, dk, dwq, dwk, workspace, st)
                        : bwd<__nv_bfloat16, 64>(a, dq_out, dk_out, dq, dk, dwq, dwk, workspace, st);
    return D == 128 ? bwd<float, 128>(a, dq_out, dk_out, dq, dk, dwq, dwk, workspace, st)
                    : bwd<float, 64>(a, dq_out, dk_out, dq, dk, dwq, dwk, workspace, st);
}

}  // namespace sas
