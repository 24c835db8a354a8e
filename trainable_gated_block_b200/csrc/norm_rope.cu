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
// lanes (head_row.cuh); the lanes of a row take up to four heads of one
// token, so that four rows' loads are in flight for each lane and the token's
// angles are read once for the four (the table rows are L1 hits for the
// token's other heads).
#include "head_row.cuh"
#include "launch.h"

namespace sas {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = kUnitHeads;

template <int D>
constexpr int kSlots = kThreads / HeadRow<D>::kLanes;      // row slots of a CTA

// Position of token row t; -1 (flagged) outside the table.
__device__ __forceinline__ int token_pos(const NormRopeArgs& a, long long t) {
    const int pos = a.positions != nullptr ? __ldg(a.positions + t) : (int)(t % a.S);
    if (pos < 0 || pos >= a.max_pos) {
        flag_status(a.status, kStatusBadData);
        return -1;
    }
    return pos;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const NormRopeArgs a, long long q_units, long long units, T* __restrict__ q_out, T* __restrict__ k_out) {
    const int l = threadIdx.x % HeadRow<D>::kLanes;
    long long u = (long long)blockIdx.x * kSlots<D> + threadIdx.x / HeadRow<D>::kLanes;
    const bool live = u < units, is_k = u >= q_units;
    if (is_k) u -= q_units;
    const int H = is_k ? a.Hkv : a.Hq, parts = unit_parts(H);
    const long long t = live ? u / parts : 0;
    const int h0 = (int)(u % parts);
    const T* src = static_cast<const T*>(is_k ? a.k : a.q) + t * (is_k ? a.ld_k : a.ld_q);
    T* dst = (is_k ? k_out : q_out) + t * H * D;
    const T* weight = static_cast<const T*>(is_k ? a.k_weight : a.q_weight);
    norm_rope_unit<T, D>(src, dst, H, h0, weight, a.table, a.eps, l, live, [&] { return token_pos(a, t); });
}

// Gradient. Each CTA walks its share of the query units, then of the key
// units, with the lane's 16 weight gradients in registers; the CTA's sums go
// to the workspace and norm_rope_dw_kernel adds them in CTA order, so that
// the result does not depend on timing.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
norm_rope_bwd_kernel(const NormRopeArgs a, const T* __restrict__ dq_out, const T* __restrict__ dk_out,
                     T* __restrict__ dq, T* __restrict__ dk, float* __restrict__ part) {
    __shared__ float acc[kSlots<D>][D];
    const int l = threadIdx.x % HeadRow<D>::kLanes, slot = threadIdx.x / HeadRow<D>::kLanes;
    for (int which = 0; which < 2; ++which) {
        const int H = which ? a.Hkv : a.Hq, parts = unit_parts(H);
        const long long units = a.T * parts, ld = which ? a.ld_k : a.ld_q;
        const T* src = static_cast<const T*>(which ? a.k : a.q);
        const T* up = which ? dk_out : dq_out;
        T* dst = which ? dk : dq;
        const T* weight = static_cast<const T*>(which ? a.k_weight : a.q_weight);
        float w[16], dw[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) dw[e] = 0.f;
        if (weight != nullptr) load_weight<T, D>(weight, l, w);
        for (long long base = (long long)blockIdx.x * kSlots<D>; base < units; base += (long long)gridDim.x * kSlots<D>) {
            const long long u = base + slot;
            const bool live = u < units;
            const long long t = live ? u / parts : 0;
            const int h0 = (int)(u % parts);
            Raw8<T> xl[kHeads], xh[kHeads], gl[kHeads], gh[kHeads];
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int h = h0 + i * parts;
                xl[i].zero(), xh[i].zero(), gl[i].zero(), gh[i].zero();
                if (live && h < H) {
                    const T* p = src + t * ld + h * D + 8 * l;
                    const T* g = up + (t * H + h) * D + 8 * l;
                    xl[i].load(p), xh[i].load(p + D / 2), gl[i].load(g), gh[i].load(g + D / 2);
                }
            }
            const int pos = live ? token_pos(a, t) : -1;
            Angles ang;
            ang.load<D>(a.table, max(pos, 0), l);
            float dwu[16];      // this unit's part: few terms are added before the long sum
#pragma unroll
            for (int e = 0; e < 16; ++e) dwu[e] = 0.f;
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int h = h0 + i * parts;
                float x[16], g[16];
                xl[i].get(x), xh[i].get(x + 8), gl[i].get(g), gh[i].get(g + 8);
                ang.turn_back(g);
                if (weight != nullptr) {
                    const float r = row_rrms<D>(x, a.eps);
                    float dot = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        x[e] *= r;
                        if (pos >= 0) dwu[e] = fmaf(g[e], x[e], dwu[e]);
                        g[e] *= w[e];
                        dot = fmaf(g[e], x[e], dot);
                    }
                    dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
                    for (int e = 0; e < 16; ++e) g[e] = r * fmaf(-x[e], dot, g[e]);
                }
                if (pos < 0) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) g[e] = 0.f;
                }
                if (live && h < H) {
                    T* p = dst + (t * H + h) * D + 8 * l;
                    store8(p, g);
                    store8(p + D / 2, g + 8);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) dw[e] += dwu[e];
        }
        if (weight == nullptr) continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[slot][8 * l + e] = dw[e];
            acc[slot][D / 2 + 8 * l + e] = dw[e + 8];
        }
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += kThreads) {
            float s = 0.f;
            for (int i = 0; i < kSlots<D>; ++i) s += acc[i][d];
            part[((long long)which * gridDim.x + blockIdx.x) * D + d] = s;
        }
    }
}

// dw[which][d] = sum of the CTAs' parts, in their order. One CTA for each weight.
template <int D>
__global__ void __launch_bounds__(1024)
norm_rope_dw_kernel(const float* __restrict__ part, int n, float* __restrict__ dwq, float* __restrict__ dwk) {
    __shared__ float acc[1024 / D][D];
    float* dst = blockIdx.x ? dwk : dwq;
    if (dst == nullptr) return;
    const int d = threadIdx.x % D, g = threadIdx.x / D;
    float s = 0.f;
    for (int i = g; i < n; i += 1024 / D) s += part[((long long)blockIdx.x * n + i) * D + d];
    acc[g][d] = s;
    __syncthreads();
    if (g) return;
    for (int i = 1; i < 1024 / D; ++i) s += acc[i][d];
    dst[d] = s;
}

long long units_of(long long T, int H) { return T * unit_parts(H); }

template <typename T, int D>
cudaError_t fwd(const NormRopeArgs& a, void* q_out, void* k_out, cudaStream_t st) {
    const long long uq = units_of(a.T, a.Hq), n = uq + units_of(a.T, a.Hkv);
    const long long grid = (n + kSlots<D> - 1) / kSlots<D>;
    norm_rope_kernel<T, D><<<(unsigned)grid, kThreads, 0, st>>>(a, uq, n, static_cast<T*>(q_out), static_cast<T*>(k_out));
    count_launches(1);
    return cudaGetLastError();
}

// CTAs of the gradient kernel: enough for every unit of the larger tensor, at most three for each SM.
int bwd_grid(long long T, int Hq, int Hkv, int D) {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    const long long slots = kThreads / (D / 16);
    const long long need = (units_of(T, Hq > Hkv ? Hq : Hkv) + slots - 1) / slots;
    return (int)(need < 1 ? 1 : need < 3LL * sms ? need : 3LL * sms);
}

template <typename T, int D>
cudaError_t bwd(const NormRopeArgs& a, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq,
                float* dwk, void* workspace, cudaStream_t st) {
    const int grid = bwd_grid(a.T, a.Hq, a.Hkv, D);
    float* part = static_cast<float*>(workspace);
    norm_rope_bwd_kernel<T, D><<<grid, kThreads, 0, st>>>(a, static_cast<const T*>(dq_out), static_cast<const T*>(dk_out),
                                                           static_cast<T*>(dq), static_cast<T*>(dk), part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (dwq == nullptr && dwk == nullptr) return cudaSuccess;
    norm_rope_dw_kernel<D><<<2, 1024, 0, st>>>(part, grid, dwq, dwk);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

size_t norm_rope_bwd_workspace(long long T, int Hq, int Hkv, int D) {
    return sizeof(float) * 2 * (size_t)bwd_grid(T, Hq, Hkv, D) * D;
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
