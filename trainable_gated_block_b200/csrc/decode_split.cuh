// How the paged decode kernels split their work over CTAs, and the kernel that
// joins the parts.
//
// A work item is (sequence n, KV head h) with K + 1 block slots (the kept
// blocks, then the current one); the items' slots lie end to end and are cut
// into one contiguous range for each CTA. A CTA that leaves an item writes one
// partial (m, l, o) for each of its query heads: row max in log2 units, sum of
// exponentials, weighted values.
#pragma once

#include "common.cuh"

namespace sas {
namespace {

constexpr int kD = 128;

// CTA c owns block slots [c V / grid, (c + 1) V / grid); cta_of is its inverse.
__host__ __device__ __forceinline__ long long slot_begin(long long c, long long V, int grid) { return c * V / grid; }
__host__ __device__ __forceinline__ int cta_of(long long s, long long V, int grid) {
    return (int)(((s + 1) * grid - 1) / V);
}

// One CTA for each (sequence, query head). A row without a readable block gets
// `none` and an lse of -inf.
__global__ void __launch_bounds__(kD)
decode_combine_kernel(const float* __restrict__ part_o, const float* __restrict__ part_ml, int nslot, int Hq, int Hkv,
                      int G, int K, long long V, int grid, __nv_bfloat16* __restrict__ o, float* __restrict__ lse, float none) {
    // launched as a programmatic dependent of decode_kernel: its blocks may be
    // resident before the decode grid ends; wait for that grid's writes here
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long row = blockIdx.x;          // n * Hq + hq
    const int d = threadIdx.x;
    const long long n = row / Hq;
    const int hq = (int)(row % Hq);
    const long long item = n * Hkv + hq / G;
    const long long s0 = item * (K + 1);
    const int nsl = cta_of(s0 + K, V, grid) - cta_of(s0, V, grid) + 1;
    const float* ml = part_ml + row * nslot * 2;
    float M = -INFINITY;
    for (int s = 0; s < nsl; ++s) M = fmaxf(M, ml[2 * s]);
    float Lsum = 0.f, acc = 0.f;
    if (M != -INFINITY) {
        for (int s = 0; s < nsl; ++s) {
            const float w = exp2f(ml[2 * s] - M);     // 0 for empty partials (m = -inf)
            Lsum = fmaf(ml[2 * s + 1], w, Lsum);
            acc = fmaf(part_o[(row * nslot + s) * kD + d], w, acc);
        }
    }
    o[row * kD + d] = __float2bfloat16_rn(M == -INFINITY ? none : acc / Lsum);
    if (lse != nullptr && d == 0) lse[row] = M == -INFINITY ? M : (M + log2f(Lsum)) * kLn2;
}

struct Layout {
    long long V;
    int grid, nslot;
};
Layout layout(int N, int Hkv, int K) {
    Layout r;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    r.V = (long long)N * Hkv * (K + 1);
    r.grid = (int)(r.V < sms ? r.V : sms);
    if (r.grid < 1) r.grid = 1;
    const long long mn = r.V / r.grid;                       // shortest CTA range
    const long long span = (K + 1 + mn - 1) / mn + 1;        // CTAs one item's slots can touch
    r.nslot = (int)(span < r.grid ? span : r.grid);
    return r;
}

}  // namespace
}  // namespace sas
