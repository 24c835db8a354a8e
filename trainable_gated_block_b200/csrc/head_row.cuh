// One head row (D values) held by D / 16 neighbouring lanes, for the kernels
// that norm and rotate queries and keys.
//
// Lane l of a row holds the dimensions 8l .. 8l+7 and D/2 + 8l .. D/2 + 8l+7:
// both halves of its eight rotation pairs (i, i + D/2), so the rotation needs
// no exchange between lanes, and each half is one 16-byte access in bf16 (two
// in fp32). Only the sum of squares crosses the row's lanes.
#pragma once

#include "common.cuh"

namespace sas {

template <int D>
struct HeadRow {
    static_assert(D == 64 || D == 128, "head size");
    static constexpr int kLanes = D / 16;            // lanes of one row
    static constexpr int kPerWarp = 32 / kLanes;     // rows a warp holds at a time
};

// Eight consecutive values at p (16-byte aligned), as fp32. Inputs are read
// once: they bypass L1, which the rotation table's rows are to stay in.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 w;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(p));
    return w;
}
template <typename T> struct Raw8;                   // eight values as loaded
template <> struct Raw8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = ld_stream(p); }
    __device__ __forceinline__ void load_cached(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = bf16x2_to_f32(v[e]);
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
        }
    }
};
template <> struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ld_stream(p);
        b = ld_stream(p + 4);
    }
    __device__ __forceinline__ void load_cached(const float* p) {
        a = __ldg(reinterpret_cast<const uint4*>(p));
        b = __ldg(reinterpret_cast<const uint4*>(p + 4));
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[e]);
    }
};

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf16x2_of(x[0], x[1]), bf16x2_of(x[2], x[3]), bf16x2_of(x[4], x[5]), bf16x2_of(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Sum over the lanes of a row (all lanes of the warp take part).
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = HeadRow<D>::kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 1 / rms of the row: rsqrt(mean(x^2) + eps), in fp32.
template <int D>
__device__ __forceinline__ float row_rrms(const float (&x)[16], float eps) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
    return rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
}

// The lane's eight angles of one position: cos and sin from a table row
// [cos(D/2) | sin(D/2)] in fp32.
struct Angles {
    float c[8], s[8];
    template <int D>
    __device__ __forceinline__ void load(const float* table, int pos, int l) {
        const float* row = table + (long long)pos * D + 8 * l;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + e));
            const float4 b = __ldg(reinterpret_cast<const float4*>(row + D / 2 + e));
            c[e] = a.x, c[e + 1] = a.y, c[e + 2] = a.z, c[e + 3] = a.w;
            s[e] = b.x, s[e + 1] = b.y, s[e + 2] = b.z, s[e + 3] = b.w;
        }
    }
    // (x_i, x_{i + D/2}) turned by the angle; `back` by its negative (the transpose).
    __device__ __forceinline__ void turn(float (&x)[16]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = x[e + 8];
            x[e] = fmaf(a, c[e], -b * s[e]);
            x[e + 8] = fmaf(b, c[e], a * s[e]);
        }
    }
    __device__ __forceinline__ void turn_back(float (&x)[16]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = x[e + 8];
            x[e] = fmaf(a, c[e], b * s[e]);
            x[e + 8] = fmaf(b, c[e], -a * s[e]);
        }
    }
};

// The lane's 16 weights of a head norm.
template <typename T, int D>
__device__ __forceinline__ void load_weight(const T* w, int l, float (&x)[16]) {
    Raw8<T> a, b;
    a.load_cached(w + 8 * l);
    b.load_cached(w + D / 2 + 8 * l);
    a.get(x);
    b.get(x + 8);
}

constexpr int kUnitHeads = 4;       // heads of one token that a row slot takes

__host__ __device__ __forceinline__ int unit_parts(int H) { return (H + kUnitHeads - 1) / kUnitHeads; }

// Norm and rotation of the heads h0, h0 + parts, ... of one token row (`src`
// to `dst`, both [H, D]) by the lanes of a row slot. The rows' loads are
// issued before `position()` is asked for, which may have to search. A
// negative position writes zeros; without `live` nothing is read or written
// (the lanes still take part in the warp's sums).
template <typename T, int D, typename Position>
__device__ __forceinline__ void norm_rope_unit(const T* src, T* dst, int H, int h0, const T* weight, const float* table,
                                               float eps, int l, bool live, Position position) {
    const int parts = unit_parts(H);
    Raw8<T> lo[kUnitHeads], hi[kUnitHeads];
#pragma unroll
    for (int i = 0; i < kUnitHeads; ++i) {
        const int h = h0 + i * parts;
        lo[i].zero();
        hi[i].zero();
        if (live && h < H) {
            lo[i].load(src + h * D + 8 * l);
            hi[i].load(src + h * D + D / 2 + 8 * l);
        }
    }
    const int pos = live ? position() : -1;
    Angles ang;
    ang.load<D>(table, max(pos, 0), l);
    float w[16];
    if (weight != nullptr) load_weight<T, D>(weight, l, w);
#pragma unroll
    for (int i = 0; i < kUnitHeads; ++i) {
        const int h = h0 + i * parts;
        float x[16];
        lo[i].get(x);
        hi[i].get(x + 8);
        if (weight != nullptr) {
            const float r = row_rrms<D>(x, eps);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
        }
        ang.turn(x);
        if (pos < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        if (live && h < H) {
            store8(dst + h * D + 8 * l, x);
            store8(dst + h * D + D / 2 + 8 * l, x + 8);
        }
    }
}

}  // namespace sas
