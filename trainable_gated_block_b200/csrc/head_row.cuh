// One head row (D values) held by D / 16 neighbouring lanes, for the kernels
// that norm and rotate queries and keys.
//
// Lane l of a row holds eight dimensions of its lower half and the same eight
// of its upper half: both values of its rotation pairs (i, i + D/2), so the
// rotation needs no exchange between lanes. Each half is one 16-byte access in
// bf16 (8l .. 8l+7) and two in fp32 (4l .. 4l+3 and D/4 + 4l .. + 3), so that the
// lanes of a row always touch neighbouring 16-byte pieces: with 32 consecutive
// bytes for each lane in fp32 every sector moved twice (65% of the copy rate
// instead of HBM's). Only the sum of squares crosses the row's lanes. Values are kept
// two to a 64-bit register for the f32x2 arithmetic of sm_100a (each half is
// rounded like the scalar instruction), which halves the instructions of rows
// that are otherwise bound by HBM.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace sas {

using f2 = unsigned long long;
using sm100::f2_add;
using sm100::f2_fma;
using sm100::f2_mul;
using sm100::f2_pack;
using sm100::f2_unpack;

template <int D>
struct HeadRow {
    static_assert(D == 64 || D == 128, "head size");
    static constexpr int kLanes = D / 16;            // lanes of one row
    static constexpr int kPerWarp = 32 / kLanes;     // rows a warp holds at a time
};

// A lane's 16 values: a of the lower half of the row, b those D/2 further.
struct Half {
    f2 v[4];
};
struct Row {
    Half a, b;
};

// Eight consecutive values as loaded: 16-byte pieces.
// Piece i of lane l starts at dimension i * D / 4 + l * kStep of the half row.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    static constexpr int kPieces = 1, kStep = 8;
    static __device__ __forceinline__ Half get(const uint4 (&p)[1]) {
        const uint32_t w[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
        Half h;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f32(w[i]);
            h.v[i] = f2_pack(f.x, f.y);
        }
        return h;
    }
};
template <> struct Raw8<float> {
    static constexpr int kPieces = 2, kStep = 4;
    static __device__ __forceinline__ Half get(const uint4 (&p)[2]) {
        const uint32_t w[8] = {p[0].x, p[0].y, p[0].z, p[0].w, p[1].x, p[1].y, p[1].z, p[1].w};
        Half h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h.v[i] = f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        return h;
    }
};

// Inputs are read once: they bypass L1, which the rotation table's rows are to stay in.
// (Not by the read-only path, as all loads of these kernels: dependent.cuh.)
__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 w;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(p));
    return w;
}

__device__ __forceinline__ uint32_t bf16x2_of(f2 v) {
    const float2 f = f2_unpack(v);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The lane's eight values to a half row at p.
template <int D>
__device__ __forceinline__ void store_half(__nv_bfloat16* p, int l, const Half& h) {
    *reinterpret_cast<uint4*>(p + 8 * l) =
        make_uint4(bf16x2_of(h.v[0]), bf16x2_of(h.v[1]), bf16x2_of(h.v[2]), bf16x2_of(h.v[3]));
}
template <int D>
__device__ __forceinline__ void store_half(float* p, int l, const Half& h) {
    *reinterpret_cast<ulonglong2*>(p + 4 * l) = make_ulonglong2(h.v[0], h.v[1]);
    *reinterpret_cast<ulonglong2*>(p + D / 4 + 4 * l) = make_ulonglong2(h.v[2], h.v[3]);
}
template <int D, typename T>
__device__ __forceinline__ void store_row(T* p, int l, const Row& r) {
    store_half<D>(p, l, r.a);
    store_half<D>(p + D / 2, l, r.b);
}

// Sum over the lanes of a row (all lanes of the warp take part).
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = HeadRow<D>::kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float f2_sum(f2 v) {
    const float2 f = f2_unpack(v);
    return f.x + f.y;
}

// Sum over the row of the products of two rows' values.
template <int D>
__device__ __forceinline__ float row_dot(const Row& x, const Row& y) {
    f2 s = f2_mul(x.a.v[0], y.a.v[0]), t = f2_mul(x.b.v[0], y.b.v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        s = f2_fma(x.a.v[i], y.a.v[i], s);
        t = f2_fma(x.b.v[i], y.b.v[i], t);
    }
    return row_sum<D>(f2_sum(f2_add(s, t)));
}

// 1 / rms of the row: rsqrt(mean(x^2) + eps), in fp32.
template <int D>
__device__ __forceinline__ float row_rrms(const Row& x, float eps) {
    return rsqrtf(row_dot<D>(x, x) * (1.f / D) + eps);
}

// The lane's eight angles of one position: cos and sin from a table row
// [cos(D/2) | sin(D/2)] in fp32.
struct Angles {
    Half c, s;
};
template <typename T, int D>
__device__ __forceinline__ Angles load_angles(const float* table, int pos, int l) {
    // in 16-byte pieces: the second four dimensions of the lane's eight follow the first, or lie D / 4 further
    constexpr int kSecond = sizeof(T) == 2 ? 1 : D / 16;
    const ulonglong2* row = reinterpret_cast<const ulonglong2*>(table + (long long)pos * D + Raw8<T>::kStep * l);
    const ulonglong2 c0 = row[0], c1 = row[kSecond], s0 = row[D / 8], s1 = row[D / 8 + kSecond];
    Angles g;
    g.c.v[0] = c0.x, g.c.v[1] = c0.y, g.c.v[2] = c1.x, g.c.v[3] = c1.y;
    g.s.v[0] = s0.x, g.s.v[1] = s0.y, g.s.v[2] = s1.x, g.s.v[3] = s1.y;
    return g;
}

// The lane's 16 weights of a head norm (ones without weights).
template <typename T, int D>
__device__ __forceinline__ Row load_weight(const T* w, int l) {
    Row r;
    if (w == nullptr) {
        const f2 one = f2_pack(1.f, 1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.a.v[i] = r.b.v[i] = one;
        return r;
    }
    uint4 p[Raw8<T>::kPieces], q[Raw8<T>::kPieces];
#pragma unroll
    for (int i = 0; i < Raw8<T>::kPieces; ++i) {
        const T* at = w + i * (D / 4) + Raw8<T>::kStep * l;
        p[i] = *reinterpret_cast<const uint4*>(at);
        q[i] = *reinterpret_cast<const uint4*>(at + D / 2);
    }
    r.a = Raw8<T>::get(p);
    r.b = Raw8<T>::get(q);
    return r;
}

// Weight and rotation in one: y_a = r (x_a (w_a c) - x_b (w_b s)), y_b = r (x_b (w_b c) + x_a (w_a s)),
// with coefficients that all heads of a token share.
struct Turn {
    Half ac, bs, bc, as;        // w_a c, -(w_b s), w_b c, w_a s
    __device__ __forceinline__ Turn(const Angles& g, const Row& w) {
        const f2 neg = f2_pack(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ac.v[i] = f2_mul(w.a.v[i], g.c.v[i]);
            bs.v[i] = f2_mul(f2_mul(w.b.v[i], g.s.v[i]), neg);
            bc.v[i] = f2_mul(w.b.v[i], g.c.v[i]);
            as.v[i] = f2_mul(w.a.v[i], g.s.v[i]);
        }
    }
    __device__ __forceinline__ Row operator()(const Row& x, float r) const {
        const f2 rr = f2_pack(r, r);
        Row y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y.a.v[i] = f2_mul(rr, f2_fma(x.a.v[i], ac.v[i], f2_mul(x.b.v[i], bs.v[i])));
            y.b.v[i] = f2_mul(rr, f2_fma(x.b.v[i], bc.v[i], f2_mul(x.a.v[i], as.v[i])));
        }
        return y;
    }
};

// 16 bytes from global to shared memory without a register (zeroes without
// `live`); each thread copies and later reads its own pieces only, so that the
// groups need no barrier.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t p) {
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(p)
                 : "memory");
    return w;
}

// A head row of a thread's pieces: copy from global memory (src: the row), and
// read. From half to half: kPieces * kThreads * 16 bytes.
template <typename T, int D, int kThreads>
__device__ __forceinline__ void copy_row(uint32_t at, const T* src, int l, bool live) {
    constexpr int kP = Raw8<T>::kPieces;
#pragma unroll
    for (int i = 0; i < 2 * kP; ++i)
        copy16(at + i * kThreads * 16, src + i / kP * (D / 2) + i % kP * (D / 4) + Raw8<T>::kStep * l, live);
}
template <typename T, int kThreads>
__device__ __forceinline__ Row read_row(uint32_t at) {
    constexpr int kP = Raw8<T>::kPieces;
    uint4 p[kP], q[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
        p[i] = ld_shared16(at + i * kThreads * 16);
        q[i] = ld_shared16(at + (kP + i) * kThreads * 16);
    }
    return {Raw8<T>::get(p), Raw8<T>::get(q)};
}

__host__ __device__ __forceinline__ uint32_t parts_of(int H, int heads) { return ((uint32_t)H + heads - 1) / heads; }

}  // namespace sas
