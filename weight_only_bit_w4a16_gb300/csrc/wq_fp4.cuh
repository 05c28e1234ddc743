// wq_fp4.cuh -- quantisation of fp32 values to microscaled 4-bit floats in
// registers, shared by the quantiser (wq_fp4_quant.cu) and the norm kernels
// (wq_norm.cu), and the scale layout the block-scaled matrix instruction
// takes.
//
// A group is 16 (NVFP4) or 32 (MXFP4) consecutive k of a row, a = max |x|:
//   NVFP4  s = e4m3(min(448, a / (6 t))), code = e2m1(x / (s t)), t the
//          tensor scale (1 without one);
//   MXFP4  E = max(floor(log2 a) - 2, -127), code = e2m1(x / 2^E) (OCP MX:
//          2 is the exponent of e2m1's largest value).
// Both round to nearest even and saturate at 6.  A group with an infinity or
// a NaN gets the NaN scale (0x7F / 0xFF) and codes 0, so all its values are
// NaN: saturating an infinity would hide it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "wq_common.cuh"

namespace wq {

// Byte of the scale of row r, group g in the tiled layout: 512-byte blocks of
// 128 rows x 4 groups, ordered by (r / 128, g / 4); gblocks = ceil(groups / 4).
// Inside a block row r has its four bytes at 16 (r mod 32) + 4 (r / 32): the
// 32 x 16 byte image that one tensor-memory copy spreads over the lanes.
__host__ __device__ __forceinline__ size_t tiled_scale_offset(int r, int g, int gblocks) {
    return ((size_t)(r >> 7) * gblocks + (g >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (g & 3);
}

template <int FMT>
constexpr int kGroupOf = FMT == kNVFP4 ? 16 : 32;

// 16 bytes that the stream's previous kernel may have written.  The kernels
// start while that kernel runs, so such inputs change under them until
// griddepcontrol.wait: the load is a coherent one (not .nc) and, being
// volatile, stays behind the wait.  Narrower inputs are read by plain loads,
// which the wait's memory clobber holds back just as well.
__device__ __forceinline__ uint4 ld_stream_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// two fp32 in one 64-bit register pair: the packed fp32 instructions
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// eight fp32 -> eight e2m1 codes of one word, value i in nibble i
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

__device__ __forceinline__ uint32_t f32_to_e4m3(float v) {   // v in 0 .. 448
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
    return d & 0xFFu;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
    const uint32_t h = e4m3x2_to_f16x2(byte);
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

// the approximate reciprocal and one Newton step r + r (1 - x r)
__device__ __forceinline__ float rcp_newton(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return fmaf(r, fmaf(-x, r, 1.0f), r);
}

// A reciprocal that stays finite: with a tensor scale of 0 (the recommended one
// of an all-zero tensor) a group's 0 / 0 then gives scale 0, and any other
// value code 0 through the step, which is 0.
__device__ __forceinline__ float rcp_finite(float x) { return fminf(rcp_newton(x), 0x1.fffffep127f); }

// What a group's values are quantised with.
struct GroupScale {
    uint32_t byte;   // the stored scale
    float step;      // the value of code 2 (1.0 in e2m1): s t, or 2^E; NaN for a group that is not finite
    float inv;       // 1 / step (MXFP4: exact); 0 where every code is 0
    bool bad;        // the group holds an infinity or a NaN: codes 0
    bool far;        // NVFP4: a value's quotient by the step may pass fp32's range
};

// amax_bits: the largest fp32 bit pattern of |x| over the group (a NaN or an
// infinity is the largest of all); t: the tensor scale, rcp6t = rcp_finite(6 t).
template <int FMT>
__device__ __forceinline__ GroupScale group_scale(uint32_t amax_bits, float t, float rcp6t) {
    GroupScale g;
    g.bad = amax_bits >= 0x7F800000u;
    if constexpr (FMT == kNVFP4) {
        const float a = __uint_as_float(amax_bits);
        // a / (6 t): q0 = a r and one remainder step q0 + r (a - 6 t q0)
        // (Markstein's division), within 2^-21 of the quotient; the clamp
        // first, where it may overflow
        const float q0 = a * rcp6t;
        const float q1 = fmaf(fmaf(-q0, 6.0f * t, a), rcp6t, q0);
        const uint32_t b = f32_to_e4m3(q0 >= 448.0f ? 448.0f : q1);
        g.byte = g.bad ? 0x7Fu : b;
        const float s = e4m3_to_f32(b) * t;
        g.inv = s > 0.0f && !g.bad ? rcp_newton(s) : 0.0f;
        g.step = g.bad ? __uint_as_float(0x7FC00000u) : s;
        g.far = a * g.inv >= 0x1p127f;   // (a tensor scale far below the data; not so where a is not finite)
    } else {
        const int e = (int)(amax_bits >> 23);            // biased; subnormals have 0
        const uint32_t b = e > 2 ? e - 2 : 0;            // 2 = the exponent of 6.0 .. 4.0
        g.byte = g.bad ? 0xFFu : b;
        g.inv = g.bad ? 0.0f : __uint_as_float((254u - b) << 23);
        g.step = g.bad ? __uint_as_float(0x7FC00000u)
                       : (b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u));
        g.far = false;
    }
    return g;
}

// Codes of eight values of a group.  NVFP4 divides by the step: q = x inv and
// one remainder step (Markstein's), q + inv (x - q step), which makes a
// quotient that lies exactly on the tie between two codes come out exactly
// (x inv alone lands above the tie for scales of mantissa 1.875, where the tie
// goes down).  A quotient past fp32's range would leave no sign behind (an
// infinity, and NaN as its remainder), so groups that may hold one are first
// cut to 8 steps, which saturate just as well.
template <int FMT>
__device__ __forceinline__ uint32_t quantize8(const float (&values)[8], const GroupScale& g) {
    float x[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = values[i];
    if (FMT == kNVFP4 && g.far) {
        const float end = 8.0f * g.step;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -end), end);
    }
    const uint64_t inv = f32x2(g.inv, g.inv);
    const uint64_t nstep = f32x2(-g.step, -g.step);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t xx = f32x2(x[2 * i], x[2 * i + 1]);
        uint64_t q = f32x2_mul(xx, inv);
        if constexpr (FMT == kNVFP4) q = f32x2_fma(f32x2_fma(q, nstep, xx), inv, q);
        f32x2_split(q, v[2 * i], v[2 * i + 1]);
    }
    const uint32_t c = e2m1x8(v);
    return g.bad ? 0u : c;
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// the bf16 image of eight codes: code value * step, rounded once
__device__ __forceinline__ uint4 values8(uint32_t codes, float step) {
    uint32_t h[4], o[4];
    e2m1x8_to_f16x2(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi) : "r"(h[i]));
        o[i] = bf16x2_of(lo * step, hi * step);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace wq
