// wq_norm.cu -- the norms between two blocks, in one pass over the row:
//   b  = branch                      (the output of the block)
//   b  = N(b; post weight, bias)     optional norm after the block
//   b *= gate[row group]             optional
//   x' = alpha x + beta b            the residual stream, stored in its type
//   u  = N(x'; weight, bias)         the norm before the next block, stored as
//                                    bf16, fp32 or 4-bit codes and scales
// N is the RMS norm v / sqrt(mean v^2 + eps) or the layer norm
// (v - mean v) / sqrt(mean (v - mean v)^2 + eps), times the weight, plus the
// bias.
//
// All of it is fp32; u is formed from the unrounded x', so the stream's
// storage type does not enter it.  The bound is HBM: every input is read once
// and every output written once.  TPR threads share a row and keep it in
// registers (VPT vectors of 8 elements each), so the statistics cost no second
// read; short rows share a warp; with many rows a block takes row after row and
// loads ahead.  The layer norm's variance is the mean square of the deviations,
// a second sum over registers, not a difference of moments.  A row wider than
// 16384 runs row_loop_kernel, which reads it again for each sum (from L2): at
// 32768 the registers of one block no longer hold it.
#include "wq_fp4.cuh"
#include "wq_internal.h"
#include "wq_tc.cuh"

namespace wq {

namespace {

struct NormArgs {
    wq_norm n;
    int rows_per_gate;
    float inv_d;
    int gblocks;   // 4-bit output, tiled scales: ceil(groups / 4)
};

// Dependents may start once the predecessor has completed, but not those of
// 4-bit output before it is all written: it may be the weight of a call that
// reads its weights ahead (see quantize_kernel).
__device__ __forceinline__ void let_dependents_start(const NormArgs& a) {
    if (a.n.out_type < WQ_NORM_OUT_NVFP4) sm100::grid_dependents_launch();
}

// How a row's elements are shared out.  kVector: a thread's eight are
// consecutive, in one or two 16-byte accesses (every row 16-byte aligned).
// kPieces: the same eight, element by element (unaligned slices of a width of
// whole vectors).  kScalar, other widths: element by element, the thread's
// eight `stride` apart, so that a warp's access is one run of the row (1000
// rows of 1001: 13.1 us with consecutive elements).
enum Access { kVector, kScalar, kPieces };

// element e (0 .. 7) of the eight that start at i
template <Access ACC>
__device__ __forceinline__ int elem_of(int i, int e, int stride) {
    return ACC == kScalar ? i + e * stride : i + e;
}

// the thread's eight elements of a row as fp32; elements past d are 0
template <Access ACC>
__device__ __forceinline__ void load8(const void* base, int f32, long long off, int i, int stride, int d,
                                      float (&v)[8]) {
    constexpr bool ALIGNED = ACC == kVector;
    if (f32) {
        const float* p = static_cast<const float*>(base) + off + i;
        if constexpr (ALIGNED) {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int o = elem_of<ACC>(0, e, stride);
                v[e] = i + o < d ? p[o] : 0.0f;
            }
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + off + i;
        if constexpr (ALIGNED) {
            const uint4 a = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(w[e] << 16);
                v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int o = elem_of<ACC>(0, e, stride);
                v[e] = i + o < d ? __uint_as_float((uint32_t)p[o] << 16) : 0.0f;
            }
        }
    }
}

template <Access ACC>
__device__ __forceinline__ void store8(void* base, int f32, long long off, int i, int stride, int d,
                                       const float (&v)[8]) {
    constexpr bool ALIGNED = ACC == kVector;
    if (f32) {
        float* p = static_cast<float*>(base) + off + i;
        if constexpr (ALIGNED) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int o = elem_of<ACC>(0, e, stride);
                if (i + o < d) p[o] = v[e];
            }
        }
    } else {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + off + i;
        if constexpr (ALIGNED) {
            *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]),
                                                      bf16x2_of(v[4], v[5]), bf16x2_of(v[6], v[7]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int o = elem_of<ACC>(0, e, stride);
                if (i + o < d) p[o] = __float2bfloat16_rn(v[e]);
            }
        }
    }
}

// Room for the sums of a row: each of its four (two norms, a mean and a mean
// square) has a buffer of its own, so one barrier a sum is enough.
template <int TPR>
struct __align__(16) RowSums {
    float part[4][TPR > 32 ? (TPR / 32 + 3) / 4 * 4 : 4];
};

// Sum over the TPR threads of a row, in a fixed order; every thread gets it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, RowSums<TPR>& sums, int which) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        if ((threadIdx.x & 31) == 0) sums.part[which][threadIdx.x >> 5] = v;
        __syncthreads();
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < W; w += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&sums.part[which][w]);
            s[0] += f.x;
            if (w + 1 < W) s[1] += f.y;
            if (w + 2 < W) s[2] += f.z;
            if (w + 3 < W) s[3] += f.w;
        }
        v = (s[0] + s[1]) + (s[2] + s[3]);
    }
    return v;
}

// first element of thread t's vector j: consecutive vectors, or strided elements
template <int TPR, Access ACC>
__device__ __forceinline__ int first_of(int j, int t) {
    return ACC == kScalar ? j * TPR * 8 + t : (j * TPR + t) * 8;
}

// v = N(v): statistics over the row, then weight and bias.
template <int TPR, int VPT, Access ACC>
__device__ __forceinline__ void norm_row(float (&v)[VPT][8], const NormArgs& a, const void* weight, const void* bias,
                                         int t, RowSums<TPR>& sums, int which) {
    const int d = a.n.d;
    if (a.n.kind == WQ_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[j][e];
        const float mean = row_sum<TPR>(s, sums, which) * a.inv_d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first_of<TPR, ACC>(j, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = elem_of<ACC>(i, e, TPR) < d ? v[j][e] - mean : 0.0f;
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
    const float scale = 1.0f / sqrtf(row_sum<TPR>(s, sums, which + 1) * a.inv_d + a.n.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = first_of<TPR, ACC>(j, t);
        if (i >= d) continue;
        float w[8], c[8];
        if (weight) {
            load8<ACC>(weight, 0, 0, i, TPR, d, w);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 1.0f;
        }
        if (bias) {
            load8<ACC>(bias, 0, 0, i, TPR, d, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = fmaf(v[j][e] * scale, w[e], c[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * scale * w[e];
        }
    }
}

// Eight values of a row as codes and, from the group's first lane, its scale.
// Lanes hold consecutive vectors, so a group is 2 (NVFP4) or 4 (MXFP4)
// neighbouring lanes, all live or all past d (d is a multiple of 32).
template <int FMT>
__device__ __forceinline__ void store_codes(const NormArgs& a, int row, int i, const float (&v)[8], float t,
                                            float rcp6t) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if constexpr (FMT == kMXFP4) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const GroupScale g = group_scale<FMT>(top, t, rcp6t);
    const uint32_t codes = quantize8<FMT>(v, g);
    if (i >= a.n.d) return;
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.n.out) + ((size_t)row * a.n.d + i) / 2) = codes;
    constexpr int kG = kGroupOf<FMT>;
    if (i % kG == 0) {
        const int G = a.n.d / kG, gi = i / kG;
        if (a.n.out_scale_layout == WQ_SCALES_TILED) {
            uint8_t* p = static_cast<uint8_t*>(a.n.out_scales) + tiled_scale_offset(row, gi, a.gblocks);
            *p = (uint8_t)g.byte;
            if (gi == G - 1)
                for (int k = 1; (gi + k) & 3; ++k) p[k] = 0;
        } else {
            static_cast<uint8_t*>(a.n.out_scales)[(size_t)row * G + gi] = (uint8_t)g.byte;
        }
    }
}

template <int TPR, int VPT, Access ACC>
__device__ __forceinline__ void store_u(const NormArgs& a, int row, int t, const float (&v)[VPT][8]) {
    const int d = a.n.d;
    if constexpr (ACC != kScalar) {
        if (a.n.out_type == WQ_NORM_OUT_NVFP4 || a.n.out_type == WQ_NORM_OUT_MXFP4) {
            float ts = 1.0f, rcp6t = 1.0f / 6.0f;
            if (a.n.out_tensor_scale) {
                ts = *a.n.out_tensor_scale;
                rcp6t = rcp_finite(6.0f * ts);
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {   // every lane, for the shuffles
                const int i = first_of<TPR, ACC>(j, t);
                if (a.n.out_type == WQ_NORM_OUT_NVFP4) store_codes<kNVFP4>(a, row, i, v[j], ts, rcp6t);
                else store_codes<kMXFP4>(a, row, i, v[j], ts, rcp6t);
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = first_of<TPR, ACC>(j, t);
        if (i < d) store8<ACC>(a.n.out, a.n.out_type == WQ_NORM_OUT_F32, (long long)row * a.n.ldo, i, TPR, d, v[j]);
    }
}

// Blocks an SM is to hold, which sets the registers of a thread: 1536 threads
// with up to 42, or 1024 with 64 for two vectors a thread.  A row's time is the
// latency of its loads and of its two sums, and the work of a 16-bit row is
// bound by instructions (430 for a warp's 256 elements, the issue slots 69 %
// busy) as much as by HBM, so rows in flight count.  Measured, 8192 rows, fp32
// stream and a gate for each element / bf16 and a gate for each channel:
// 3072 wide 65 / 56 us (70 / 53 with two vectors a thread, 81 us with three
// and 128 threads), 8192 wide 198 / 147 us (211 / 169 with one vector, 1024
// threads).
template <int TPR, int VPT>
constexpr int kMinBlocks = (VPT > 1 ? 1024 : 1536) / (TPR <= 32 ? 128 : TPR);

// Up to 32 threads a row: 128 / TPR rows in a block of 128; else one row in a
// block.
template <int TPR, int VPT, Access ACC>
__global__ void __launch_bounds__(TPR <= 32 ? 128 : TPR, kMinBlocks<TPR, VPT>)
    row_kernel(const __grid_constant__ NormArgs a) {
    __shared__ RowSums<TPR> sums;
    sm100::grid_dependency_wait();
    let_dependents_start(a);
    const int d = a.n.d;
    int row = TPR <= 32 ? blockIdx.x * (128 / TPR) + threadIdx.x / TPR : blockIdx.x;
    int t = TPR <= 32 ? threadIdx.x % TPR : threadIdx.x;
    if (row >= a.n.rows) {
        if constexpr (TPR >= 32) return;   // whole warps; above 32 never
        // other lanes of the warp may have rows: these stay for the sums' and
        // the groups' shuffles, past the end of a row that there is
        row = a.n.rows - 1;
        t = d;
    }
    const long long grow = a.n.gate && a.n.gate_rows > 1 ? (long long)(row / a.rows_per_gate) * d : 0;
    float x[VPT][8], b[VPT][8], g[VPT][8];
    // all of the row's loads at once, the gate's too: none waits for a sum
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = first_of<TPR, ACC>(j, t);
        if (i < d) {
            if (a.n.branch) load8<ACC>(a.n.branch, a.n.branch_type, (long long)row * a.n.ldb, i, TPR, d, b[j]);
            load8<ACC>(a.n.x, a.n.x_type, (long long)row * a.n.ldx, i, TPR, d, x[j]);
            if (a.n.gate) load8<ACC>(a.n.gate, 0, grow, i, TPR, d, g[j]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] = b[j][e] = g[j][e] = 0.0f;
        }
    }
    if (a.n.branch) {
        if (a.n.post) norm_row<TPR, VPT, ACC>(b, a, a.n.post_weight, a.n.post_bias, t, sums, 0);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (a.n.gate) {
#pragma unroll
                for (int e = 0; e < 8; ++e) b[j][e] *= g[j][e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] = fmaf(a.n.branch_scale, b[j][e], a.n.residual_scale * x[j][e]);
        }
    } else if (a.n.residual_scale != 1.0f) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] *= a.n.residual_scale;
    }
    if (a.n.x_out) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first_of<TPR, ACC>(j, t);
            if (i < d) store8<ACC>(a.n.x_out, a.n.x_type, (long long)row * a.n.ldxo, i, TPR, d, x[j]);
        }
    }
    if (a.n.out_type == WQ_NORM_OUT_NONE) return;
    norm_row<TPR, VPT, ACC>(x, a, a.n.weight, a.n.bias, t, sums, 2);
    store_u<TPR, VPT, ACC>(a, row, t, x);
}

// ---------------------------------------------------------------------------
// many rows: a block takes row after row and loads the next one while it works
// on the current one
// ---------------------------------------------------------------------------
// row_kernel's arithmetic in the same order, so a row gets the same bits from
// either.  What it saves: a row's loads wait for no block to start and for no
// sum, the weights (and a gate of one row) stay in registers, and addresses are
// formed once.  8192 rows of 3072, fp32 stream and a gate for each element 65
// -> 56 us (6.2 TB/s), bf16 and a gate for each channel 53 -> 41 us.
template <int VPT>
struct RowRaw {
    uint4 x0[VPT], x1[VPT], b[VPT], g[VPT];   // fp32 x: both; bf16: x0
};

__device__ __forceinline__ void unpack_bf16(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}

// norm_row with the weight's raw bf16 in registers
template <int TPR, int VPT>
__device__ __forceinline__ void norm_vectors(float (&v)[VPT][8], const NormArgs& a, const uint4 (&weight)[VPT],
                                             const void* bias, RowSums<TPR>& sums, int which) {
    const int d = a.n.d, t = threadIdx.x;
    if (a.n.kind == WQ_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[j][e];
        const float mean = row_sum<TPR>(s, sums, which) * a.inv_d;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = (j * TPR + t) * 8 < d ? v[j][e] - mean : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
    const float scale = 1.0f / sqrtf(row_sum<TPR>(s, sums, which + 1) * a.inv_d + a.n.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = (j * TPR + t) * 8;
        float w[8];
        unpack_bf16(weight[j], w);
        if (bias) {
            if (i >= d) continue;
            float c[8];
            load8<kVector>(bias, 0, 0, i, 1, d, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = fmaf(v[j][e] * scale, w[e], c[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * scale * w[e];
        }
    }
}

// Blocks an SM is to hold: up to 1024 threads (64 registers and more; three
// blocks of 384 threads and 56 registers: 61 us where two take 56), 512 with
// two vectors a thread.
template <int TPR, int VPT>
constexpr int kStreamBlocks = (VPT > 1 ? 512 : 1024) / TPR;

template <int TPR, int VPT, bool XF32>
__global__ void __launch_bounds__(TPR, kStreamBlocks<TPR, VPT>) stream_kernel(const __grid_constant__ NormArgs a) {
    __shared__ RowSums<TPR> sums[2];   // rows in turn: a row may have one sum only, and so one barrier
    sm100::grid_dependency_wait();
    let_dependents_start(a);
    const int d = a.n.d, t = threadIdx.x;
    const bool gates = a.n.gate && a.n.gate_rows > 1;
    const uint4 zero = make_uint4(0, 0, 0, 0), one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    auto vec = [&](const void* p, int i) {
        return p ? i < d ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i) : zero : one;
    };
    uint4 w[VPT], pw[VPT], g0[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = (j * TPR + t) * 8;
        w[j] = vec(a.n.weight, i);
        pw[j] = vec(a.n.post_weight, i);
        g0[j] = gates ? zero : vec(a.n.gate, i);
    }
    float ts = 1.0f, rcp6t = 1.0f / 6.0f;
    if (a.n.out_type >= WQ_NORM_OUT_NVFP4 && a.n.out_tensor_scale) {
        ts = *a.n.out_tensor_scale;
        rcp6t = rcp_finite(6.0f * ts);
    }
    auto fetch = [&](int row, RowRaw<VPT>& r) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = (j * TPR + t) * 8;
            r.x0[j] = r.x1[j] = r.b[j] = r.g[j] = zero;
            if (i >= d) continue;
            if (a.n.branch)
                r.b[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.n.branch) +
                                                         (long long)row * a.n.ldb + i);
            if constexpr (XF32) {
                const uint4* p =
                    reinterpret_cast<const uint4*>(static_cast<const float*>(a.n.x) + (long long)row * a.n.ldx + i);
                r.x0[j] = p[0];
                r.x1[j] = p[1];
            } else {
                r.x0[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.n.x) +
                                                          (long long)row * a.n.ldx + i);
            }
            if (gates)
                r.g[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.n.gate) +
                                                         (long long)(row / a.rows_per_gate) * d + i);
        }
    };
    RowRaw<VPT> next;
    int row = blockIdx.x;
    fetch(row, next);   // the grid has no more blocks than rows
    for (int turn = 0; row < a.n.rows; row += gridDim.x, turn ^= 1) {
        const RowRaw<VPT> cur = next;
        if (a.n.rows - row > (int)gridDim.x) fetch(row + gridDim.x, next);
        float x[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if constexpr (XF32) {
                const uint32_t q[8] = {cur.x0[j].x, cur.x0[j].y, cur.x0[j].z, cur.x0[j].w,
                                       cur.x1[j].x, cur.x1[j].y, cur.x1[j].z, cur.x1[j].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] = __uint_as_float(q[e]);
            } else {
                unpack_bf16(cur.x0[j], x[j]);
            }
        }
        if (a.n.branch) {
            float b[VPT][8];
#pragma unroll
            for (int j = 0; j < VPT; ++j) unpack_bf16(cur.b[j], b[j]);
            if (a.n.post) norm_vectors<TPR, VPT>(b, a, pw, a.n.post_bias, sums[turn], 0);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (a.n.gate) {
                    float g[8];
                    unpack_bf16(gates ? cur.g[j] : g0[j], g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) b[j][e] *= g[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] = fmaf(a.n.branch_scale, b[j][e], a.n.residual_scale * x[j][e]);
            }
        } else if (a.n.residual_scale != 1.0f) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] *= a.n.residual_scale;
        }
        if (a.n.x_out) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = (j * TPR + t) * 8;
                if (i < d) store8<kVector>(a.n.x_out, XF32, (long long)row * a.n.ldxo, i, 1, d, x[j]);
            }
        }
        if (a.n.out_type == WQ_NORM_OUT_NONE) continue;
        norm_vectors<TPR, VPT>(x, a, w, a.n.bias, sums[turn], 2);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = (j * TPR + t) * 8;
            if (a.n.out_type == WQ_NORM_OUT_NVFP4) store_codes<kNVFP4>(a, row, i, x[j], ts, rcp6t);
            else if (a.n.out_type == WQ_NORM_OUT_MXFP4) store_codes<kMXFP4>(a, row, i, x[j], ts, rcp6t);
            else if (i < d) store8<kVector>(a.n.out, a.n.out_type == WQ_NORM_OUT_F32, (long long)row * a.n.ldo, i, 1, d, x[j]);
        }
    }
}

template <int TPR, int VPT>
cudaError_t launch_stream(const NormArgs& a, cudaStream_t s) {
    const long long most = (long long)sm_count() * kStreamBlocks<TPR, VPT>;
    const unsigned blocks = (unsigned)(a.n.rows < most ? a.n.rows : most);
    return a.n.x_type == WQ_TYPE_F32 ? launch_dependent(stream_kernel<TPR, VPT, true>, blocks, TPR, 1, 0, s, a)
                                     : launch_dependent(stream_kernel<TPR, VPT, false>, blocks, TPR, 1, 0, s, a);
}

// ---------------------------------------------------------------------------
// rows wider than the registers hold: 1024 threads, 8192 elements at a time,
// the row read again for each sum
// ---------------------------------------------------------------------------
constexpr int kLoopThreads = 1024;

struct Stat {
    float mean, scale;
};

// mean (layer) and 1 / sqrt(mean square + eps) of f(i) over the row
template <typename F>
__device__ __forceinline__ Stat row_stat(const NormArgs& a, RowSums<kLoopThreads>& sums, int which, F f) {
    const int d = a.n.d, t = threadIdx.x;
    Stat st{0.0f, 0.0f};
    if (a.n.kind == WQ_NORM_LAYER) {
        float s = 0.0f;
        for (int i = t * 8; i < d; i += kLoopThreads * 8) {
            float v[8];
            f(i, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += i + e < d ? v[e] : 0.0f;
        }
        st.mean = row_sum<kLoopThreads>(s, sums, which) * a.inv_d;
    }
    float s = 0.0f;
    for (int i = t * 8; i < d; i += kLoopThreads * 8) {
        float v[8];
        f(i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = i + e < d ? v[e] - st.mean : 0.0f;
            s = fmaf(c, c, s);
        }
    }
    st.scale = 1.0f / sqrtf(row_sum<kLoopThreads>(s, sums, which + 1) * a.inv_d + a.n.eps);
    return st;
}

template <Access ACC>
__device__ __forceinline__ void apply_norm(const Stat& st, const void* weight, const void* bias, int i, int d,
                                           float (&v)[8]) {
    float w[8], c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f, c[e] = 0.0f;
    if (weight) load8<ACC>(weight, 0, 0, i, 1, d, w);
    if (bias) load8<ACC>(bias, 0, 0, i, 1, d, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - st.mean) * st.scale, w[e], c[e]);
}

template <Access ACC>
__global__ void __launch_bounds__(kLoopThreads) row_loop_kernel(const __grid_constant__ NormArgs a) {
    __shared__ RowSums<kLoopThreads> sums;
    sm100::grid_dependency_wait();
    let_dependents_start(a);
    const int row = blockIdx.x, d = a.n.d, t = threadIdx.x;
    Stat post{0.0f, 1.0f};
    if (a.n.branch && a.n.post)
        post = row_stat(a, sums, 0, [&](int i, float (&v)[8]) {
            load8<ACC>(a.n.branch, a.n.branch_type, (long long)row * a.n.ldb, i, 1, d, v);
        });
    // x' of elements i .. i + 7, formed again wherever it is needed; x_out is
    // written by the last pass, as it may be x itself
    auto xnew = [&](int i, float (&v)[8]) {
        load8<ACC>(a.n.x, a.n.x_type, (long long)row * a.n.ldx, i, 1, d, v);
        if (!a.n.branch) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= a.n.residual_scale;
            return;
        }
        float b[8], g[8];
        load8<ACC>(a.n.branch, a.n.branch_type, (long long)row * a.n.ldb, i, 1, d, b);
        if (a.n.post) apply_norm<ACC>(post, a.n.post_weight, a.n.post_bias, i, d, b);
        if (a.n.gate) {
            load8<ACC>(a.n.gate, 0, (long long)(row / a.rows_per_gate) * d, i, 1, d, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(a.n.branch_scale, b[e], a.n.residual_scale * v[e]);
    };
    Stat pre{0.0f, 1.0f};
    if (a.n.out_type != WQ_NORM_OUT_NONE) pre = row_stat(a, sums, 2, xnew);
    const bool fp4 = a.n.out_type == WQ_NORM_OUT_NVFP4 || a.n.out_type == WQ_NORM_OUT_MXFP4;
    float ts = 1.0f, rcp6t = 1.0f / 6.0f;
    if (fp4 && a.n.out_tensor_scale) {
        ts = *a.n.out_tensor_scale;
        rcp6t = rcp_finite(6.0f * ts);
    }
    for (int i0 = 0; i0 < d; i0 += kLoopThreads * 8) {   // the same trips for every lane: store_codes shuffles
        const int i = i0 + t * 8;
        float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (i < d) {
            xnew(i, v);
            if (a.n.x_out) store8<ACC>(a.n.x_out, a.n.x_type, (long long)row * a.n.ldxo, i, 1, d, v);
        }
        if (a.n.out_type == WQ_NORM_OUT_NONE) continue;
        if (i < d) apply_norm<ACC>(pre, a.n.weight, a.n.bias, i, d, v);
        if (a.n.out_type == WQ_NORM_OUT_NVFP4) store_codes<kNVFP4>(a, row, i, v, ts, rcp6t);
        else if (a.n.out_type == WQ_NORM_OUT_MXFP4) store_codes<kMXFP4>(a, row, i, v, ts, rcp6t);
        else if (i < d) store8<ACC>(a.n.out, a.n.out_type == WQ_NORM_OUT_F32, (long long)row * a.n.ldo, i, 1, d, v);
    }
}

template <int TPR, int VPT>
cudaError_t launch_rows(const NormArgs& a, Access acc, cudaStream_t s) {
    constexpr unsigned kRows = TPR <= 32 ? 128 / TPR : 1;
    const unsigned blocks = ((unsigned)a.n.rows + kRows - 1) / kRows, threads = TPR <= 32 ? 128 : TPR;
    switch (acc) {
        case kVector: return launch_dependent(row_kernel<TPR, VPT, kVector>, blocks, threads, 1, 0, s, a);
        case kScalar: return launch_dependent(row_kernel<TPR, VPT, kScalar>, blocks, threads, 1, 0, s, a);
        default: return launch_dependent(row_kernel<TPR, VPT, kPieces>, blocks, threads, 1, 0, s, a);
    }
}

}  // namespace

int launch_block_norm(const wq_norm& n, cudaStream_t stream) {
    NormArgs a;
    a.n = n;
    a.inv_d = 1.0f / (float)n.d;
    a.rows_per_gate = n.gate ? n.rows / n.gate_rows : 1;
    const int group = n.out_type == WQ_NORM_OUT_NVFP4 ? 16 : 32;
    a.gblocks = (n.d / group + 3) / 4;
    // vector loads and stores: every row of every array 16-byte aligned
    auto ok = [](const void* p, long long ld, size_t es) {
        return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ((size_t)ld * es) % 16 == 0);
    };
    auto es = [](int type) { return type == WQ_TYPE_F32 ? (size_t)4 : (size_t)2; };
    const bool plain_out = n.out_type == WQ_NORM_OUT_BF16 || n.out_type == WQ_NORM_OUT_F32;
    const bool aligned = n.d % 8 == 0 && ok(n.x, n.ldx, es(n.x_type)) && ok(n.x_out, n.ldxo, es(n.x_type)) &&
                         ok(n.branch, n.ldb, es(n.branch_type)) && ok(n.gate, n.d, 2) && ok(n.weight, 0, 2) &&
                         ok(n.bias, 0, 2) && ok(n.post_weight, 0, 2) && ok(n.post_bias, 0, 2) &&
                         (!plain_out || ok(n.out, n.ldo, n.out_type == WQ_NORM_OUT_F32 ? 4 : 2));
    const int d = n.d;
    // (widths that are whole vectors keep the vectors' order of summation, so
    // a slice gives the bits that a copy of it gives)
    const Access acc = aligned ? kVector : d % 8 == 0 ? kPieces : kScalar;
    // one vector a thread up to 4096 elements, two beyond (and up to 512, where a
    // warp then has a row of its own and needs no barrier)
    cudaError_t e;
    const int vecs = (d + 7) / 8;
    // Many rows: at least eight for each thread's place on the device (the last
    // turn then idles an eighth of it at most); up to 512 elements a warp has a
    // row of its own and gains nothing.
    const bool streams = aligned && (!n.branch || n.branch_type == WQ_TYPE_BF16) && vecs > 64 && vecs <= 1024 &&
                         (long long)n.rows * vecs >= 8LL * 1024 * sm_count();
    if (streams)
        e = vecs <= 128   ? launch_stream<128, 1>(a, stream)
            : vecs <= 192 ? launch_stream<192, 1>(a, stream)
            : vecs <= 256 ? launch_stream<256, 1>(a, stream)
            : vecs <= 384 ? launch_stream<384, 1>(a, stream)
            : vecs <= 512 ? launch_stream<512, 1>(a, stream)
            : vecs <= 768 ? launch_stream<384, 2>(a, stream)
                          : launch_stream<512, 2>(a, stream);
    // short rows (a norm over each head), of which a warp takes up to eight, a
    // vector a lane: with a row a warp most lanes hold nothing (65536 x 64, bf16,
    // norm after the block: 25.3 us, 7.7 with eight lanes a row; x 128: 25.5, 13.9
    // with sixteen)
    else if (vecs <= 4) e = launch_rows<4, 1>(a, acc, stream);
    else if (vecs <= 8) e = launch_rows<8, 1>(a, acc, stream);
    else if (vecs <= 16) e = launch_rows<16, 1>(a, acc, stream);
    else if (vecs <= 32) e = launch_rows<32, 1>(a, acc, stream);
    else if (vecs <= 64) e = launch_rows<32, 2>(a, acc, stream);
    else if (vecs <= 128) e = launch_rows<128, 1>(a, acc, stream);
    else if (vecs <= 192) e = launch_rows<192, 1>(a, acc, stream);
    else if (vecs <= 256) e = launch_rows<256, 1>(a, acc, stream);
    else if (vecs <= 384) e = launch_rows<384, 1>(a, acc, stream);
    else if (vecs <= 512) e = launch_rows<512, 1>(a, acc, stream);
    else if (vecs <= 768) e = launch_rows<384, 2>(a, acc, stream);
    else if (vecs <= 1024) e = launch_rows<512, 2>(a, acc, stream);
    else if (vecs <= 2048) e = launch_rows<1024, 2>(a, acc, stream);
    else if (aligned) e = launch_dependent(row_loop_kernel<kVector>, (unsigned)n.rows, kLoopThreads, 1, 0, stream, a);
    else e = launch_dependent(row_loop_kernel<kPieces>, (unsigned)n.rows, kLoopThreads, 1, 0, stream, a);
    return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

}  // namespace wq
