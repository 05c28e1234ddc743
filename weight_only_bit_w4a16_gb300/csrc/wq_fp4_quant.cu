// wq_fp4_quant.cu -- rows of bf16 or fp32 to NVFP4 / MXFP4 codes and scales,
// and the re-ordering of row-major scales for the 4-bit product.
//
// The mathematics is in wq_fp4.cuh.  One thread takes 16 consecutive k of a
// row: one NVFP4 group, half an MXFP4 group (the neighbouring lane has the
// other half; one shuffle joins their maxima).  Everything is read once and
// written once; the bound is HBM.  16 per thread, so that the scale's ~25
// instructions are shared by 16 values: at the copy rate an SM has about 11
// issue slots for each bf16 value.
#include "wq_fp4.cuh"
#include "wq_internal.h"
#include "wq_tc.cuh"

namespace wq {

namespace {

// n / d for 0 <= n < 2^31 by one high multiply: with 2^l >= d the multiplier
// m = ceil(2^(31 + l) / d) is below 2^32 and exceeds 2^(31 + l) / d by less
// than 1, so n m / 2^(31 + l) exceeds n / d by less than n / 2^(31 + l) < 1 / d
// and the floor is the quotient.
struct FastDiv {
    uint32_t d, m, shift;
};

FastDiv fast_div(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    FastDiv f;
    f.d = d;
    f.shift = l;
    f.m = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
    return f;
}

__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
    return (uint32_t)(((uint64_t)n * f.m) >> (31 + f.shift));
}

struct QuantArgs {
    const void* x;
    const float* tensor_scale;
    uint8_t* packed;
    uint8_t* scales;
    uint16_t* values;   // bf16 image, or null
    long long ldx;      // elements between rows
    int row0;           // first row of this launch
    uint32_t units;     // rows * K / 16 of this launch
    FastDiv per_row;    // K / 16
    int K;
    int gblocks;        // tiled layout: ceil(groups / 4)
    int tiled;
};

// 16 consecutive values as fp32, and the largest bit pattern of |x|; the
// address is 16-byte aligned
template <typename T>
__device__ __forceinline__ uint32_t load16(const T* p, float (&v)[16]) {
    uint32_t top = 0;
    if constexpr (sizeof(T) == 2) {
        const uint4 a = ld_stream_v4(p), b = ld_stream_v4(p + 8);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        // |x| of bf16 pairs compare as unsigned 16-bit integers
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        }
        top = max(m << 16, m & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    return top;
}

// The same for rows of any alignment, by the whole warp: half a warp at a time
// loads one lane's 16 values, an element a lane, and they change places in
// shared memory (17 words a lane: no two lanes' words share a bank).  With each
// lane loading its own elements the loads of a warp fell in 16 to 32 different
// lines: 65536 x 2048 bf16 154 us, against 96 us aligned.
// p: this lane's values, null if it has none.
template <typename T>
__device__ __forceinline__ uint32_t load16_any(const T* p, float* stage, float (&v)[16]) {
    const int lane = threadIdx.x & 31, half = lane >> 4, e = lane & 15;
    float f[16];   // all loads first
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const T* q = reinterpret_cast<const T*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), 2 * i + half));
        f[i] = 0.0f;
        if (q) {
            if constexpr (sizeof(T) == 2) f[i] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(q)[e] << 16);
            else f[i] = q[e];
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) stage[(2 * i + half) * 17 + e] = f[i];
    __syncwarp();
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = stage[lane * 17 + i];
        top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    return top;
}

template <int FMT, typename T, bool ALIGNED, bool VALUES>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
    sm100::grid_dependency_wait();
    // No early start of dependents: what is written here may be a weight, and a
    // WQ_LAUNCH_OVERLAP call lets its own dependents start before its
    // predecessor has completed, so the call after it would read the weight
    // while it is being written.  (Costs a following product 0.5 to 0.9 us.)
    const uint32_t u = blockIdx.x * 256u + threadIdx.x;
    // MXFP4: units come in pairs of one group, so a lane and its partner are
    // both in range or both out of it; lanes out of range stay for the shuffle
    const bool live = u < a.units;
    const uint32_t lr = live ? div_by(u, a.per_row) : 0u;
    const uint32_t c = live ? u - lr * a.per_row.d : 0u;
    const int r = a.row0 + (int)lr;
    float v[16];
    uint32_t top = 0;
    const T* p = live ? static_cast<const T*>(a.x) + (long long)r * a.ldx + 16 * c : nullptr;
    if constexpr (ALIGNED) {
        if (live) top = load16<T>(p, v);
    } else {
        __shared__ float stage[8][32 * 17];
        top = load16_any<T>(p, stage[threadIdx.x >> 5], v);
    }
    if constexpr (FMT == kMXFP4) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (!live) return;
    float t = 1.0f, rcp6t = 1.0f / 6.0f;
    if (FMT == kNVFP4 && a.tensor_scale) {
        t = *a.tensor_scale;
        rcp6t = rcp_finite(6.0f * t);
    }
    const GroupScale g = group_scale<FMT>(top, t, rcp6t);
    const float(&v0)[8] = *reinterpret_cast<const float(*)[8]>(&v[0]);
    const float(&v1)[8] = *reinterpret_cast<const float(*)[8]>(&v[8]);
    const uint32_t c0 = quantize8<FMT>(v0, g), c1 = quantize8<FMT>(v1, g);
    const size_t e = (size_t)r * a.K + 16 * c;   // element
    *reinterpret_cast<uint2*>(a.packed + (e >> 1)) = make_uint2(c0, c1);
    if constexpr (VALUES) {
        uint4* o = reinterpret_cast<uint4*>(a.values + e);
        o[0] = values8(c0, g.step);
        o[1] = values8(c1, g.step);
    }
    if (FMT == kNVFP4 || !(c & 1)) {
        const int G = a.K / kGroupOf<FMT>;
        const int gi = FMT == kNVFP4 ? c : c >> 1;
        if (a.tiled) {
            uint8_t* p = a.scales + tiled_scale_offset(r, gi, a.gblocks);
            *p = (uint8_t)g.byte;
            // the row's last block of four: no group, scale 0
            if (gi == G - 1)
                for (int k = 1; (gi + k) & 3; ++k) p[k] = 0;
        } else {
            a.scales[(size_t)r * G + gi] = (uint8_t)g.byte;
        }
    }
}

template <int FMT, typename T>
cudaError_t launch_quant(const QuantArgs& a, bool aligned, unsigned blocks, cudaStream_t s) {
    if (aligned) {
        if (a.values) return launch_dependent(quantize_kernel<FMT, T, true, true>, blocks, 256, 1, 0, s, a);
        return launch_dependent(quantize_kernel<FMT, T, true, false>, blocks, 256, 1, 0, s, a);
    }
    if (a.values) return launch_dependent(quantize_kernel<FMT, T, false, true>, blocks, 256, 1, 0, s, a);
    return launch_dependent(quantize_kernel<FMT, T, false, false>, blocks, 256, 1, 0, s, a);
}

// One thread per four scales of a row (one 4-byte word of the tiled layout).
__global__ void __launch_bounds__(256)
    tile_scales_kernel(const uint8_t* __restrict__ in, uint8_t* __restrict__ out, int rows, int G, int gblocks,
                       long long words, uint32_t mask) {
    for (long long w = (long long)blockIdx.x * 256 + threadIdx.x; w < words; w += (long long)gridDim.x * 256) {
        const long long blk = w >> 7;
        const int in_blk = (int)(w & 127);
        const long long rb = blk / gblocks;
        const int gb = (int)(blk - rb * gblocks);
        const long long r = rb * 128 + (in_blk >> 2) + 32 * (in_blk & 3);
        uint32_t v = 0;
        if (r < rows) {
            const uint8_t* p = in + r * G + 4 * gb;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * gb + j < G) v |= (uint32_t)__ldg(p + j) << (8 * j);
        }
        reinterpret_cast<uint32_t*>(out)[w] = v & mask;
    }
}

}  // namespace

size_t fp4_scale_bytes(int rows, int K, int fmt, int tiled) {
    const size_t G = (size_t)K / (fmt == kNVFP4 ? 16 : 32);
    return tiled ? ((size_t)rows + 127) / 128 * ((G + 3) / 4) * 512 : (size_t)rows * G;
}

int launch_fp4_quantize(const void* x, bool x_f32, long long ldx, int rows, int K, int fmt, const float* tensor_scale,
                        uint8_t* packed, uint8_t* scales, bool tiled, void* values, cudaStream_t stream) {
    QuantArgs a;
    a.x = x;
    a.tensor_scale = tensor_scale;
    a.packed = packed;
    a.scales = scales;
    a.values = static_cast<uint16_t*>(values);
    a.ldx = ldx;
    a.K = K;
    a.gblocks = (K / (fmt == kNVFP4 ? 16 : 32) + 3) / 4;
    a.tiled = tiled ? 1 : 0;
    const uint32_t per_row = (uint32_t)K / 16;
    a.per_row = fast_div(per_row);
    const size_t es = x_f32 ? 4 : 2;
    const bool aligned = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ((size_t)ldx * es) % 16 == 0;
    // launches of fewer than 2^31 units (the index arithmetic's range)
    const int slab = (int)((0x7FFFFF00u / per_row) < (uint32_t)rows ? 0x7FFFFF00u / per_row : (uint32_t)rows);
    for (int r = 0; r < rows; r += slab) {
        const int n = rows - r < slab ? rows - r : slab;
        a.row0 = r;
        a.units = (uint32_t)n * per_row;
        const unsigned blocks = (a.units + 255) / 256;
        const cudaError_t e = fmt == kNVFP4 ? (x_f32 ? launch_quant<kNVFP4, float>(a, aligned, blocks, stream)
                                                     : launch_quant<kNVFP4, __nv_bfloat16>(a, aligned, blocks, stream))
                                            : (x_f32 ? launch_quant<kMXFP4, float>(a, aligned, blocks, stream)
                                                     : launch_quant<kMXFP4, __nv_bfloat16>(a, aligned, blocks, stream));
        if (e != cudaSuccess) return WQ_ERR_CUDA;
        if (n == rows - r) break;   // r + slab may pass the range of int
    }
    return WQ_OK;
}

int launch_fp4_tile_scales(const uint8_t* scales, uint8_t* tiled, int rows, int K, int fmt, cudaStream_t stream) {
    const int G = K / (fmt == kNVFP4 ? 16 : 32), gblocks = (G + 3) / 4;
    const long long words = (long long)(fp4_scale_bytes(rows, K, fmt, 1) / 4);
    long long blocks = (words + 255) / 256;
    if (blocks > 65536) blocks = 65536;
    // NVFP4 scales are used as |e4m3|; the matrix unit wants the sign bit 0
    const uint32_t mask = fmt == kNVFP4 ? 0x7F7F7F7Fu : 0xFFFFFFFFu;
    tile_scales_kernel<<<(unsigned)blocks, 256, 0, stream>>>(scales, tiled, rows, G, gblocks, words, mask);
    return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

}  // namespace wq
