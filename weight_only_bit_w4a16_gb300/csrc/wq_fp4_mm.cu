// wq_fp4_mm.cu -- C = A4 . B4^T, both operands microscaled 4-bit floats, on
// the block-scaled tcgen05 matrix instruction.
//
//   C[m, n] = f( t_A t_B sum_g s_A[m, g] s_B[n, g] sum_(k in g) a[m, k] b[n, k] )
//
// with e2m1 codes a, b, group scales s (NVFP4: e4m3 per 16 k, MXFP4: 2^E per
// 32 k), tensor scales t and the library's epilogue f.  The instruction takes
// the codes from shared memory and the scales from tensor memory and adds up
// in fp32; nothing is decoded in registers.
//
// Tile: 128 rows of one operand (P, the instruction's M) x bn rows of the
// other (Q, its N), k in steps of 256 (four instructions of 64).
//   * warp 0, one lane: TMA producer.  A stage is P's 128 x 128 bytes and Q's
//     bn x 128 bytes of codes (128-byte swizzle) and the two operands' scale
//     blocks, which are contiguous in the tiled scale order (512 bytes for
//     128 rows x 4 groups), so they come as plain bulk copies.
//   * warp 1, one lane: copies the stage's scale blocks to tensor memory (one
//     tcgen05.cp spreads a block's 32 x 16 bytes over the lanes) and issues
//     the stage's matrix instructions; tcgen05.commit frees the stage.
//   * warps 2..5: epilogue, accumulator to C.
// The instruction treats its two sides alike, so P can be either operand: the
// weights for few activation rows (P's 128 rows are then full and Q is as
// narrow as the activations), the activations otherwise (a thread then holds
// consecutive columns of C).
//
// Every wait is bounded; one that runs out records WQ_ERR_DEVICE_TIMEOUT, and
// the CTA unwinds.
#include <cstdio>
#include <cstdlib>

#include "wq_fp4.cuh"
#include "wq_internal.h"
#include "wq_tc.cuh"

namespace wq {

static __device__ int g_fp4_status = 0;

int read_and_clear_fp4_status() {
    int v = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_fp4_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_fp4_status, &zero, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
    return v;
}

namespace {

using namespace sm100;

constexpr int kP = 128;             // rows of P per tile
constexpr int kQMax = 256;          // rows of Q per tile at most
constexpr int kBK = 256;            // k per stage: 128 bytes of codes a row
constexpr int kStagesMax = 8;
constexpr int kThreads = 192;
constexpr int kPBytes = kP * 128;
constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s
constexpr uint64_t kDrainNs = 100000000ull;   // 0.1 s
constexpr size_t kMaxSmem = 227 * 1024;

template <int FMT>
constexpr int kChunkK = FMT == kNVFP4 ? 64 : 128;        // k of one scale block (four groups)
template <int FMT>
constexpr int kChunks = kBK / kChunkK<FMT>;              // scale blocks of a stage for 128 rows
template <int FMT>
constexpr int kScaleBytes = kChunks<FMT> * 512;

// Tensor memory: the accumulator in columns 0 .. bn - 1, then the scales of a
// stage: a block is 4 columns; P has kChunks blocks, Q twice as many (256
// rows).  Column of P's block q: kColP + 4 q; of Q's block q, rows 128 i ..:
// kColQ + 8 q + 4 i, so that Q's rows 32 j .. are column 8 q + j.
constexpr int kColP = 256;
constexpr int kColQ = 288;

struct MmArgs {
    const uint8_t* p_scales;
    const uint8_t* q_scales;
    const float* ta;     // tensor scales or null
    const float* tb;
    void* C;
    int M, N, K;
    int P, Q;            // rows of the two operands
    int bn;              // Q rows per tile, a multiple of 16
    int nt_p;            // tiles along P
    int nks;             // stages: ceil(K / 256)
    int chunks;          // scale blocks along K: ceil(K / kChunkK)
    int stages;
    int stage_bytes;
    int off_q, off_ps, off_qs;   // offsets in a stage
    uint32_t idesc;
    int swap;            // P is the weights
    int out_f32;
    int vec;             // C's rows 16-byte aligned (and the residual's)
    Epilogue epi;
};

struct __align__(8) MmShared {
    uint64_t full[kStagesMax];
    uint64_t empty[kStagesMax];
    uint64_t accfull;
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ void record_timeout() { atomicExch(&g_fp4_status, WQ_ERR_DEVICE_TIMEOUT); }

// D[tmem] (+)= A[smem] . B[smem]^T, e2m1 codes, 64 k, with the block scales in
// tensor memory: 16 k a scale (NVFP4) or 32 (MXFP4)
template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
    if constexpr (FMT == kNVFP4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
}

// 32 rows of 16 bytes in shared memory to 4 columns of all four lane quarters
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// descriptor of a scale block: no swizzle, 8-row groups of 16-byte rows 128
// bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1u << 46);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// 16 accumulator columns of this thread's lane, and the wait for them
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Instruction descriptor: e2m1 A and B, both K-major, fp32 accumulator, M =
// 128; bit 23: the scales' type, e8m0 or e4m3; the scale ids (bits 4 and 29)
// are added per instruction.
__host__ __device__ constexpr uint32_t idesc_fp4(int bn, bool e8m0) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(bn >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) | (1u << 27);
}

// Sixteen consecutive columns n .. n + 15 of row m (P the activations): gated,
// they are the 8 gate and 8 up values of 8 outputs.
__device__ __forceinline__ void store_cols(const MmArgs& a, int m, int n, float (&v)[16]) {
    if (a.epi.bias) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (n + i < a.N) v[i] += bf16_at(a.epi.bias, n + i);
    }
    int cnt = 16, o = n, ldc = a.N;
    if (a.epi.gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu_f32(v[i]) * v[8 + i];
        cnt = 8;
        o = n >> 1;
        ldc = a.N >> 1;
    }
    const size_t idx = (size_t)m * ldc + o;
    if (a.vec && o + cnt <= ldc) {
        if (a.epi.residual) {
            const uint4* r = reinterpret_cast<const uint4*>(a.epi.residual + idx);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (8 * h >= cnt) break;
                const uint4 q = __ldg(r + h);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[8 * h + 2 * i] += __uint_as_float(w[i] << 16);
                    v[8 * h + 2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
                }
            }
        }
        if (a.out_f32) {
            float4* c = reinterpret_cast<float4*>(static_cast<float*>(a.C) + idx);
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (4 * h < cnt) c[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
        } else {
            uint4* c = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.C) + idx);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (8 * h < cnt)
                    c[h] = make_uint4(bf16x2_of(v[8 * h], v[8 * h + 1]), bf16x2_of(v[8 * h + 2], v[8 * h + 3]),
                                      bf16x2_of(v[8 * h + 4], v[8 * h + 5]), bf16x2_of(v[8 * h + 6], v[8 * h + 7]));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i >= cnt || o + i >= ldc) continue;
        float y = v[i];
        if (a.epi.residual) y += bf16_at(a.epi.residual, idx + i);
        if (a.out_f32) static_cast<float*>(a.C)[idx + i] = y;
        else static_cast<__nv_bfloat16*>(a.C)[idx + i] = __float2bfloat16_rn(y);
    }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    mm_kernel(const __grid_constant__ CUtensorMap tmapP, const __grid_constant__ CUtensorMap tmapQ, const MmArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    MmShared& sh = *reinterpret_cast<MmShared*>(smem + a.stages * a.stage_bytes);
    volatile int* abort = &sh.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int p0 = (blockIdx.x % a.nt_p) * kP, q0 = (blockIdx.x / a.nt_p) * a.bn;

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        mbar_init(smem_u32(&sh.accfull), 1);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sh.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            if (a.nks > 0) {
                prefetch_tensormap(&tmapP);
                prefetch_tensormap(&tmapQ);
            }
            // scale blocks of 128 rows that exist in Q for this tile
            const int q_blocks = min((a.bn + 127) / 128, (a.Q - q0 + 127) / 128);
            int k = 0;
            for (; k < a.nks; ++k) {
                const int s = k % a.stages;
                if (!mbar_wait_bounded(smem_u32(&sh.empty[s]), ((k / a.stages) & 1) ^ 1, abort, kWaitNs)) {
                    record_timeout();
                    break;
                }
                const uint32_t st = smem_u32(smem + s * a.stage_bytes), fb = smem_u32(&sh.full[s]);
                const int c0 = k * kChunks<FMT>;
                const uint32_t sb = 512u * min(kChunks<FMT>, a.chunks - c0);   // bytes of a row block's scales
                mbar_arrive_expect_tx(fb, kPBytes + a.bn * 128 + sb * (1 + q_blocks));
                tma_load_2d(st, &tmapP, fb, k * 128, p0);
                tma_load_2d(st + a.off_q, &tmapQ, fb, k * 128, q0);
                bulk_load(st + a.off_ps, a.p_scales + ((size_t)(p0 / 128) * a.chunks + c0) * 512, sb, fb);
                for (int i = 0; i < q_blocks; ++i)
                    bulk_load(st + a.off_qs + i * kScaleBytes<FMT>,
                              a.q_scales + ((size_t)(q0 / 128 + i) * a.chunks + c0) * 512, sb, fb);
            }
            for (int j = k > a.stages ? k - a.stages : 0; j < k; ++j)   // no copy in flight past the CTA
                mbar_wait_timeout(smem_u32(&sh.full[j % a.stages]), (j / a.stages) & 1, kDrainNs);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const int q_blocks = (a.bn + 127) / 128;
            bool ok = true;
            for (int k = 0; k < a.nks; ++k) {
                const int s = k % a.stages;
                if (!mbar_wait_bounded(smem_u32(&sh.full[s]), (k / a.stages) & 1, abort, kWaitNs)) {
                    record_timeout();
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * a.stage_bytes);
                const int kleft = a.K - k * kBK;
                const uint64_t ps = scale_desc(st + a.off_ps), qs = scale_desc(st + a.off_qs);
#pragma unroll
                for (int c = 0; c < kChunks<FMT>; ++c) {
                    if (c * kChunkK<FMT> >= kleft) break;
                    cp_scales(tmem + kColP + 4 * c, ps + c * 32);
                    for (int i = 0; i < q_blocks; ++i)
                        cp_scales(tmem + kColQ + 8 * c + 4 * i, qs + (i * kChunks<FMT> + c) * 32);
                }
                const uint64_t pd = smem_desc_sw128_kmajor(st), qd = smem_desc_sw128_kmajor(st + a.off_q);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j * 64 >= kleft) break;
                    // MXFP4: a block serves two instructions, scale bytes 0, 1 and 2, 3
                    const int c = FMT == kNVFP4 ? j : j >> 1;
                    const uint32_t id = FMT == kNVFP4 ? 0u : (uint32_t)(j & 1) * 2u;
                    mma_fp4<FMT>(tmem, pd + 2 * j, qd + 2 * j, a.idesc | (id << 4) | (id << 29),
                                 tmem + kColP + 4 * c, tmem + kColQ + 8 * c, (k | j) ? 1u : 0u);
                }
                tc_commit(smem_u32(&sh.empty[s]));
            }
            if (ok) tc_commit(smem_u32(&sh.accfull));
            tc_commit(smem_u32(&sh.drain));
            mbar_wait_timeout(smem_u32(&sh.drain), 0, kDrainNs);
        }
    } else {
        const int q = warp & 3, row = q * 32 + lane;
        bool ok = true;
        if (a.nks > 0) ok = mbar_wait_bounded(smem_u32(&sh.accfull), 0, abort, kWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            tc_fence_after();
            const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
            float alpha = 1.0f;
            if (a.ta) alpha = __ldg(a.ta);
            if (a.tb) alpha *= __ldg(a.tb);
            for (int c = 0; c < a.bn; c += 16) {
                float v[16];
                if (a.nks > 0) {
                    tmem_ld16(lane_base + c, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= alpha;
                if (a.swap) {
                    const int n = p0 + row;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int m = q0 + c + i;
                        const float u = a.epi.gated ? __shfl_xor_sync(0xffffffffu, v[i], 8) : 0.0f;
                        if (m < a.M && n < a.N && !(a.epi.gated && (row & 8)))
                            store_epilogue(a.epi, a.C, a.out_f32, a.N, m, n, v[i], u);
                    }
                } else if (p0 + row < a.M && q0 + c < a.N) {
                    store_cols(a, p0 + row, q0 + c, v);
                }
            }
        } else if (lane == 0) {
            record_timeout();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

int launch_gemm_fp4(const Fp4Operand& A, const Fp4Operand& B, void* C, int M, int N, int K, int fmt, bool out_f32,
                    const Epilogue& epi, cudaStream_t stream) {
    MmArgs a{};
    a.swap = M <= 64;
    const Fp4Operand& P = a.swap ? B : A;
    const Fp4Operand& Q = a.swap ? A : B;
    a.P = a.swap ? N : M;
    a.Q = a.swap ? M : N;
    a.p_scales = P.scales;
    a.q_scales = Q.scales;
    a.ta = A.tensor_scale;
    a.tb = B.tensor_scale;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    a.bn = a.Q >= kQMax ? kQMax : (a.Q + 15) / 16 * 16;
    a.nt_p = (a.P + kP - 1) / kP;
    const long long tiles = (long long)a.nt_p * ((a.Q + a.bn - 1) / a.bn);
    if (tiles > 0x7FFFFFFF) return WQ_ERR_UNSUPPORTED;
    a.nks = (K + kBK - 1) / kBK;
    const int chunk_k = fmt == kNVFP4 ? 64 : 128, sbytes = kBK / chunk_k * 512;
    a.chunks = (K + chunk_k - 1) / chunk_k;
    a.off_q = kPBytes;
    a.off_ps = a.off_q + (a.bn * 128 + 1023) / 1024 * 1024;
    a.off_qs = a.off_ps + sbytes;
    a.stage_bytes = (a.off_qs + (a.bn + 127) / 128 * sbytes + 1023) / 1024 * 1024;
    const int fit = (int)((kMaxSmem - 1024 - sizeof(MmShared)) / a.stage_bytes);
    a.stages = fit < kStagesMax ? fit : kStagesMax;
    a.idesc = idesc_fp4(a.bn, fmt == kMXFP4);
    a.out_f32 = out_f32 ? 1 : 0;
    const int cols = epi.gated ? N / 2 : N;
    a.vec = cols % 8 == 0 && (!epi.residual || (reinterpret_cast<uintptr_t>(epi.residual) & 15) == 0);
    a.epi = epi;
    CUtensorMap tp, tq;
    if (K > 0) {
        if (!encode_2d(&tp, CU_TENSOR_MAP_DATA_TYPE_UINT8, P.packed, (uint64_t)K / 2, a.P, (uint64_t)K / 2, 128, kP,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, Q.packed, (uint64_t)K / 2, a.Q, (uint64_t)K / 2, 128, a.bn,
                       CU_TENSOR_MAP_SWIZZLE_128B))
            return WQ_ERR_UNSUPPORTED;
    } else {
        tp = CUtensorMap{};
        tq = CUtensorMap{};
    }
    const size_t smem = 1024 + (size_t)a.stages * a.stage_bytes + sizeof(MmShared);
    auto kern = fmt == kNVFP4 ? mm_kernel<kNVFP4> : mm_kernel<kMXFP4>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return WQ_ERR_CUDA;
    kern<<<(unsigned)tiles, kThreads, smem, stream>>>(tp, tq, a);
    return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

}  // namespace wq
