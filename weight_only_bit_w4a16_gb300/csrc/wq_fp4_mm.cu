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
// Two kernels:
//   * rows_kernel: P (the instruction's 128 rows) is the weights, Q (its N)
//     the activations.  For few activation rows, where the weights are what
//     has to be streamed: Q is as narrow as the activations, and where the
//     tiles would leave SMs idle a thread-block cluster shares a tile's k
//     steps and adds the partial sums up through distributed shared memory.
//
//   * pair_kernel: P is the activations, Q the weights, for many activation
//     rows.  Two CTAs of a cluster run one tile of 256 x bn: the instruction of
//     a CTA pair reads P's 256 rows and Q's bn rows half from either SM, so
//     an SM fetches 128 + bn / 2 rows for 128 x bn outputs.  One CTA alone
//     would fetch 384 rows for 128 x 256, and its copies alone took 440 ns a
//     stage against 270 ns of matrix instructions.
//
// What bounds it (8192^3, NVFP4, 152 SMs): the matrix pipe is 80 % busy, the
// scale copies run in it too (12 a stage, about 8 cycles each against 512 of
// products), and without any product the operands alone would take 143 of the
// 158 us, some 64 to 72 bytes a cycle into an SM.  Longer runs meet the power
// limit (1350 W, 1660 MHz): 178 us.  Small calls are a launch, about 2.4 us to
// the first stage, the stages, and 1 to 2 us of epilogue.
//
// Common to both: k in stages of 256 (128 bytes of codes a row, 128-byte
// swizzle; four instructions of 64 k).
//   * warp 0: TMA producer (one elected lane issues): a stage's codes, and its scale blocks,
//     which are contiguous in the tiled scale order (512 bytes for 128 rows x
//     4 groups).
//   * warp 1: copies the stage's scale blocks to tensor memory (one
//     tcgen05.cp spreads a block's 32 x 16 bytes over the lanes) and issues
//     the stage's matrix instructions; tcgen05.commit frees the stage.  The
//     copies and the instructions of one thread run in the order in which
//     they are issued, so one set of scale columns serves every stage.
//   * the other eight: epilogue, accumulator to C.
// Every wait is bounded, from the predecessor's completion on; one that runs out
// records WQ_ERR_DEVICE_TIMEOUT, and the CTA unwinds.
#include <atomic>
#include <cstdlib>
#include <cstring>
#include <unistd.h>

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

constexpr int kP = 128;             // rows of P per CTA
constexpr int kQMax = 256;          // rows of Q per tile at most
constexpr int kBK = 256;            // k per stage: 128 bytes of codes a row
constexpr int kStagesMax = 8;
constexpr int kThreads = 320;       // producer, issuer, eight epilogue warps
constexpr int kPBytes = kP * 128;
constexpr int kClusterMax = 8;      // the portable cluster size
constexpr int kSplitMax = kClusterMax / 2;   // (the sums below are written out for four)
constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s
constexpr uint64_t kDrainNs = 100000000ull;   // 0.1 s
constexpr uint64_t kLingerNs = 1000000ull;    // 1 ms
constexpr size_t kMaxSmem = 227 * 1024;

template <int FMT>
constexpr int kChunkK = FMT == kNVFP4 ? 64 : 128;        // k of one scale block (four groups)
template <int FMT>
constexpr int kChunks = kBK / kChunkK<FMT>;              // scale blocks of a stage for 128 rows
template <int FMT>
constexpr int kScaleBytes = kChunks<FMT> * 512;

struct RowsArgs {
    const uint8_t* p_scales;
    const uint8_t* q_scales;
    const float* ta;     // tensor scales or null
    const float* tb;
    void* C;
    int M, N, K;
    int bn;              // Q rows (activations) per tile, a multiple of 16
    int nt_p;            // tiles along P
    int nks;             // stages of a tile: ceil(K / 256)
    int chunks;          // scale blocks along K: ceil(K / kChunkK)
    int split;           // CTAs of the cluster that shares a tile's stages
    int stages;
    int stage_bytes;
    int off_q, off_ps, off_qs;   // offsets in a stage
    int tmem_cols;       // allocated: a power of two
    int col_p, col_q;    // tensor-memory columns of the scales: P's block q at col_p + 4 q, Q's at col_q + q_cols q
    int q_cols;
    uint32_t idesc;
    int out_f32;
    int ahead;           // the weights may be read before the predecessor has completed
    unsigned long long acc_wait_ns;   // bound of the epilogue's wait for the sums
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

// an element of the bias or the residual: a plain load, as they may be the
// predecessor's outputs (see ld_stream_v4)
__device__ __forceinline__ float epi_at(const uint16_t* p, size_t i) {
    return __uint_as_float((uint32_t)p[i] << 16);
}

// The tensor scales' product as the factors that the sums are multiplied by, one
// after the other: 1 and t_A t_B, or, where that product leaves the normal
// range although t_A t_B sum may be in it, t_A and t_B.
struct Factors {
    float first, second;
};

__device__ __forceinline__ Factors tensor_scales(const float* ta, const float* tb) {
    const float a = ta ? *ta : 1.0f, b = tb ? *tb : 1.0f, p = a * b, m = fabsf(p);
    const bool normal = m >= 0x1p-126f && m <= 0x1.fffffep127f;
    return normal ? Factors{1.0f, p} : Factors{a, b};
}

__device__ __forceinline__ void record_timeout() { atomicExch(&g_fp4_status, WQ_ERR_DEVICE_TIMEOUT); }

// A whole warp's wait for a phase, bounded in wall time; false, for all lanes,
// once it gave up or another warp of the CTA did.  The clock is read only
// after 32 failed tries (each of which may suspend the warp for a while).  A
// limit of 0 gives up at once (the host sets it only to run the failure path).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns = kWaitNs) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; limit_ns > 0; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 31) == 0) {
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (__any_sync(0xffffffffu, *abort != 0 || t - t0 > limit_ns)) break;
        }
    }
    *abort = 1;
    record_timeout();
    return false;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// The same wait where a test was made earlier: `ready` is its result.  The
// issuing warps test the next stage's barrier before they issue the current
// stage's work and ask for the result after it, so that a test's ~100 cycles
// are not on their path.  (A test, not a try: a try suspends the warp while
// the phase is open, which cost 4 us a call.)
__device__ __forceinline__ bool wait_warp_tried(bool ready, uint32_t bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, ready) || wait_warp(bar, parity, abort);
}

// A position in the stage ring: the stage and the parity of its use.  Kept by
// increments: a division by the run-time stage count is some 100 cycles, and
// the issuing warps' loops are the pipeline's critical path.
struct RingPos {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
};

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

// 64 accumulator columns and the wait for them
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// Instruction descriptor: e2m1 A and B, both K-major, fp32 accumulator, M =
// 128; bit 23: the scales' type, e8m0 or e4m3; the scale ids (bits 4 and 29)
// are added per instruction.
__host__ __device__ constexpr uint32_t idesc_fp4(int bn, bool e8m0) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(bn >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) | (1u << 27);
}

// ---------------------------------------------------------------------------
// pairs of CTAs
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                                 int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// each CTA's own shared memory to its own tensor memory
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// arrive on the barrier at this offset in both CTAs (their bits of the
// cluster's mask) once this thread's earlier tcgen05 operations have completed
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint32_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)mask) : "memory");
}
template <int FMT>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                             uint32_t sb, uint32_t accumulate) {
    if constexpr (FMT == kNVFP4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
}
// An arrival at a barrier of a CTA of the cluster (a shared::cluster address).
// What the pair hands over by its barriers is tensor memory and the ring's
// stages, never plain memory, so the tcgen05 fences and the copies' own
// completion order it: the arriving warp's loads of tensor memory have completed
// (tcgen05.wait::ld) and are fenced before the arrival, and the issuing warp
// fences after its wait.  A cluster-wide memory fence at the waits cost 0.8 us a
// tile.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
struct PairArgs {
    const float* ta;
    const float* tb;
    void* C;             // null: stored through the tensor map
    int out_f32, rows16; // SPLIT: C's type, and whether its rows are 16-byte multiples
    int split;           // SPLIT: pairs of a cluster
    int M, N, K;
    int bn;              // columns (weight rows) of a tile, a multiple of 64
    int nt_m, nt_n, tiles;
    int nks;
    int stages, stage_bytes;
    int off_q, off_ps, off_qs, off_stg;
    int q_blocks;        // 128-row scale blocks that a tile's columns can touch
    int acc1;            // column of the second accumulator
    int share;           // the accumulators share columns acc1 .. bn - 1
    uint32_t idesc;
    int tx_bytes;        // bytes of a stage, both CTAs
    int ahead;           // the weights may be read before the predecessor has completed
    int res_vec;         // the residual's rows are 16-byte aligned
    unsigned long long acc_wait_ns;   // bound of the epilogue's wait for the sums
    Epilogue epi;
};

// Scale columns of tensor memory: P's block q at kPairColP + 4 q, Q's two at
// kPairColQ + 8 q (rows 32 j .. of the two are column j).
constexpr int kPairColP = 448;
constexpr int kPairColQ = 464;
constexpr int kBand = 8;             // tiles along M that run together (see pair_tile)
constexpr int kStgWarp = 4096;       // staging of an epilogue warp: a box of 32 rows of at most 128 bytes

struct __align__(8) PairShared {
    uint64_t full[kStagesMax];
    uint64_t empty[kStagesMax];
    uint64_t accfull[2];    // one per accumulator
    uint64_t accempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// Tiles in bands of kBand along M, along N within a band: the tiles that run
// at a time then share both operands' rows.
__device__ __forceinline__ void pair_tile(const PairArgs& a, int t, int& tm, int& tn) {
    const int per = kBand * a.nt_n, band = t / per, r = t - band * per;
    const int h = min(kBand, a.nt_m - band * kBand);
    tm = band * kBand + r % h;
    tn = r / h;
}

// x / (1 + e^-x): of large negative x 0, as the reciprocal of 1 + e^-x is
// flushed to it below 2^-126 (past -87.3; the result there is under 89 2^-126 in
// magnitude); of -inf NaN, as of the quotient itself.  EXACT, for fp32 output:
// the rounding error of the power of two's exponent is put back to first order
// and the approximate reciprocal gets a Newton step, which need a finite
// exponential (hence the bounds of y); largest relative error over |x| <= 86,
// against 64 bits at 4 million points, 2^-21.7.  Otherwise neither: 2^-18.0
// (2^-19.9 for |x| <= 20), 1/500 of bf16's rounding: the gated 128 x 16384 x
// 3072 took 9.0 us for 9.7, 2048 x 16384 x 3072 39 for 45.  Without the
// instructions' scaling of subnormal numbers they take 8.9 and 36, the latter
// with fp32 output 44 for 47.
template <bool EXACT>
__device__ __forceinline__ float silu_short(float x) {
    constexpr float kLog2e = 1.44269504088896340736f, kLog2eLo = 1.92596299112661746887e-8f;
    constexpr float kLn2 = 0.693147180559945309417f;
    const float y = EXACT ? fminf(fmaxf(-x, -88.5f), 88.5f) : -x;
    const float t = y * kLog2e;
    float e, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    if constexpr (EXACT) e = fmaf(e * kLn2, fmaf(y, kLog2eLo, fmaf(y, kLog2e, -t)), e);
    const float d = 1.0f + e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(d));
    if constexpr (EXACT) q = fmaf(q, fmaf(-d, q, 1.0f), q);   // (0 stays 0)
    return x * q;
}

// 32 accumulator columns n .. of one row to outputs, in place: alpha, bias, gate
// (outputs v[0 .. 15] then), residual.
template <bool F32, bool GATED>
__device__ __forceinline__ void pair_epilogue(const PairArgs& a, const Factors& alpha, int m, int n, float (&v)[32]) {
    if (alpha.first != 1.0f) {   // (rare)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= alpha.first;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= alpha.second;
    if (a.epi.bias) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (n + i < a.N) v[i] += epi_at(a.epi.bias, n + i);
    }
    constexpr int kOut = GATED ? 16 : 32;
    if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float lo = silu_short<F32>(v[i]) * v[8 + i], hi = silu_short<F32>(v[16 + i]) * v[24 + i];
            v[i] = lo;
            v[8 + i] = hi;
        }
    }
    if (a.epi.residual && m < a.M) {
        const int cols = GATED ? a.N >> 1 : a.N, o = GATED ? n >> 1 : n;
        const size_t idx = (size_t)m * cols + o;
        if (a.res_vec && o + kOut <= cols) {
            const uint4* r = reinterpret_cast<const uint4*>(a.epi.residual + idx);
#pragma unroll
            for (int h = 0; h < kOut / 8; ++h) {
                const uint4 q = r[h];
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[8 * h + 2 * i] += __uint_as_float(w[i] << 16);
                    v[8 * h + 2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kOut; ++i)
                if (o + i < cols) v[i] += epi_at(a.epi.residual, idx + i);
        }
    }
}

// Sixteen accumulator columns n .. of 32 rows to C, a lane's row m; the whole
// warp calls it.  Where a lane's outputs are not whole vectors they go through
// the warp's staging, so that a store covers whole runs of rows (129 x 89 x
// 7392: a lane storing its own row took 4 us more).
__device__ __forceinline__ void store_cols(const PairArgs& a, const Factors& alpha, int m, int n, float (&v)[16], float* stg) {
    const bool live = m < a.M;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = v[i] * alpha.first * alpha.second;
        if (a.epi.bias && n + i < a.N) v[i] += epi_at(a.epi.bias, n + i);
    }
    const int cols = a.epi.gated ? a.N >> 1 : a.N, o = a.epi.gated ? n >> 1 : n, cnt = a.epi.gated ? 8 : 16;
    if (a.epi.gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu_short<true>(v[i]) * v[8 + i];
    }
    const size_t idx = (size_t)m * cols + o;
    if (a.epi.residual && live) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < cnt && o + i < cols) v[i] += epi_at(a.epi.residual, idx + i);
    }
    if (a.rows16 && o + cnt <= cols) {
        if (!live) return;
        if (a.out_f32) {
            float* c = static_cast<float*>(a.C) + idx;
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (i < cnt) *reinterpret_cast<float4*>(c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
            __nv_bfloat16* c = static_cast<__nv_bfloat16*>(a.C) + idx;
#pragma unroll
            for (int i = 0; i < 16; i += 8)
                if (i < cnt)
                    *reinterpret_cast<uint4*>(c + i) = make_uint4(bf16x2_of(v[i], v[i + 1]), bf16x2_of(v[i + 2], v[i + 3]),
                                                                  bf16x2_of(v[i + 4], v[i + 5]), bf16x2_of(v[i + 6], v[i + 7]));
        }
        return;
    }
    constexpr int kLd = 17;   // floats of a staged row: no two lanes in a bank
    const int lane = threadIdx.x & 31, col = lane & (cnt - 1), m0 = m - lane;
    __syncwarp();   // the piece before this one has been read
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < cnt) stg[lane * kLd + i] = v[i];
    __syncwarp();
    if (o + col >= cols) return;
    const int rows = min(32, a.M - m0), per = 32 / cnt;
    size_t at = (size_t)(m0 + lane / cnt) * cols + o + col;
#pragma unroll 4
    for (int r = lane / cnt; r < rows; r += per, at += (size_t)per * cols) {
        const float y = stg[r * kLd + col];
        if (a.out_f32) static_cast<float*>(a.C)[at] = y;
        else static_cast<__nv_bfloat16*>(a.C)[at] = __float2bfloat16_rn(y);
    }
}

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// SPLIT: the tile's stages are shared by the a.split pairs of one cluster, each
// with a contiguous part; they add their partial sums up through distributed
// shared memory, in pair order, and each stores a share of the tile (F32 and
// GATED are not used).  One tile a cluster.
template <int FMT, bool F32, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmapP, const __grid_constant__ CUtensorMap tmapQ,
                const __grid_constant__ CUtensorMap tmapPS, const __grid_constant__ CUtensorMap tmapQS,
                const __grid_constant__ CUtensorMap tmapC, const PairArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PairShared& sh = *reinterpret_cast<PairShared*>(smem + a.off_stg + 8 * kStgWarp);
    volatile int* abort = &sh.abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // place in the pair, and the leader's rank in the cluster
    const int crank = (int)cluster_ctarank(), rank = crank & 1, lead = crank & ~1;
    const uint32_t mask = 3u << lead;
    // this pair's tiles, and its stages of each
    const int part = SPLIT ? crank >> 1 : 0;
    const int pair = SPLIT ? blockIdx.x / (2 * a.split) : blockIdx.x >> 1, pairs = SPLIT ? a.tiles : gridDim.x >> 1;
    const int k0 = SPLIT ? (int)((long long)part * a.nks / a.split) : 0;
    const int k1 = SPLIT ? (int)((long long)(part + 1) * a.nks / a.split) : a.nks;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmapP);
        prefetch_tensormap(&tmapQ);
        prefetch_tensormap(&tmapPS);
        prefetch_tensormap(&tmapQS);
        if (!a.C) prefetch_tensormap(&tmapC);
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sh.accfull[b]), 1);
            mbar_init(smem_u32(&sh.accempty[b]), 16);   // the eight epilogue warps of either CTA
        }
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&sh.tmem_base), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // the other CTA's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);

    if (warp == 0) {
        // ---- producer: this CTA's 128 rows of P and its half of Q; all copies
        // of the pair complete on the leader's (rank 0) barrier
        const uint32_t base = smem_u32(smem), empty = smem_u32(&sh.empty[0]), full = smem_u32(&sh.full[0]);
        const uint32_t lfull = mapa_shared(full, lead);
        auto load_q = [&](int k, int s, int q0) {   // one lane
            const uint32_t st = base + s * a.stage_bytes, fb = lfull + 8 * s;
            if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, a.tx_bytes);
            tma_load_2d_pair(st + a.off_q, &tmapQ, fb, k * 128, q0 + rank * (a.bn >> 1));
            tma_load_3d_pair(st + a.off_qs, &tmapQS, fb, 0, k * kChunks<FMT>, q0 >> 7);
        };
        // weights of the ring's first fill, ahead of the dependency
        int early = 0;
        if (a.ahead) {
            int tm, tn;
            pair_tile(a, pair, tm, tn);
            early = min(k1 - k0, a.stages);
            for (int k = 0; k < early; ++k) {
                if (elect_one()) load_q(k0 + k, k, tn * a.bn);
                __syncwarp();
            }
        }
        grid_dependency_wait();
        grid_dependents_launch();
        int g = 0;
        RingPos pos;
        bool ok = true, ready = true;   // the ring starts empty
        for (int t = pair; ok && t < a.tiles; t += pairs) {
            int tm, tn;
            pair_tile(a, t, tm, tn);
            const int p0 = tm * 256 + rank * kP, q0 = tn * a.bn;
            for (int k = k0; k < k1; ++k, ++g) {
                if (!wait_warp_tried(ready, empty + 8 * pos.s, pos.parity ^ 1, abort)) {
                    ok = false;
                    break;
                }
                const uint32_t st = base + pos.s * a.stage_bytes, fb = lfull + 8 * pos.s;
                RingPos next = pos;
                next.next(a.stages);
                ready = mbar_test(empty + 8 * next.s, next.parity ^ 1);
                if (elect_one()) {
                    if (g >= early) load_q(k, pos.s, q0);
                    tma_load_2d_pair(st, &tmapP, fb, k * 128, p0);
                    tma_load_3d_pair(st + a.off_ps, &tmapPS, fb, 0, k * kChunks<FMT>, p0 >> 7);
                }
                __syncwarp();
                pos = next;
            }
        }
        // No copy in flight past the pair: all of them complete here.  After a
        // wait gave up the other CTA may have issued fewer, and it has no
        // barrier of its own to ask: a millisecond covers any copy.
        if (rank == 0) {
            for (int j = g > a.stages ? g - a.stages : 0; j < g; ++j)
                mbar_wait_timeout(smem_u32(&sh.full[j % a.stages]), (j / a.stages) & 1, ok ? kDrainNs : kLingerNs);
        } else if (!ok) {
            for (const uint64_t t = globaltimer_ns(); globaltimer_ns() - t < kLingerNs;) __nanosleep(1000);
        }
    } else if (warp == 1) {
        // ---- matrix instructions: the leader issues them for both CTAs
        if (rank == 0) {
            grid_dependency_wait();   // (the bounds of the waits begin here)
            const uint32_t base = smem_u32(smem), empty = smem_u32(&sh.empty[0]), full = smem_u32(&sh.full[0]);
            const uint32_t cq = tmem + kPairColQ;
            int i = 0;
            RingPos pos;
            bool ok = true, ready = false;
            for (int t = pair; ok && t < a.tiles; t += pairs, ++i) {
                int tm, tn;
                pair_tile(a, t, tm, tn);
                const uint32_t shift = (uint32_t)(tn * a.bn & 127) >> 5;   // the tile's first row in its scale block
                const uint32_t acc = tmem + ((i & 1) ? a.acc1 : 0);
                // The accumulator is free: apart, once the tile before last has
                // been read; where the two share columns, once the last one has
                // been read so far (see the epilogue).
                const int w = i - (a.share ? 1 : 2);
                if (w >= 0 && !wait_warp(smem_u32(&sh.accempty[w & 1]), (w >> 1) & 1, abort)) break;
                tc_fence_after();
                for (int k = k0; k < k1; ++k) {
                    if (!wait_warp_tried(ready, full + 8 * pos.s, pos.parity, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = base + pos.s * a.stage_bytes, eb = empty + 8 * pos.s;
                    RingPos next = pos;
                    next.next(a.stages);
                    ready = mbar_test(full + 8 * next.s, next.parity);
                    const int kleft = a.K - k * kBK;
                    const uint64_t ps = scale_desc(st + a.off_ps), qs = scale_desc(st + a.off_qs);
                    const uint64_t pd = smem_desc_sw128_kmajor(st), qd = smem_desc_sw128_kmajor(st + a.off_q);
                    if (elect_one()) {
#pragma unroll
                        for (int c = 0; c < kChunks<FMT>; ++c) {
                            cp_scales_pair(tmem + kPairColP + 4 * c, ps + c * 32);
                            cp_scales_pair(cq + 8 * c, qs + c * 32);
                            if (a.q_blocks > 1) cp_scales_pair(cq + 8 * c + 4, qs + (kChunks<FMT> + c) * 32);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j * 64 >= kleft) break;
                            const int c = FMT == kNVFP4 ? j : j >> 1;
                            const uint32_t id = FMT == kNVFP4 ? 0u : (uint32_t)(j & 1) * 2u;
                            mma_fp4_pair<FMT>(acc, pd + 2 * j, qd + 2 * j, a.idesc | (id << 4) | (id << 29),
                                              tmem + kPairColP + 4 * c, cq + 8 * c + shift,
                                              (k > k0 || j) ? 1u : 0u);
                        }
                        tc_commit_pair(eb, mask);
                        if (k == k1 - 1) tc_commit_pair(smem_u32(&sh.accfull[i & 1]), mask);
                    }
                    __syncwarp();
                    pos = next;
                }
            }
            if (elect_one()) tc_commit_pair(smem_u32(&sh.drain), mask);
            __syncwarp();
            mbar_wait_timeout(smem_u32(&sh.drain), 0, kDrainNs);
        }
    } else if constexpr (!SPLIT) {
        // ---- epilogue: this CTA's 128 rows of the tile, a warp's 32 rows at a
        // time through its own staging boxes (128-byte swizzle) and one bulk
        // tensor store a box
        constexpr int kOut = GATED ? 32 : 64;                       // outputs of 64 accumulator columns
        constexpr int kRowBytes = GATED && !F32 ? 64 : 128;         // a box row, and its swizzle
        constexpr int kBoxCols = kRowBytes / (F32 ? 4 : 2);         // 32, 64 or (gated bf16) 32
        const int q = warp & 3, set = (warp - 2) >> 2;   // lane quarter; which of the 64-column pieces
        const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
        uint8_t* buf = smem + a.off_stg + (warp - 2) * kStgWarp;
        const uint32_t release0 = mapa_shared(smem_u32(&sh.accempty[0]), lead), accfull = smem_u32(&sh.accfull[0]);
        grid_dependency_wait();   // C, the tensor scales and the residual may be the predecessor's
        const Factors alpha = tensor_scales(a.ta, a.tb);
        const int ncols = GATED ? a.N >> 1 : a.N;
        int i = 0;
        for (int t = pair; t < a.tiles; t += pairs, ++i) {
            int tm, tn;
            pair_tile(a, t, tm, tn);
            if (!wait_warp(accfull + 8 * (i & 1), (i >> 1) & 1, abort, a.acc_wait_ns)) break;
            tc_fence_after();
            const int m0 = tm * 256 + rank * kP + q * 32, n0 = tn * a.bn;
            const uint32_t acc = lane_base + ((i & 1) ? a.acc1 : 0);
            const int nc = a.bn >> 6;
            const uint32_t release = release0 + 8 * (i & 1);
            // Accumulators apart: this one is free once every warp has read
            // its pieces.  Accumulators that share columns (acc1 .. bn - 1, at
            // most 64: the first one's last, the second one's first): the next
            // tile's instructions may start once those have been read, which
            // are set 0's first piece, and every warp is here, done with the
            // tile before this one.
            bool held = true;
            if (set >= nc || (a.share && set != 0)) {
                held = false;
                tc_fence_before();   // its loads of the tile before this one have completed (wait::ld)
                if (lane == 0) mbar_arrive_cluster(release);
            }
            for (int b = set; b < nc; b += 2) {
                const int c = ((i & 1) ? b : nc - 1 - b) * 64;
                float v[64];
                tmem_ld64(acc + c, v);
                if (held && (a.share || b + 2 >= nc)) {
                    held = false;
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_cluster(release);
                }
                float(&lo)[32] = *reinterpret_cast<float(*)[32]>(&v[0]);
                float(&hi)[32] = *reinterpret_cast<float(*)[32]>(&v[32]);
                pair_epilogue<F32, GATED>(a, alpha, m0 + lane, n0 + c, lo);
                pair_epilogue<F32, GATED>(a, alpha, m0 + lane, n0 + c + 32, hi);
                // outputs kOut of this row: v[0 ..], and gated v[32 ..] for the second half
                const int o0 = (GATED ? n0 >> 1 : n0) + (GATED ? c >> 1 : c);
#pragma unroll
                for (int x = 0; x < kOut / kBoxCols; ++x) {
                    if (lane == 0) bulk_wait_read0();   // the box before this one has left
                    __syncwarp();
                    uint8_t* rowp = buf + lane * kRowBytes;
                    // 16-byte unit u of a row sits at u ^ (row mod 8), or in 64-byte rows u ^ (row / 2 mod 4)
                    const int xr = kRowBytes == 128 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
                    for (int u = 0; u < kRowBytes / 16; ++u) {
                        constexpr int kPer = F32 ? 4 : 8;   // outputs of a unit
                        float w[kPer];
#pragma unroll
                        for (int e = 0; e < kPer; ++e) {
                            const int o = x * kBoxCols + u * kPer + e;
                            w[e] = GATED ? (o < 16 ? v[o] : v[32 + o - 16]) : v[o];
                        }
                        uint4 pk;
                        if constexpr (F32)
                            pk = make_uint4(__float_as_uint(w[0]), __float_as_uint(w[1]), __float_as_uint(w[2]),
                                            __float_as_uint(w[3]));
                        else
                            pk = make_uint4(bf16x2_of(w[0], w[1]), bf16x2_of(w[2], w[3]), bf16x2_of(w[4], w[5]),
                                            bf16x2_of(w[6], w[7]));
                        *reinterpret_cast<uint4*>(rowp + ((u ^ xr) << 4)) = pk;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    const int oc = o0 + x * kBoxCols;
                    if (a.C == nullptr) {
                        if (lane == 0) {
                            if (m0 < a.M && oc < ncols) tma_store_2d(&tmapC, smem_u32(buf), oc, m0);
                            bulk_commit();
                        }
                    } else {
                        // C's rows are not 16-byte multiples: the warp stores
                        // a row of the box at a time, four in flight (460 x
                        // 15717 x 1504: bf16 14.4 us, fp32 19.3; 16.0 and 23.4
                        // one by one; eight took 13.9 and 18.7, but their code
                        // cost aligned rows 1 %)
                        __syncwarp();
                        constexpr int kEs = F32 ? 4 : 2;
                        const int live = min(32, a.M - m0);
                        const size_t step = (size_t)ncols * kEs;
                        const int by = lane * kEs, unit = by >> 4;
                        uint8_t* dst = static_cast<uint8_t*>(a.C) + ((size_t)m0 * ncols + oc) * kEs + by;
                        const uint8_t* src = buf + (by & 15);
#pragma unroll 4
                        for (int rr = 0; rr < 32; ++rr) {
                            const int rx = kRowBytes == 128 ? rr & 7 : (rr >> 1) & 3;
#pragma unroll
                            for (int h = 0; h < kBoxCols; h += 32) {
                                const uint8_t* from = src + rr * kRowBytes + (((unit + h * kEs / 16) ^ rx) << 4);
                                if (rr < live && oc + h + lane < ncols) {
                                    if constexpr (F32)
                                        *reinterpret_cast<uint32_t*>(dst + h * kEs) = *reinterpret_cast<const uint32_t*>(from);
                                    else
                                        *reinterpret_cast<uint16_t*>(dst + h * kEs) = *reinterpret_cast<const uint16_t*>(from);
                                }
                            }
                            dst += step;
                        }
                        __syncwarp();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait0();
        __syncwarp();
    }
    if constexpr (SPLIT) {
        const int w = warp - 2, q = warp & 3;
        // over the ring: [column][128 rows], so that a warp's remote load is one
        // run of 128 bytes ([row][column] with 16-byte loads was 1 to 5 us slower)
        float* sums = reinterpret_cast<float*>(smem);
        bool ok = true;
        Factors alpha{1.0f, 1.0f};
        int tm, tn;
        pair_tile(a, pair, tm, tn);
        if (warp >= 2) {
            grid_dependency_wait();
            alpha = tensor_scales(a.ta, a.tb);
            ok = wait_warp(smem_u32(&sh.accfull[0]), 0, abort, a.acc_wait_ns);
            tc_fence_after();
            if (ok) {
                const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
                for (int c = (w >> 2) * 64; c < a.bn; c += 128) {
                    float v[64];
                    tmem_ld64(acc + c, v);
#pragma unroll
                    for (int e = 0; e < 64; ++e) sums[(c + e) * kP + q * 32 + lane] = v[e];
                }
            }
        }
        cluster_sync_all();
        if (warp >= 2) {
            // pieces of 16 columns x 32 rows, dealt to the pairs' warps
            float* stg = reinterpret_cast<float*>(smem + a.off_stg + w * kStgWarp);
            uint32_t src[kSplitMax];
#pragma unroll
            for (int p = 0; p < kSplitMax; ++p)
                src[p] = p < a.split ? mapa_shared(smem_u32(sums), (uint32_t)(2 * p + rank)) : 0u;
            for (int u = part * 8 + w; u < a.bn >> 2; u += a.split * 8) {
                const int c = (u >> 2) * 16, r = (u & 3) * 32 + lane, m = tm * 256 + rank * kP + r, n = tn * a.bn + c;
                if (tm * 256 + rank * kP + (u & 3) * 32 >= a.M || n >= a.N) continue;
                const uint32_t at = (uint32_t)(c * kP + r) * 4u;
                float x[kSplitMax][16];   // all loads first
#pragma unroll
                for (int p = 0; p < kSplitMax; ++p)
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[p][e] = p < a.split ? ld_dsmem_f32(src[p] + at + 512u * e) : 0.0f;
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = ((x[0][e] + x[1][e]) + x[2][e]) + x[3][e];   // pair order
                if (ok) store_cols(a, alpha, m, n, v, stg);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // neither CTA's memory goes while the pair's instructions may use it
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------------------
// few activation rows
// ---------------------------------------------------------------------------
template <int FMT>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const __grid_constant__ CUtensorMap tmapP, const __grid_constant__ CUtensorMap tmapQ,
                const RowsArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    MmShared& sh = *reinterpret_cast<MmShared*>(smem + a.stages * a.stage_bytes);
    volatile int* abort = &sh.abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = a.split > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / a.split;
    const int p0 = (tile % a.nt_p) * kP, q0 = (tile / a.nt_p) * a.bn;
    // this CTA's share of the tile's stages
    const int k0 = (int)((long long)rank * a.nks / a.split), k1 = (int)((long long)(rank + 1) * a.nks / a.split);
    const int nk = k1 - k0;

    if (threadIdx.x == 0) {
        if (a.nks > 0) {
            prefetch_tensormap(&tmapP);
            prefetch_tensormap(&tmapQ);
        }
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
        tmem_alloc(smem_u32(&sh.tmem_base), a.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);

    if (warp == 0) {
        if (nk > 0) {
            // scale blocks of 128 rows that exist in Q for this tile
            const int q_blocks = min((a.bn + 127) / 128, (a.M - q0 + 127) / 128);
            const uint32_t base = smem_u32(smem), empty = smem_u32(&sh.empty[0]), full = smem_u32(&sh.full[0]);
            auto load_p = [&](int k, int s) {
                const int ks = k0 + k, c0 = ks * kChunks<FMT>;
                const uint32_t st = base + s * a.stage_bytes, fb = full + 8 * s;
                const uint32_t sb = 512u * min(kChunks<FMT>, a.chunks - c0);   // bytes of a row block's scales
                const uint8_t* src = a.p_scales + ((size_t)(p0 / 128) * a.chunks + c0) * 512;
                if (elect_one()) {
                    mbar_arrive_expect_tx(fb, kPBytes + a.bn * 128 + sb * (1 + q_blocks));
                    tma_load_2d(st, &tmapP, fb, ks * 128, p0);
                    bulk_load(st + a.off_ps, src, sb, fb);
                }
                __syncwarp();
            };
            auto load_q = [&](int k, int s) {
                const int ks = k0 + k, c0 = ks * kChunks<FMT>;
                const uint32_t st = base + s * a.stage_bytes, fb = full + 8 * s;
                const uint32_t sb = 512u * min(kChunks<FMT>, a.chunks - c0);
                const uint8_t* src = a.q_scales + ((size_t)(q0 / 128) * a.chunks + c0) * 512;
                if (elect_one()) {
                    tma_load_2d(st + a.off_q, &tmapQ, fb, ks * 128, q0);
                    bulk_load(st + a.off_qs, src, sb, fb);
                    if (q_blocks > 1) bulk_load(st + a.off_qs + kScaleBytes<FMT>, src + (size_t)a.chunks * 512, sb, fb);
                }
                __syncwarp();
            };
            // the ring's first fill; the weights' copies ahead of the
            // dependency where the caller allows it
            const int fill = min(nk, a.stages);
            if (a.ahead)
                for (int k = 0; k < fill; ++k) load_p(k, k);
            grid_dependency_wait();
            grid_dependents_launch();
            for (int k = 0; k < fill; ++k) {
                if (!a.ahead) load_p(k, k);
                load_q(k, k);
            }
            int k = fill;
            RingPos pos;
            for (; k < nk; ++k) {
                if (!wait_warp(empty + 8 * pos.s, pos.parity, abort)) break;
                load_p(k, pos.s);
                load_q(k, pos.s);
                pos.next(a.stages);
            }
            for (int j = k > a.stages ? k - a.stages : 0; j < k; ++j)   // no copy in flight past the CTA
                mbar_wait_timeout(smem_u32(&sh.full[j % a.stages]), (j / a.stages) & 1, kDrainNs);
        }
    } else if (warp == 1) {
        grid_dependency_wait();   // (the bounds of the waits begin here)
        const int q_blocks = (a.bn + 127) / 128;
        const uint32_t base = smem_u32(smem), empty = smem_u32(&sh.empty[0]), full = smem_u32(&sh.full[0]);
        RingPos pos;
        for (int k = 0; k < nk; ++k) {
            if (!wait_warp(full + 8 * pos.s, pos.parity, abort)) break;
            tc_fence_after();
            const uint32_t st = base + pos.s * a.stage_bytes, eb = empty + 8 * pos.s;
            const int kleft = a.K - (k0 + k) * kBK;
            const uint64_t ps = scale_desc(st + a.off_ps), qs = scale_desc(st + a.off_qs);
            const uint64_t pd = smem_desc_sw128_kmajor(st), qd = smem_desc_sw128_kmajor(st + a.off_q);
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < kChunks<FMT>; ++c) {
                    if (c * kChunkK<FMT> >= kleft) break;
                    cp_scales(tmem + a.col_p + 4 * c, ps + c * 32);
                    cp_scales(tmem + a.col_q + a.q_cols * c, qs + c * 32);
                    if (q_blocks > 1) cp_scales(tmem + a.col_q + a.q_cols * c + 4, qs + (kChunks<FMT> + c) * 32);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j * 64 >= kleft) break;
                    // MXFP4: a block serves two instructions, scale bytes 0, 1 and 2, 3
                    const int c = FMT == kNVFP4 ? j : j >> 1;
                    const uint32_t id = FMT == kNVFP4 ? 0u : (uint32_t)(j & 1) * 2u;
                    mma_fp4<FMT>(tmem, pd + 2 * j, qd + 2 * j, a.idesc | (id << 4) | (id << 29),
                                 tmem + a.col_p + 4 * c, tmem + a.col_q + a.q_cols * c, (k | j) ? 1u : 0u);
                }
                tc_commit(eb);
                if (k == nk - 1) tc_commit(smem_u32(&sh.accfull));
            }
            __syncwarp();
            pos.next(a.stages);
        }
        // every instruction has completed before the CTA tears down
        if (elect_one()) {
            if (nk == 0) tc_commit(smem_u32(&sh.accfull));
            tc_commit(smem_u32(&sh.drain));
        }
        __syncwarp();
        mbar_wait_timeout(smem_u32(&sh.drain), 0, kDrainNs);
    }
    // the epilogue's warps (a failure does not leave the path to the barriers)
    const int w = warp - 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    const int live = min(a.bn, a.M - q0);   // columns that are rows of C
    bool ok = true;
    Factors alpha{1.0f, 1.0f};
    if (warp >= 2) {
        grid_dependency_wait();   // C, the tensor scales and the residual may be the predecessor's
        ok = wait_warp(smem_u32(&sh.accfull), 0, abort, a.acc_wait_ns);
        tc_fence_after();
        alpha = tensor_scales(a.ta, a.tb);
    }
    // What a weight row's outputs share is formed once: its bias, its column of
    // C (gated: rows 16b .. + 7 hold outputs 8b .., their up rows follow).
    const bool gated = a.epi.gated != 0;
    const int ldc = gated ? a.N >> 1 : a.N;
    auto column = [&](int n) { return gated ? ((n >> 4) << 3) | (n & 7) : n; };
    auto bias_of = [&](int n) { return a.epi.bias && n < a.N ? epi_at(a.epi.bias, n) : 0.0f; };
    if (a.split == 1) {
        // a lane's 32 columns at a time: one output of each activation row, 32
        // consecutive outputs to a warp
        if (warp >= 2 && ok) {
            const int n = p0 + row, o = column(n), set = w >> 2;
            const bool mine = n < a.N && !(gated && (row & 8));
            const float bias = bias_of(n);
            for (int c = set * 16; c < live; c += 32) {
                float v[16];
                if (nk > 0) {
                    tmem_ld16(lane_base + c, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0.0f;   // K = 0: an empty sum
                }
                size_t idx = (size_t)(q0 + c) * ldc + o;
#pragma unroll
                for (int i = 0; i < 16; ++i, idx += ldc) {
                    float y = fmaf(v[i] * alpha.first, alpha.second, bias);
                    if (gated) y = silu_short<true>(y) * __shfl_xor_sync(0xffffffffu, y, 8);   // a gate row's up row is lane + 8
                    if (!mine || c + i >= live) continue;
                    if (a.epi.residual) y += epi_at(a.epi.residual, idx);
                    if (a.out_f32) static_cast<float*>(a.C)[idx] = y;
                    else static_cast<__nv_bfloat16*>(a.C)[idx] = __float2bfloat16_rn(y);
                }
            }
        }
    } else {
        // Partial sums to the ring (its copies and instructions are done), as
        // [column][128 rows]; then each CTA adds, in rank order, the partial
        // sums of its share of the columns, a warp a column, and stores them.
        float* part = reinterpret_cast<float*>(smem);
        if (warp >= 2 && ok) {
            for (int c = (w >> 2) * 16; c < live; c += 32) {
                float v[16];
                tmem_ld16(lane_base + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < live) part[(c + i) * kP + row] = v[i];
            }
        }
        cluster_sync_all();
        if (warp >= 2) {
            uint32_t src[kClusterMax];
#pragma unroll
            for (int s = 0; s < kClusterMax; ++s) src[s] = s < a.split ? mapa_shared(smem_u32(part), (uint32_t)s) : 0u;
            const int r = lane * 4, n = p0 + r, o = column(n);   // this lane's rows r .. r + 3: four outputs in a row
            const float bias[4] = {bias_of(n), bias_of(n + 1), bias_of(n + 2), bias_of(n + 3)};
            const bool mine = ok && n < a.N && !(gated && (r & 8)), four = n + 3 < a.N && ldc % 4 == 0;
            for (int c = rank + a.split * w; c < live; c += a.split * 8) {
                float4 x[kClusterMax];
#pragma unroll
                for (int s = 0; s < kClusterMax; ++s)
                    x[s] = s < a.split ? ld_dsmem_f4(src[s] + (uint32_t)(c * kP + r) * 4u) : make_float4(0.f, 0.f, 0.f, 0.f);
                float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kClusterMax; ++s) {   // rank order
                    y[0] += x[s].x;
                    y[1] += x[s].y;
                    y[2] += x[s].z;
                    y[3] += x[s].w;
                }
                const size_t idx = (size_t)(q0 + c) * ldc + o;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = fmaf(y[e] * alpha.first, alpha.second, bias[e]);
                    if (gated) y[e] = silu_short<true>(y[e]) * __shfl_xor_sync(0xffffffffu, y[e], 2);   // row + 8
                    if (a.epi.residual && mine && n + e < a.N) y[e] += epi_at(a.epi.residual, idx + e);
                }
                if (!mine) continue;
                if (a.out_f32) {
                    float* C = static_cast<float*>(a.C) + idx;
                    if (four) {
                        *reinterpret_cast<float4*>(C) = make_float4(y[0], y[1], y[2], y[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < a.N) C[e] = y[e];
                    }
                } else {
                    __nv_bfloat16* C = static_cast<__nv_bfloat16*>(a.C) + idx;
                    if (four) {
                        *reinterpret_cast<uint2*>(C) = make_uint2(bf16x2_of(y[0], y[1]), bf16x2_of(y[2], y[3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < a.N) C[e] = __float2bfloat16_rn(y[e]);
                    }
                }
            }
        }
        cluster_sync_all();   // no CTA leaves while another reads its sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, a.tmem_cols);
}

// launch_dependent with the kernel's shared-memory limit raised once per device
// (`id` counts the kernels)
template <typename... Params, typename... Args>
int launch(int id, void (*kern)(Params...), unsigned grid, unsigned threads, unsigned cluster, size_t smem,
           cudaStream_t stream, const Args&... args) {
    static std::atomic<uint64_t> raised[16];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WQ_ERR_CUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised[id].load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess)
            return WQ_ERR_CUDA;
        raised[id].fetch_or(bit, std::memory_order_release);
    }
    return launch_dependent(kern, grid, threads, cluster, smem, stream, args...) == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

// The tiled scales as [row blocks][blocks along K][512 bytes]: one copy takes a
// stage's blocks of up to two row blocks.
bool encode_scales(CUtensorMap* map, const uint8_t* scales, int rows, int kchunks, int chunks, int row_blocks) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(p) : nullptr;
    }();
    const cuuint64_t dims[3] = {128, (cuuint64_t)kchunks, ((cuuint64_t)rows + 127) / 128};   // 4-byte elements
    const cuuint64_t strides[2] = {512, (cuuint64_t)kchunks * 512};
    const cuuint32_t box[3] = {128, (cuuint32_t)chunks, (cuuint32_t)row_blocks}, step[3] = {1, 1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(scales), dims, strides, box,
                            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Switches for tests and tuning, read at each call:
//   WQ_FP4_PAIR     columns of a pair's tile; 0: rows_kernel
//   WQ_FP4_SPLIT    pairs that share a tile's stages
//   WQ_FP4_WAIT_NS  the bound of the epilogue's wait for its sums (0: give up)
// One pass over the environment tells a call without any of them, the usual
// one (0.1 us for each getenv where a call takes 5).
struct Switches {
    bool force = false;
    int bn = 0, split = 0;
    unsigned long long acc_wait_ns = kWaitNs;
};

Switches switches() {
    Switches w;
    bool any = false;
    for (char** e = environ; e && *e && !any; ++e) any = strncmp(*e, "WQ_FP4_", 7) == 0;
    if (!any) return w;
    if (const char* e = getenv("WQ_FP4_PAIR")) {
        w.force = true;
        w.bn = atoi(e);
    }
    if (const char* e = getenv("WQ_FP4_SPLIT")) w.split = atoi(e);
    if (const char* e = getenv("WQ_FP4_WAIT_NS")) w.acc_wait_ns = strtoull(e, nullptr, 10);
    return w;
}

uint32_t pow2_cols(int c) {
    uint32_t n = 32;
    while ((int)n < c) n *= 2;
    return n;
}

// Clusters of s CTAs, one an SM, that the device runs at a time, asked once per
// device and size: GPCs hold different numbers of SMs, so it is less than
// SMs / s (152 SMs: 23 clusters of 6, and a 24th ran after them).
int max_clusters(int s) {
    static std::atomic<int> known[64][kClusterMax + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][s].load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = rows_kernel<kNVFP4>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)s, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = kMaxSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)s;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();   // a refused query leaves no error behind
            n = 0;
        }
        n = n > 0 ? n : -1;
        known[dev][s].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int FMT>
int launch_pair_of(bool f32, bool gated, unsigned grid, size_t smem, cudaStream_t stream,
                   const CUtensorMap (&t)[5], const PairArgs& a) {
    constexpr int id = FMT == kNVFP4 ? 2 : 7;
    auto go = [&](int i, auto kern) {
        return launch(id + i, kern, grid, kThreads, 2 * a.split, smem, stream, t[0], t[1], t[2], t[3], t[4], a);
    };
    if (a.split > 1) return go(0, pair_kernel<FMT, false, false, true>);
    if (f32) return gated ? go(1, pair_kernel<FMT, true, true, false>) : go(2, pair_kernel<FMT, true, false, false>);
    return gated ? go(3, pair_kernel<FMT, false, true, false>) : go(4, pair_kernel<FMT, false, false, false>);
}

struct PairPlan {
    int bn;      // columns of a tile
    int split;   // pairs that share a tile's stages
    long long cost;
};

// The plan of least time, in cycles past what every plan needs.  A stage takes
// about what its bytes need at 64 bytes a cycle; a tile's end costs some 300
// cycles, 900 where the accumulators share columns; the last tile's epilogue
// 600 for each two of its pieces.  Shared stages: one tile a cluster, all
// clusters at a time, and the sums, whose time grows with the square of the
// width.  The constants of both kernels' plans are fitted together to 1019
// products (M = 18 to 1024, N = 32 to 32768, K = 576 to 16384), each measured
// with every width from 64 to 256, the splits and rows_kernel: the choice loses
// 0.7 % to the best on average (1.2 % on products left out of the fit), more
// than 6 % on 53, and 20 % at worst (90 x 3328 x 1664).
// bn_only > 0: that width.
PairPlan pair_plan(int M, int N, int K, int fmt, int bn_only) {
    const long long pairs = sm_count() / 2, nks = (K + kBK - 1) / kBK;
    const int sbytes = fmt == kNVFP4 ? 2048 : 1024;
    PairPlan best{0, 1, 0};
    for (int bn = 64; bn <= kQMax; bn += 64) {
        if (bn_only > 0 && bn != bn_only) continue;
        const long long tiles = (long long)((M + 255) / 256) * ((N + bn - 1) / bn);
        const long long stage = (kPBytes + bn * 64 + sbytes * (bn > 128 ? 3 : 2)) / 64;
        for (int split = 1; split <= kSplitMax; ++split) {
            if (split > 1 && (split > nks || tiles > max_clusters(2 * split))) break;
            const long long cost =
                split == 1 ? (tiles + pairs - 1) / pairs * (nks * stage + (bn > 192 ? 900 : 300)) + 600 * ((bn + 127) / 128)
                           : (nks + split - 1) / split * stage + 2300 + bn * bn / 64 * 12;
            if (best.bn == 0 || cost < best.cost) best = {bn, split, cost};
        }
    }
    return best;
}

struct RowsPlan {
    int bn;      // activation rows of a tile
    int split;   // CTAs that share a tile's stages
    long long cost;
};

// rows_kernel's tiles: few of them are shared by as many CTAs as there are SMs
// for, all clusters at a time.  Its time in the same unit: the epilogue grows
// with the rows.
RowsPlan rows_plan(int M, int N, int K, int fmt, bool gated) {
    RowsPlan p{M >= kQMax ? kQMax : (M + 15) / 16 * 16, 1, 0};
    const long long nks = (K + kBK - 1) / kBK, sms = sm_count();
    const long long tiles = (long long)((N + kP - 1) / kP) * ((M + p.bn - 1) / p.bn);
    if (tiles * 2 <= sms) {
        long long s = sms / tiles;
        if (s > kClusterMax) s = kClusterMax;
        if (s > nks) s = nks;
        while (s > 1 && max_clusters((int)s) < tiles) --s;
        if (s > 1) p.split = (int)s;
    }
    const int sbytes = fmt == kNVFP4 ? 2048 : 1024;
    const long long stage = (kPBytes + p.bn * 128 + sbytes * (p.bn > 128 ? 3 : 2)) / 64;
    p.cost = (tiles * p.split + sms - 1) / sms * ((nks + p.split - 1) / p.split * stage * 4 / 5) + 500 +
             (long long)p.bn * (p.split <= 2 ? (gated ? 55 : 45) : 10 + 170 / p.split);
    return p;
}

// P the weights, Q the activations
int launch_rows(const Fp4Operand& A, const Fp4Operand& B, void* C, int M, int N, int K, int fmt, bool out_f32,
                const Epilogue& epi, bool ahead, unsigned long long acc_wait_ns, cudaStream_t stream) {
    RowsArgs a{};
    a.p_scales = B.scales;
    a.q_scales = A.scales;
    a.ta = A.tensor_scale;
    a.tb = B.tensor_scale;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    const RowsPlan plan = rows_plan(M, N, K, fmt, epi.gated);
    a.bn = plan.bn;
    a.split = plan.split;
    a.nt_p = (N + kP - 1) / kP;
    a.nks = (K + kBK - 1) / kBK;
    const long long tiles = (long long)a.nt_p * ((M + a.bn - 1) / a.bn);
    const int sms = sm_count();
    if (tiles * a.split > 0x7FFFFFFF) return WQ_ERR_UNSUPPORTED;
    const int chunk_k = fmt == kNVFP4 ? 64 : 128, chunks = kBK / chunk_k, sbytes = chunks * 512;
    const int q_blocks = (a.bn + 127) / 128;
    a.chunks = (K + chunk_k - 1) / chunk_k;
    a.off_q = kPBytes;
    a.off_ps = a.off_q + (a.bn * 128 + 1023) / 1024 * 1024;
    a.off_qs = a.off_ps + sbytes;
    a.stage_bytes = (a.off_qs + q_blocks * sbytes + 1023) / 1024 * 1024;
    // Two CTAs an SM where there are tiles for them: one's set-up and epilogue
    // under the other's stream.
    const size_t room = (tiles > sms && a.bn <= 128 ? kMaxSmem / 2 - 1024 : kMaxSmem) - 1024 - sizeof(MmShared);
    const int fit = (int)(room / a.stage_bytes), need = (a.nks + a.split - 1) / a.split;
    a.stages = fit < kStagesMax ? fit : kStagesMax;
    if (a.split == 1 && need < a.stages) a.stages = need > 0 ? need : 1;
    a.col_p = a.bn;
    a.col_q = a.col_p + 4 * chunks;
    a.q_cols = 4 * q_blocks;
    a.tmem_cols = pow2_cols(a.col_q + a.q_cols * chunks);
    a.idesc = idesc_fp4(a.bn, fmt == kMXFP4);
    a.out_f32 = out_f32 ? 1 : 0;
    a.ahead = ahead ? 1 : 0;
    a.acc_wait_ns = acc_wait_ns;
    a.epi = epi;
    CUtensorMap tp{}, tq{};
    if (K > 0 && (!encode_2d(&tp, CU_TENSOR_MAP_DATA_TYPE_UINT8, B.packed, (uint64_t)K / 2, N, (uint64_t)K / 2, 128, kP,
                             CU_TENSOR_MAP_SWIZZLE_128B) ||
                  !encode_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, A.packed, (uint64_t)K / 2, M, (uint64_t)K / 2, 128,
                             a.bn, CU_TENSOR_MAP_SWIZZLE_128B)))
        return WQ_ERR_UNSUPPORTED;
    const size_t smem = 1024 + (size_t)a.stages * a.stage_bytes + sizeof(MmShared);
    return launch(fmt == kNVFP4 ? 0 : 1, fmt == kNVFP4 ? rows_kernel<kNVFP4> : rows_kernel<kMXFP4>,
                  (unsigned)(tiles * a.split), kThreads, (unsigned)a.split, smem, stream, tp, tq, a);
}

// P the activations, Q the weights
int launch_pair(const Fp4Operand& A, const Fp4Operand& B, void* C, int M, int N, int K, int fmt, bool out_f32,
                const Epilogue& epi, int bn, int split, bool ahead, unsigned long long acc_wait_ns,
                cudaStream_t stream) {
    // the epilogue's pieces of 64 columns; and a tile, which starts at a
    // multiple of 64 rows of Q, then touches at most two 128-row scale blocks,
    // and one up to 128 rows
    if (bn < 64 || bn > kQMax || bn % 64 != 0) return WQ_ERR_UNSUPPORTED;
    PairArgs a{};
    a.ta = A.tensor_scale;
    a.tb = B.tensor_scale;
    a.M = M;
    a.N = N;
    a.K = K;
    a.bn = bn;
    a.nt_m = (M + 255) / 256;
    a.nt_n = (N + bn - 1) / bn;
    if ((long long)a.nt_m * a.nt_n > 0x3FFFFFFF) return WQ_ERR_UNSUPPORTED;
    a.tiles = a.nt_m * a.nt_n;
    a.nks = (K + kBK - 1) / kBK;
    const int chunk_k = fmt == kNVFP4 ? 64 : 128, chunks = kBK / chunk_k, sbytes = chunks * 512;
    const int kchunks = (K + chunk_k - 1) / chunk_k;
    a.q_blocks = bn > 128 ? 2 : 1;
    a.off_q = kPBytes;
    a.off_ps = a.off_q + bn * 64;
    a.off_qs = a.off_ps + sbytes;
    a.stage_bytes = (a.off_qs + a.q_blocks * sbytes + 1023) / 1024 * 1024;
    a.tx_bytes = 2 * (a.off_qs + a.q_blocks * sbytes);
    const int fit = (int)((kMaxSmem - 1024 - 8 * kStgWarp - sizeof(PairShared)) / a.stage_bytes);
    a.stages = fit < kStagesMax ? fit : kStagesMax;
    a.off_stg = a.stages * a.stage_bytes;
    a.acc1 = bn < 192 ? bn : 192;
    a.share = a.acc1 < bn;
    a.idesc = idesc_fp4(bn, fmt == kMXFP4) + (1u << 27);   // M = 256
    a.ahead = ahead ? 1 : 0;
    a.acc_wait_ns = acc_wait_ns;
    a.epi = epi;
    const int cols = epi.gated ? N / 2 : N;
    a.res_vec = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(epi.residual) & 15) == 0;
    // C through a tensor map where its rows are 16-byte multiples
    const bool rows16 = (size_t)cols * (out_f32 ? 4 : 2) % 16 == 0;
    a.split = split;
    a.C = rows16 && split == 1 ? nullptr : C;
    a.out_f32 = out_f32 ? 1 : 0;
    a.rows16 = rows16 ? 1 : 0;
    CUtensorMap t[5] = {};
    const uint64_t kb = (uint64_t)K / 2;
    if (!encode_2d(&t[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, A.packed, kb, M, kb, 128, kP, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&t[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, B.packed, kb, N, kb, 128, bn / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_scales(&t[2], A.scales, M, kchunks, chunks, 1) ||
        !encode_scales(&t[3], B.scales, N, kchunks, chunks, a.q_blocks) ||
        (rows16 && !encode_2d(&t[4], out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, C, cols, M,
                   (uint64_t)cols * (out_f32 ? 4 : 2), out_f32 || epi.gated ? 32 : 64, 32,
                   epi.gated && !out_f32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B)))
        return WQ_ERR_UNSUPPORTED;
    const size_t smem = 1024 + (size_t)a.off_stg + 8 * kStgWarp + sizeof(PairShared);
    const int pairs = sm_count() / 2;
    const unsigned grid = 2u * (unsigned)(split > 1 ? a.tiles * split : a.tiles < pairs ? a.tiles : pairs);
    return fmt == kNVFP4 ? launch_pair_of<kNVFP4>(out_f32, epi.gated, grid, smem, stream, t, a)
                         : launch_pair_of<kMXFP4>(out_f32, epi.gated, grid, smem, stream, t, a);
}

}  // namespace

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

int launch_gemm_fp4(const Fp4Operand& A, const Fp4Operand& B, void* C, int M, int N, int K, int fmt, bool out_f32,
                    const Epilogue& epi, bool ahead, cudaStream_t stream) {
    // The kernel of less time by the plans' costs; rows_kernel up to 16 rows,
    // where it was ahead on 35 of 36 measured shapes and level on the other
    // (1 x 8192 x 3072: 5.2 against 8.0 us), and for K = 0, which has no stages.
    const Switches sw = switches();
    if (K > 0 && (!sw.force || sw.bn > 0)) {
        const bool rows = !sw.force && M <= 16;
        const PairPlan plan = rows ? PairPlan{} : pair_plan(M, N, K, fmt, sw.bn);
        if (!rows && (plan.bn == 0 || sw.split > kSplitMax || sw.split > (K + kBK - 1) / kBK)) return WQ_ERR_UNSUPPORTED;
        if (!rows && (sw.force || plan.cost <= rows_plan(M, N, K, fmt, epi.gated).cost))
            return launch_pair(A, B, C, M, N, K, fmt, out_f32, epi, plan.bn, sw.split > 0 ? sw.split : plan.split, ahead,
                               sw.acc_wait_ns, stream);
    }
    return launch_rows(A, B, C, M, N, K, fmt, out_f32, epi, ahead, sw.acc_wait_ns, stream);
}

}  // namespace wq
