// wq_attn.cu -- attention of a batch that shares a prefix:
//   out[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q . k_j - m),
//   c = scale log2 e, m a bound of the exponents,
// over the prefix's keys and those of the token's own sequence.  The sums over
// the two, and over parts of each, are independent up to their m:
//   (m, l, o) and (m', l', o')  ->  M = max(m, m'),
//   l 2^(m - M) + l' 2^(m' - M),  o 2^(m - M) + o' 2^(m' - M),
// so each part of the keys is read once, with all the query rows that see it,
// and combine_kernel joins the parts of a row.
//
// rows_kernel: CTAs of four warps, a warp with 16 keys at a time.  The products
// are taken transposed (S^T = K Q^T, O^T = V^T P^T), so that the 16 rows of
// an mma.sync tile are keys or values of v and its 8 columns query rows: a
// decode step has few of those (the query heads of one key head).
#include "wq_attn.cuh"
#include "wq_common.cuh"

#include <cstring>

namespace wq {

static __device__ int g_attn_status = 0;

int read_and_clear_attn_status() {
    int v = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
    return v;
}

namespace {

using namespace sm100;
using namespace attn;

constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s
constexpr uint64_t kDrainNs = 100000000ull;   // 0.1 s

__device__ __forceinline__ void record_timeout() { atomicExch(&g_attn_status, WQ_ERR_DEVICE_TIMEOUT); }

// 2^x, results below 2^-126 as 0 (weights that small do not count next to the
// row's largest, 1); -inf gives 0
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// few query rows: mma.sync
// ---------------------------------------------------------------------------
constexpr size_t kSmemSM = 228 * 1024;   // of an SM; a CTA takes 1 KB more than it asks for
constexpr int kWarps = 4;
constexpr int kBK = 16;
template <int DH>
constexpr int kStages = DH == 2 ? 3 : 6;   // 24 KB a warp
template <int DH>
constexpr int kStageBytes = 2 * DH * 2048; // K, V: DH halves of 16 rows x 128 bytes each

struct RowsShared {
    uint64_t full[kWarps][6];
    float m[kWarps][32];
    float l[kWarps][32];
    Plan plan;
    int abort;
};

template <int NT, int DH>
struct RowsSmem {
    static constexpr int ring = 0;
    static constexpr int red = kWarps * kStages<DH> * kStageBytes<DH>;      // float [kWarps][8][68]
    static constexpr int q = red + kWarps * 8 * 68 * 4;                     // bf16 [8 NT][64 DH + 8]
    static constexpr int shared = q + 8 * NT * (64 * DH + 8) * 2;
    static constexpr int plan = shared + (int)((sizeof(RowsShared) + 15) / 16 * 16);
    static size_t bytes(int sequences) { return 1024 + plan + plan_smem(sequences); }
};

template <int NT, int DH>
__global__ void __launch_bounds__(kWarps * 32, 2)
rows_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap kmap,
            const __grid_constant__ CUtensorMap vmap) {
    constexpr int ROWS = 8 * NT, DP = 64 * DH, ST = kStages<DH>, STB = kStageBytes<DH>;
    using L = RowsSmem<NT, DH>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    RowsShared& sh = *reinterpret_cast<RowsShared*>(smem + L::shared);
    const wq_attention& t = a.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem);
    const uint32_t ring = base + L::ring + warp * ST * STB;
    const uint32_t bar0 = smem_u32(&sh.full[warp][0]);

    if (lane == 0) {
        for (int s = 0; s < ST; ++s) mbar_init(bar0 + 8 * s, 1);
        if (warp == 0) {
            sh.abort = 0;
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        fence_mbarrier_init();
    }
    grid_dependency_wait();
    grid_dependents_launch();
    make_plan<kWarps * 32, ROWS, kBK>(sh.plan, a, smem + L::plan);
    const Plan& plan = sh.plan;
    if (blockIdx.x == 0) publish_plan<kWarps * 32>(plan, a);

    const long long x0 = blockIdx.x * plan.run;
    const long long x1 = x0 + plan.run < plan.line ? x0 + plan.run : plan.line;
    if (x0 >= x1) return;
    // the warp's blocks: x0 + warp, and every kWarps-th from there
    const long long mine = x1 - x0 - warp;
    const int steps = mine > 0 ? (int)((mine + kWarps - 1) / kWarps) : 0;

    // Loads run ahead of the products by ST blocks.  Where 32 blocks lie is
    // found by the 32 lanes at once, so that a page number's latency is paid
    // once for all of them.
    int d_slot = 0, d_head = 0, d_page = 0;
    auto issue = [&](int i) {
        if ((i & 31) == 0) {
            const long long x = x0 + warp + (long long)(i + lane) * kWarps;
            if (x < x1) {
                const Unit u = unit_of<ROWS, kBK>(plan, a, x);
                const int key = (int)(x - u.first) * kBK;
                d_page = page_of(t, u.seq, key);
                d_slot = key % t.cache.page_size;
                d_head = u.head;
            }
        }
        const int slot = __shfl_sync(0xffffffffu, d_slot, i & 31);
        const int head = __shfl_sync(0xffffffffu, d_head, i & 31);
        const int page = __shfl_sync(0xffffffffu, d_page, i & 31);
        if (lane == 0) {
            const int s = i % ST;
            const uint32_t dst = ring + s * STB, bar = bar0 + 8 * s;
            mbar_arrive_expect_tx(bar, STB);
#pragma unroll
            for (int h = 0; h < DH; ++h) tma_load_4d(dst + h * 2048, &kmap, bar, 64 * h, slot, head, page);
#pragma unroll
            for (int h = 0; h < DH; ++h) tma_load_4d(dst + (DH + h) * 2048, &vmap, bar, 64 * h, slot, head, page);
        }
    };
    int ahead = 0;   // blocks asked for
    for (; ahead < ST && ahead < steps; ++ahead) issue(ahead);

    const int D = t.head_dim;
    const int c = lane & 3, g = lane >> 2;
    // ldmatrix rows: the 16 keys of K in two 8-row matrices times two 16-byte
    // columns, and of V likewise with keys and columns exchanged
    const int krow = lane & 15, kcol = lane >> 4;
    const int vrow = (lane & 7) + ((lane >> 4) << 3), vcol = (lane >> 3) & 1;
    bool dead = false;   // gave up on a wait: the results are void, and reported
    int step = 0, landed = 0;

    for (long long x = x0; x < x1;) {
        const Unit u = unit_of<ROWS, kBK>(plan, a, x);
        const long long end = u.first + u.blocks < x1 ? u.first + u.blocks : x1;
        const int valid = u.n * a.group - u.tile * ROWS;   // rows of the tile
        // the query rows
        for (int i = tid; i < ROWS * (DP / 8); i += kWarps * 32) {
            const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < valid && d < D) {
                const int row = u.tile * ROWS + r, tok = u.t0 + row / a.group, hq = u.head * a.group + row % a.group;
                v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(t.q) + tok * t.q_token + hq * t.q_head + d);
            }
            *reinterpret_cast<uint4*>(smem + L::q + (r * (DP + 8) + d) * 2) = v;
        }
        __syncthreads();

        // keys that the lane's query columns see, and that all of them see
        int lim[NT][2], all = u.len;
        if (u.seq >= 0) all = u.len - u.n + (u.tile * ROWS) / a.group + 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = u.tile * ROWS + 8 * nt + 2 * c + e;
                lim[nt][e] = u.seq < 0 ? u.len : u.len - u.n + row / a.group + 1;
            }
        float o[4 * DH][NT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < 4 * DH; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.0f;
        }
        const uint32_t qaddr = base + L::q + ((lane & 7) * (DP + 8) + (lane >> 3) * 8) * 2;

        for (; step < steps; ++step) {
            const long long xb = x0 + warp + (long long)step * kWarps;
            if (xb >= end) break;
            const int key0 = (int)(xb - u.first) * kBK;
            const int s = step % ST;
            if (!dead) {
                const bool ok = mbar_wait_sleep(bar0 + 8 * s, (step / ST) & 1, kWaitNs);
                if (__all_sync(0xffffffffu, ok)) {
                    landed = step + 1;
                } else {
                    dead = true;
                    if (lane == 0) record_timeout();
                }
            }
            const uint32_t kb = ring + s * STB, vb = kb + DH * 2048;
            // S^T = K Q^T: 16 keys x 8 rows a tile
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
#pragma unroll
            for (int k2 = 0; k2 < 2 * DH; ++k2) {   // 32 values of the head
                uint32_t ka[4], kc[4];
                const uint32_t half = kb + (k2 >> 1) * 2048 + krow * 128;
                const int c0 = (k2 & 1) * 4 + kcol;
                ldsm_x4(half + ((c0 ^ (krow & 7)) << 4), ka);
                ldsm_x4(half + (((c0 + 2) ^ (krow & 7)) << 4), kc);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t qb[4];
                    ldsm_x4(qaddr + (nt * 8 * (DP + 8) + k2 * 32) * 2, qb);
                    mma_bf16(sc[nt], ka, qb[0], qb[1]);
                    mma_bf16(sc[nt], kc, qb[2], qb[3]);
                }
            }
            // softmax
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = sc[nt][e] * a.scale_log2;
                if (key0 + kBK > all) {
                    if (key0 + g >= lim[nt][0]) y[0] = -INFINITY;
                    if (key0 + g >= lim[nt][1]) y[1] = -INFINITY;
                    if (key0 + g + 8 >= lim[nt][0]) y[2] = -INFINITY;
                    if (key0 + g + 8 >= lim[nt][1]) y[3] = -INFINITY;
                }
                float b0 = fmaxf(y[0], y[2]), b1 = fmaxf(y[1], y[3]);
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, k));
                    b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, k));
                }
                const float n0 = fmaxf(m[nt][0], b0), n1 = fmaxf(m[nt][1], b1);
                // a row that has seen no key yet: exponents of -inf from 0
                const float z0 = n0 == -INFINITY ? 0.0f : n0, z1 = n1 == -INFINITY ? 0.0f : n1;
                if (__any_sync(0xffffffffu, n0 != m[nt][0] || n1 != m[nt][1])) {
                    const float f0 = ex2(m[nt][0] - z0), f1 = ex2(m[nt][1] - z1);
                    l[nt][0] *= f0;
                    l[nt][1] *= f1;
#pragma unroll
                    for (int mt = 0; mt < 4 * DH; ++mt) {
                        o[mt][nt][0] *= f0;
                        o[mt][nt][1] *= f1;
                        o[mt][nt][2] *= f0;
                        o[mt][nt][3] *= f1;
                    }
                    m[nt][0] = n0;
                    m[nt][1] = n1;
                }
                const float p0 = ex2(y[0] - z0), p1 = ex2(y[1] - z1), p2 = ex2(y[2] - z0), p3 = ex2(y[3] - z1);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                // the products' operand has rows and keys exchanged
                pb[nt][0] = transpose_8x8(pack_bf16(p0, p1));
                pb[nt][1] = transpose_8x8(pack_bf16(p2, p3));
            }
            // O^T += V^T P^T; slots past the last key may hold anything
            const bool tail = key0 + kBK > u.len;
            const int left = u.len - key0;
            const uint32_t k_lo = (2 * c < left ? 0xFFFFu : 0u) | (2 * c + 1 < left ? 0xFFFF0000u : 0u);
            const uint32_t k_hi = (2 * c + 8 < left ? 0xFFFFu : 0u) | (2 * c + 9 < left ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int mt = 0; mt < 4 * DH; ++mt) {
                uint32_t va[4];
                const int ch = (mt & 3) * 2 + vcol;
                ldsm_x4_trans(vb + (mt >> 2) * 2048 + vrow * 128 + ((ch ^ (vrow & 7)) << 4), va);
                if (tail) {
                    va[0] &= k_lo;
                    va[1] &= k_lo;
                    va[2] &= k_hi;
                    va[3] &= k_hi;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16(o[mt][nt], va, pb[nt][0], pb[nt][1]);
            }
            __syncwarp();   // all lanes have read the stage
            if (!dead && ahead < steps) issue(ahead++);
        }

        // join the warps' parts, and store the piece
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[nt][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (g == 0) {
                    sh.m[warp][8 * nt + 2 * c + e] = m[nt][e];
                    sh.l[warp][8 * nt + 2 * c + e] = v;
                }
            }
        __syncthreads();
        const long long piece = blockIdx.x + u.unit;
        const bool room = piece < a.max_pieces;
        if (tid < ROWS && tid < valid && room) {
            float M = sh.m[0][tid], s = 0.0f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sh.m[w][tid]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                s += M == -INFINITY ? sh.l[w][tid] : sh.l[w][tid] * ex2(sh.m[w][tid] - M);
            a.part_ml[piece * ROWS + tid] = make_float2(M, s);
        }
        float* red = reinterpret_cast<float*>(smem + L::red);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + 2 * c + e;
                float M = sh.m[0][r];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sh.m[w][r]);
                f[e] = M == -INFINITY ? 0.0f : ex2(m[nt][e] - M);
            }
#pragma unroll
            for (int h = 0; h < DH; ++h) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float(&v)[4] = o[4 * h + k][nt];
                    float* p = red + (warp * 8 + 2 * c) * 68 + 16 * k + g;
                    p[0] = v[0] * f[0];
                    p[68] = v[1] * f[1];
                    p[8] = v[2] * f[0];
                    p[68 + 8] = v[3] * f[1];
                }
                __syncthreads();
                const int r = tid >> 4, d = (tid & 15) * 4;
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(red + (w * 8 + r) * 68 + d);
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                if (8 * nt + r < valid && room)
                    *reinterpret_cast<float4*>(a.part_o + (piece * ROWS + 8 * nt + r) * DP + 64 * h + d) = s;
                __syncthreads();
            }
        }
        x = end;
    }
    // a warp that gave up still sees its copies land before it leaves
    if (dead && lane == 0)
        for (int i = landed; i < ahead; ++i) mbar_wait_timeout(bar0 + 8 * (i % ST), (i / ST) & 1, kDrainNs);
}

// ---------------------------------------------------------------------------
// the pieces of a row joined
// ---------------------------------------------------------------------------
struct Part {
    const float* o;
    const float2* ml;
    const long long* plan;
    int rows, bk, per;   // rows of a piece, keys of a block, pieces a run and unit have
    int max_pieces;
};

struct CombineArgs {
    wq_attention t;
    int group, dp;
    Part prefix, own;
};

struct Pieces {
    long long first;   // index of the first (m, l), rows apart
    int n;
    int stride;
};

__device__ __forceinline__ long long divide(long long a, long long b) {
    // 32 bits where they hold it
    return (a | b) >> 31 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// pieces of the unit `unit`, whose blocks are first .. first + blocks - 1, and row `row` in it
__device__ __forceinline__ Pieces pieces_of(const Part& p, long long run, long long unit, long long first, long long blocks,
                                            int row) {
    Pieces q{0, 0, p.rows};
    if (blocks <= 0) return q;
    const long long j0 = divide(first, run), j1 = divide(first + blocks - 1, run);
    const long long piece = (j0 + unit) * p.per;
    q.first = piece * p.rows + row;
    q.n = (int)(j1 - j0 + 1) * p.per;
    if (piece + q.n > p.max_pieces) q.n = piece < p.max_pieces ? (int)(p.max_pieces - piece) : 0;
    return q;
}

constexpr int kCombineWarps = 4;

__global__ void __launch_bounds__(kCombineWarps * 32) combine_kernel(const __grid_constant__ CombineArgs a) {
    const wq_attention& t = a.t;
    const int lane = threadIdx.x & 31;
    const int item = blockIdx.x * kCombineWarps + (threadIdx.x >> 5);
    const int tok = item / t.q_heads, h = item - tok * t.q_heads;
    grid_dependents_launch();
    // The lengths were there before the kernel that this one follows.
    int b = 0, behind = tok >= t.tokens;
    if (!behind) {
        if (t.q_start) {
            int n = 0;
            for (int i = lane; i < t.sequences; i += 32) n += seq_start(t, i) <= tok;
            b = __reduce_add_sync(0xffffffffu, n) - 1;
            behind = b < 0 || tok >= seq_start(t, t.sequences);
        } else {
            b = tok / (t.tokens / t.sequences);
            behind = b >= t.sequences;
        }
    }
    Seq s{0, 0, 0};
    if (!behind) {
        s = seq_at(t, b);
        behind = tok < s.t0 || tok >= s.t0 + s.n;   // (starts that descend)
    }
    if (behind) {
        grid_dependency_wait();
        return;
    }
    const int kh = h / a.group, hg = h - kh * a.group;
    grid_dependency_wait();

    // the prefix's pieces, then the sequence's own
    Pieces pp, po;
    {
        const long long* pl = a.prefix.plan;
        const long long run = pl[0], tiles = pl[1], blocks = pl[2];
        const long long row = (long long)tok * a.group + hg;
        const int tile = (int)(row / a.prefix.rows);
        const long long unit = kh * tiles + tile;
        pp = pieces_of(a.prefix, run, unit, unit * blocks, tiles > 0 ? blocks : 0, (int)(row - (long long)tile * a.prefix.rows));
    }
    {
        const long long* pl = a.own.plan;
        const long long run = pl[0];
        const long long w0 = pl[kPlanHead + 2 * b], w1 = pl[kPlanHead + 2 * b + 2];
        const long long u0 = pl[kPlanHead + 2 * b + 1], u1 = pl[kPlanHead + 2 * b + 3];
        const int row = (tok - s.t0) * a.group + hg, tile = row / a.own.rows;
        long long first = pl[3] + w0 * t.kv_heads + kh * (w1 - w0);
        int blocks = 0;
        for (int i = 0; i <= tile; ++i) {
            first += blocks;
            blocks = (tile_keys(s, a.group, a.own.rows, i) + a.own.bk - 1) / a.own.bk;
        }
        po = pieces_of(a.own, run, pl[1] * t.kv_heads + u0 * t.kv_heads + kh * (u1 - u0) + tile, first, blocks,
                       row - tile * a.own.rows);
    }
    const int n = pp.n + po.n;
    auto ml_at = [&](int i) {
        return i < pp.n ? a.prefix.ml[pp.first + (long long)i * pp.stride]
                        : a.own.ml[po.first + (long long)(i - pp.n) * po.stride];
    };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, ml_at(i).x);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    const bool on = 4 * lane < t.head_dim;
    for (int i0 = 0; i0 < n; i0 += 32) {
        float w = 0.0f, l = 0.0f;
        if (i0 + lane < n) {
            const float2 ml = ml_at(i0 + lane);
            // (with M = -inf no piece has a weight, but a sum that is no number still shows)
            w = M == -INFINITY ? 0.0f : ex2(ml.x - M);
            l = M == -INFINITY ? ml.y : w * ml.y;
        }
        sum += l;
        const int m = n - i0 < 32 ? n - i0 : 32;
#pragma unroll 4
        for (int i = 0; i < m; ++i) {
            const float f = __shfl_sync(0xffffffffu, w, i);
            const int k = i0 + i;
            const float* p = k < pp.n ? a.prefix.o + (pp.first + (long long)k * pp.stride) * a.dp
                                      : a.own.o + (po.first + (long long)(k - pp.n) * po.stride) * a.dp;
            if (on) {
                const float4 v = *reinterpret_cast<const float4*>(p + 4 * lane);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    // no key at all: 0
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (on) {
        uint2 v;
        v.x = pack_bf16(acc.x * inv, acc.y * inv);
        v.y = pack_bf16(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(t.out) + tok * t.out_token + h * t.out_head + 4 * lane) = v;
    }
    if (t.lse && lane == 0)
        t.lse[(long long)tok * t.q_heads + h] =
            sum == 0.0f ? -INFINITY : (M == -INFINITY ? 0.0f : M) * 0.693147180559945f + logf(sum);
}

template <int NT, int DH>
cudaError_t launch_rows(Args a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t stream) {
    const size_t smem = RowsSmem<NT, DH>::bytes(a.t.sequences);
    auto kern = rows_kernel<NT, DH>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // as many runs as CTAs fit the device at a time
    if (2 * (smem + 1024) > kSmemSM) a.runs = (a.runs + 1) / 2;
    return launch_dependent(kern, (unsigned)a.runs, kWarps * 32, 1, smem, stream, a, km, vm);
}

// query rows of a unit: 8, 16 or 32
int rows_of(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

long long units_bound(int tokens, int sequences, int kv_heads, int group, int rows) {
    const long long all = (long long)tokens * group;
    return kv_heads * ((all + rows - 1) / rows + all / rows + sequences);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// the workspace: plan | (m, l) of all pieces | their sums
struct Space {
    int rows, runs;
    long long pieces;
    size_t plan, ml, o, bytes;
};

Space space_of(int tokens, int sequences, int q_heads, int kv_heads, int head_dim) {
    Space s;
    const int group = q_heads / kv_heads;
    s.rows = rows_of((long long)tokens * group);
    s.runs = 2 * sm_count();
    s.pieces = s.runs + units_bound(tokens, sequences, kv_heads, group, s.rows);
    s.plan = 0;
    s.ml = up256(kPlanBytes);
    s.o = s.ml + up256((size_t)s.pieces * s.rows * sizeof(float2));
    s.bytes = s.o + up256((size_t)s.pieces * s.rows * (head_dim <= 64 ? 64 : 128) * sizeof(float));
    return s;
}

}  // namespace

size_t attn_workspace_bytes(int tokens, int sequences, int q_heads, int kv_heads, int head_dim) {
    return space_of(tokens, sequences, q_heads, kv_heads, head_dim).bytes;
}

int launch_prefix_attention(const wq_attention& t, cudaStream_t stream) {
    const Space sp = space_of(t.tokens, t.sequences, t.q_heads, t.kv_heads, t.head_dim);
    if (sp.pieces > 0x7FFFFFFF) return WQ_ERR_UNSUPPORTED;
    uint8_t* ws = static_cast<uint8_t*>(t.workspace);
    Args a;
    a.t = t;
    a.group = t.q_heads / t.kv_heads;
    a.prefix = t.prefix_len > 0;
    a.own = 1;
    a.runs = sp.runs;
    a.min_run = 8;
    a.box = 16;
    a.max_pieces = (int)sp.pieces;
    a.scale_log2 = t.scale * 1.44269504088896341f;
    a.part_ml = reinterpret_cast<float2*>(ws + sp.ml);
    a.part_o = reinterpret_cast<float*>(ws + sp.o);
    a.plan = reinterpret_cast<long long*>(ws + sp.plan);

    CUtensorMap km, vm;
    const wq_kv_cache& kv = t.cache;
    const int dh = t.head_dim <= 64 ? 1 : 2;
    if (kv.pages > 0) {
        const uint64_t dims[4] = {(uint64_t)t.head_dim, (uint64_t)kv.page_size, (uint64_t)t.kv_heads, (uint64_t)kv.pages};
        const uint64_t strides[3] = {(uint64_t)kv.slot_stride * 2, (uint64_t)kv.head_stride * 2,
                                     (uint64_t)kv.page_stride * 2};
        const uint32_t box[4] = {64, (uint32_t)a.box, 1, 1};
        if (!encode_4d(&km, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kv.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_4d(&vm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kv.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return WQ_ERR_UNSUPPORTED;
    } else {
        // no cache, so no keys: the kernel makes no copy
        memset(&km, 0, sizeof km);
        memset(&vm, 0, sizeof vm);
    }
    cudaError_t e;
    if (sp.rows == 8) e = dh == 1 ? launch_rows<1, 1>(a, km, vm, stream) : launch_rows<1, 2>(a, km, vm, stream);
    else if (sp.rows == 16) e = dh == 1 ? launch_rows<2, 1>(a, km, vm, stream) : launch_rows<2, 2>(a, km, vm, stream);
    else e = dh == 1 ? launch_rows<4, 1>(a, km, vm, stream) : launch_rows<4, 2>(a, km, vm, stream);
    if (e != cudaSuccess) return WQ_ERR_CUDA;

    CombineArgs ca;
    ca.t = t;
    ca.group = a.group;
    ca.dp = 64 * dh;
    ca.own = Part{a.part_o, a.part_ml, a.plan, sp.rows, kBK, 1, a.max_pieces};
    ca.prefix = ca.own;
    const long long items = (long long)t.tokens * t.q_heads;
    e = launch_dependent(combine_kernel, (unsigned)((items + kCombineWarps - 1) / kCombineWarps), kCombineWarps * 32, 1, 0,
                         stream, ca);
    return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

}  // namespace wq
