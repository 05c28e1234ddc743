// wq_rope.cu -- between the q/k/v projection and the attention, in one pass:
//   n = x / sqrt(mean x^2 + eps) w + b        for each query and key head
//       (or the layer norm, or n = x)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//       for the pairs of the first R values; t = position on the pair's axis
//       times the pair's frequency; values past R pass
// and the keys, with the values as they are, go to their slots of the cache.
//
// Angles.  t is needed modulo one turn only, so a pair's frequency is held in
// turns per position as a 64-bit fixed-point fraction F: the product of a
// 32-bit position and F modulo 2^64 is the exact fraction of a turn (error at
// most 2^31 2^-62 turns from F's own rounding), at two integer multiplies and
// with no range reduction.  An fp32 product would be off by 2^-25 of the angle
// itself: 0.004 rad at position 130000, frequency 1.  Its top 32 bits become
// an fp32 half-turn in [-1, 1), off by 2^-25 at most, and sincospi of that is
// good to an fp32 rounding.
//
// For bf16 inputs the two come from sin.approx and cos.approx on (-pi, pi],
// which are off by 2^-21: 1/2000 of a bf16 rounding, at a tenth of the
// instructions (8192 tokens of 32 + 8 + 8 heads of 128: see below).
//
// Everything between load and store is fp32.  The bound is HBM: each head is
// read once and written once.
//
// Layout.  A group of 8, 16 or 32 lanes holds one head, eight values a lane:
// four pairs (chunks of four at 4 l and R / 2 + 4 l, or 8 l and 8 l + 4 for
// adjacent pairs) or eight values past R.  A pair never leaves its lane, so
// the rotation needs no exchange, and the lane's four sines and cosines, and
// the weights, serve all heads that the group takes of its token.
#include <cuda_bf16.h>

#include "wq_internal.h"
#include "wq_tc.cuh"

namespace wq {

namespace {

struct RopeArgs {
    wq_rope r;
    int rows;       // heads a token: q, k and (with a cache) v
    int q_runs, k_runs, runs;   // groups a token for the heads of q, of q and k, and all
    int groups;     // tokens * runs
    int rot_units;  // lanes that hold pairs
    int units;      // lanes that hold anything
    float inv_d;
};

struct Half8 {
    float a[4], b[4];
};

template <bool F32>
__device__ __forceinline__ float load1(const void* p, long long i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

__device__ __forceinline__ void unpack4(uint2 w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A lane's place in a head: the first elements of its two chunks (VEC), or
// for heads of any size and alignment element e of its eight, -1 where the
// lane has none.
struct Place {
    int u, rot, R, D;
    bool rotated, any;
    template <bool ADJ>
    __device__ __forceinline__ int chunk(int c) const {
        if (!rotated) return R + 8 * (u - rot) + 4 * c;
        return ADJ ? 8 * u + 4 * c : 4 * u + c * (R >> 1);
    }
    // element of a[e] (c = 0) or b[e] (c = 1)
    template <bool ADJ>
    __device__ __forceinline__ int elem(int c, int e) const {
        if (!any) return -1;
        if (!rotated) {
            const int i = R + 8 * (u - rot) + 4 * c + e;
            return i < D ? i : -1;
        }
        const int p = 4 * u + e;
        if (2 * p >= R) return -1;
        return ADJ ? 2 * p + c : p + c * (R >> 1);
    }
};

// chunk order (x0..x3, x4..x7) <-> pair order (a, b) of adjacent pairs
__device__ __forceinline__ void to_pairs(Half8& x) {
    const Half8 y = x;
    x.a[0] = y.a[0]; x.b[0] = y.a[1]; x.a[1] = y.a[2]; x.b[1] = y.a[3];
    x.a[2] = y.b[0]; x.b[2] = y.b[1]; x.a[3] = y.b[2]; x.b[3] = y.b[3];
}
__device__ __forceinline__ void from_pairs(Half8& x) {
    const Half8 y = x;
    x.a[0] = y.a[0]; x.a[1] = y.b[0]; x.a[2] = y.a[1]; x.a[3] = y.b[1];
    x.b[0] = y.a[2]; x.b[1] = y.b[2]; x.b[2] = y.a[3]; x.b[3] = y.b[3];
}

template <bool VEC, bool ADJ, bool F32>
__device__ __forceinline__ void load_head(const void* base, long long off, const Place& pl, Half8& x) {
    if constexpr (VEC) {
        if (!pl.any) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x.a[e] = x.b[e] = 0.0f;
            return;
        }
        const long long i0 = off + pl.chunk<ADJ>(0), i1 = off + pl.chunk<ADJ>(1);
        if constexpr (F32) {
            const float4 p = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i0);
            const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i1);
            x.a[0] = p.x; x.a[1] = p.y; x.a[2] = p.z; x.a[3] = p.w;
            x.b[0] = q.x; x.b[1] = q.y; x.b[2] = q.z; x.b[3] = q.w;
        } else {
            unpack4(*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i0), x.a);
            unpack4(*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i1), x.b);
        }
        if constexpr (ADJ) to_pairs(x);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = pl.elem<ADJ>(0, e), j = pl.elem<ADJ>(1, e);
            x.a[e] = i >= 0 ? load1<F32>(base, off + i) : 0.0f;
            x.b[e] = j >= 0 ? load1<F32>(base, off + j) : 0.0f;
        }
    }
}

template <bool VEC, bool ADJ>
__device__ __forceinline__ void store_head(void* base, bool f32, long long off, const Place& pl, Half8 x) {
    if constexpr (VEC) {
        if (!pl.any) return;
        if constexpr (ADJ) from_pairs(x);
        const long long i0 = off + pl.chunk<ADJ>(0), i1 = off + pl.chunk<ADJ>(1);
        if (f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(base) + i0) = make_float4(x.a[0], x.a[1], x.a[2], x.a[3]);
            *reinterpret_cast<float4*>(static_cast<float*>(base) + i1) = make_float4(x.b[0], x.b[1], x.b[2], x.b[3]);
        } else {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i0) =
                make_uint2(pack2(x.a[0], x.a[1]), pack2(x.a[2], x.a[3]));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i1) =
                make_uint2(pack2(x.b[0], x.b[1]), pack2(x.b[2], x.b[3]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int i = pl.elem<ADJ>(c, e);
                const float v = c ? x.b[e] : x.a[e];
                if (i < 0) continue;
                if (f32) static_cast<float*>(base)[off + i] = v;
                else static_cast<__nv_bfloat16*>(base)[off + i] = __float2bfloat16_rn(v);
            }
        }
    }
}

__device__ __forceinline__ float sum8(const Half8& x) {
    return ((x.a[0] + x.a[1]) + (x.a[2] + x.a[3])) + ((x.b[0] + x.b[1]) + (x.b[2] + x.b[3]));
}
__device__ __forceinline__ float squares8(const Half8& x) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fmaf(x.a[e], x.a[e], fmaf(x.b[e], x.b[e], s));
    return s;
}

// sum over a group's lanes; `mask` has the group's bits
template <int LG>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

// one Newton step on rsqrtf (off by two units in the last place) makes it good
// to fp32 outputs
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v);
    return fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
}

// cosine and sine of the lane's four pairs at token t (1 and 0 past R)
template <bool F32>
__device__ __forceinline__ void turns(const wq_rope& r, int u, int t, float (&cs)[4], float (&sn)[4]) {
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pos[i] = i < r.axes ? r.positions[i * r.axis_stride + t] : 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int p = 4 * u + e;
        cs[e] = 1.0f;
        sn[e] = 0.0f;
        if (2 * p >= r.rotary_dim) continue;
        const unsigned long long f = r.table[p];
        const int axis = (int)(f & 3);
        const int at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
        const unsigned long long turn = (unsigned long long)(long long)at * (f & ~3ull);
        const float half = (float)(int)(turn >> 32);   // of 2^-31 half-turns
        if constexpr (F32) {
            sincospif(half * 0x1p-31f, &sn[e], &cs[e]);
        } else {
            const float x = half * (3.14159265358979f * 0x1p-31f);
            sn[e] = __sinf(x);
            cs[e] = __cosf(x);
        }
    }
}

// where token t's keys and values go, in elements; -1: nowhere
__device__ __forceinline__ long long cache_offset(const wq_rope& r, int t) {
    if (!r.with_cache) return -1;
    const unsigned slot = (unsigned)r.slots[t];
    if (slot >= (unsigned)r.cache.pages * (unsigned)r.cache.page_size) return -1;
    const unsigned page = slot / (unsigned)r.cache.page_size;
    return page * r.cache.page_stride + (slot - page * (unsigned)r.cache.page_size) * r.cache.slot_stride;
}

// A group takes HU heads of one kind (queries, keys or values) of a token, LG
// lanes a head.  VEC: chunks of four in one access; else element by element.
template <int LG, int HU, bool VEC, bool ADJ, bool F32>
__global__ void __launch_bounds__(128) rope_kernel(const __grid_constant__ RopeArgs a) {
    sm100::grid_dependency_wait();
    sm100::grid_dependents_launch();
    const wq_rope& r = a.r;
    const int g = blockIdx.x * (128 / LG) + threadIdx.x / LG;
    if (g >= a.groups) return;
    const unsigned mask = LG == 32 ? 0xffffffffu : ((1u << (LG & 31)) - 1) << (threadIdx.x & 31 & ~(LG - 1));
    const int t = (int)((unsigned)g / (unsigned)a.runs), run = g - t * a.runs;

    Place pl;
    pl.u = threadIdx.x % LG;
    pl.rot = a.rot_units;
    pl.R = r.rotary_dim;
    pl.D = r.head_dim;
    pl.rotated = pl.u < a.rot_units;
    pl.any = pl.u < a.units;

    // kind: 0 queries, 1 keys, 2 values
    const int kind = run < a.q_runs ? 0 : run < a.k_runs ? 1 : 2;
    const int h0 = (run - (kind == 0 ? 0 : kind == 1 ? a.q_runs : a.k_runs)) * HU;
    const int n = min(HU, (kind == 0 ? r.q_heads : r.kv_heads) - h0);
    const void* in = kind == 0 ? r.q : kind == 1 ? r.k : r.v;
    const long long hs = kind == 0 ? r.q_head : kind == 1 ? r.k_head : r.v_head;
    const long long off = t * (kind == 0 ? r.q_token : kind == 1 ? r.k_token : r.v_token) + h0 * hs;
    Half8 x[HU];
#pragma unroll
    for (int j = 0; j < HU; ++j)
        if (j < n) load_head<VEC, ADJ, F32>(in, off + j * hs, pl, x[j]);

    if (kind == 2) {
        const long long to = cache_offset(r, t);
        if (to < 0) return;
#pragma unroll
        for (int j = 0; j < HU; ++j)
            if (j < n) store_head<VEC, ADJ>(r.cache.v, false, to + (h0 + j) * r.cache.head_stride, pl, x[j]);
        return;
    }

    // y_a = f (a ca - b sb) + da, y_b = f (b cb + a sa) + db with the weights in
    // the cosines and sines, and the rotated biases
    Half8 wt, cw, sw, bias;
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        cs[e] = 1.0f;
        sn[e] = 0.0f;
        wt.a[e] = wt.b[e] = 1.0f;
    }
    if (pl.rotated) turns<F32>(r, pl.u, t, cs, sn);
    const void* w = kind == 0 ? r.q_weight : r.k_weight;
    const void* c = kind == 0 ? r.q_bias : r.k_bias;
    if (w) load_head<VEC, ADJ, false>(w, 0, pl, wt);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        cw.a[e] = cs[e] * wt.a[e];
        sw.a[e] = sn[e] * wt.b[e];
        cw.b[e] = cs[e] * wt.b[e];
        sw.b[e] = sn[e] * wt.a[e];
        bias.a[e] = bias.b[e] = 0.0f;
    }
    if (c) {
        load_head<VEC, ADJ, false>(c, 0, pl, wt);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bias.a[e] = fmaf(wt.a[e], cs[e], -(wt.b[e] * sn[e]));
            bias.b[e] = fmaf(wt.b[e], cs[e], wt.a[e] * sn[e]);
        }
    }

    float f[HU];
    if (r.norm == WQ_HEAD_NORM_LAYER) {
        float m[HU];
#pragma unroll
        for (int j = 0; j < HU; ++j) m[j] = j < n ? sum8(x[j]) : 0.0f;
#pragma unroll
        for (int j = 0; j < HU; ++j) m[j] = group_sum<LG>(m[j], mask) * a.inv_d;
#pragma unroll
        for (int j = 0; j < HU; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // places without an element keep their zero
                if (VEC ? pl.any : pl.elem<ADJ>(0, e) >= 0) x[j].a[e] -= m[j];
                if (VEC ? pl.any : pl.elem<ADJ>(1, e) >= 0) x[j].b[e] -= m[j];
            }
    }
    if (r.norm != WQ_HEAD_NORM_NONE) {
#pragma unroll
        for (int j = 0; j < HU; ++j) f[j] = j < n ? squares8(x[j]) : 0.0f;
#pragma unroll
        for (int j = 0; j < HU; ++j) f[j] = group_sum<LG>(f[j], mask);
#pragma unroll
        for (int j = 0; j < HU; ++j) f[j] = inverse_root(fmaf(f[j], a.inv_d, r.eps));
    } else {
#pragma unroll
        for (int j = 0; j < HU; ++j) f[j] = 1.0f;
    }

    void* out = kind == 0 ? r.q_out : r.k_out;
    const long long os = kind == 0 ? r.q_out_head : r.k_out_head;
    const long long to = t * (kind == 0 ? r.q_out_token : r.k_out_token) + h0 * os;
    const long long cache = kind == 1 ? cache_offset(r, t) : -1;
    const bool f32 = r.out_type == WQ_TYPE_F32;
#pragma unroll
    for (int j = 0; j < HU; ++j) {
        if (j >= n) break;
        Half8 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (past R an infinity stays in its place: no products with sine 0)
            y.a[e] = fmaf(f[j], fmaf(x[j].a[e], cw.a[e], pl.rotated ? -(x[j].b[e] * sw.a[e]) : 0.0f), bias.a[e]);
            y.b[e] = fmaf(f[j], fmaf(x[j].b[e], cw.b[e], pl.rotated ? x[j].a[e] * sw.b[e] : 0.0f), bias.b[e]);
        }
        if (out) store_head<VEC, ADJ>(out, f32, to + j * os, pl, y);
        if (cache >= 0) store_head<VEC, ADJ>(r.cache.k, false, cache + (h0 + j) * r.cache.head_stride, pl, y);
    }
}

template <int LG, int HU, bool VEC>
cudaError_t launch_as(const RopeArgs& a, bool adj, bool f32, cudaStream_t stream) {
    const unsigned per = 128 / LG, grid = ((unsigned)a.groups + per - 1) / per;
    auto go = [&](auto kern) { return launch_dependent(kern, grid, 128, 1, 0, stream, a); };
    if (f32) return adj ? go(rope_kernel<LG, HU, VEC, true, true>) : go(rope_kernel<LG, HU, VEC, false, true>);
    return adj ? go(rope_kernel<LG, HU, VEC, true, false>) : go(rope_kernel<LG, HU, VEC, false, false>);
}

template <int HU, bool VEC>
cudaError_t launch_heads(RopeArgs& a, bool adj, bool f32, cudaStream_t stream) {
    a.q_runs = (a.r.q_heads + HU - 1) / HU;
    a.k_runs = a.q_runs + (a.r.kv_heads + HU - 1) / HU;
    a.runs = a.k_runs + (a.r.with_cache ? (a.r.kv_heads + HU - 1) / HU : 0);
    a.groups = a.r.tokens * a.runs;
    return a.units <= 8    ? launch_as<8, HU, VEC>(a, adj, f32, stream)
           : a.units <= 16 ? launch_as<16, HU, VEC>(a, adj, f32, stream)
                           : launch_as<32, HU, VEC>(a, adj, f32, stream);
}

}  // namespace

int rope_units(int head_dim, int rotary_dim) { return (rotary_dim + 7) / 8 + (head_dim - rotary_dim + 7) / 8; }

int launch_rope(const wq_rope& r, cudaStream_t stream) {
    RopeArgs a;
    a.r = r;
    a.rows = r.q_heads + r.kv_heads + (r.with_cache ? r.kv_heads : 0);
    a.rot_units = (r.rotary_dim + 7) / 8;
    a.units = rope_units(r.head_dim, r.rotary_dim);
    a.inv_d = 1.0f / (float)r.head_dim;
    // vector accesses: whole chunks of four elements, each aligned to its size
    auto ok = [](const void* p, size_t es, long long s, long long h) {
        const uintptr_t n = 4 * es;
        return !p || (reinterpret_cast<uintptr_t>(p) % n == 0 && (uintptr_t)(s * (long long)es) % n == 0 &&
                      (uintptr_t)(h * (long long)es) % n == 0);
    };
    const size_t in = r.type == WQ_TYPE_F32 ? 4 : 2, out = r.out_type == WQ_TYPE_F32 ? 4 : 2;
    const bool vec = r.head_dim % 8 == 0 && r.rotary_dim % 8 == 0 && ok(r.q, in, r.q_token, r.q_head) &&
                     ok(r.k, in, r.k_token, r.k_head) && (!r.with_cache || (ok(r.v, in, r.v_token, r.v_head) &&
                     ok(r.cache.k, 2, r.cache.page_stride, r.cache.slot_stride) && ok(r.cache.v, 2, r.cache.head_stride, 0))) &&
                     ok(r.q_out, out, r.q_out_token, r.q_out_head) && ok(r.k_out, out, r.k_out_token, r.k_out_head) &&
                     ok(r.q_weight, 2, 0, 0) && ok(r.q_bias, 2, 0, 0) && ok(r.k_weight, 2, 0, 0) &&
                     ok(r.k_bias, 2, 0, 0);
    const bool adj = r.pairs == WQ_PAIRS_ADJACENT, f32 = r.type == WQ_TYPE_F32;
    const bool many = (long long)r.tokens * a.rows >= 16LL * 8 * sm_count();
    const cudaError_t e = !vec   ? launch_heads<1, false>(a, adj, f32, stream)
                          : many ? launch_heads<4, true>(a, adj, f32, stream)
                                 : launch_heads<1, true>(a, adj, f32, stream);
    return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

}  // namespace wq
