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
// Everything between load and store is fp32.  The bound is HBM: each head is
// read once and written once.  8192 tokens of 32 + 8 + 8 heads of 128 in bf16
// (201 MB): see launch_rope.
//
// Layout.  A group of 8, 16 or 32 lanes holds one head, eight values a lane:
// four pairs (chunks of four at 4 l and R / 2 + 4 l, or 8 l and 8 l + 4 for
// adjacent pairs) or eight values past R.  A pair never leaves its lane, so
// the rotation needs no exchange, and the lane's four sines and cosines serve
// all heads that the group takes of its token.
#include <cuda_bf16.h>

#include "wq_internal.h"
#include "wq_tc.cuh"

namespace wq {

namespace {

struct RopeArgs {
    wq_rope r;
    int rows;       // heads a token: q, k and (with a cache and v) v
    int runs;       // ceil(rows / heads a group)
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

template <int LG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
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

// LG lanes a head, HU heads a group
template <int LG, int HU, bool VEC, bool ADJ, bool F32>
__global__ void __launch_bounds__(128) rope_kernel(const __grid_constant__ RopeArgs a) {
    sm100::grid_dependency_wait();
    sm100::grid_dependents_launch();
    const wq_rope& r = a.r;
    const int g = blockIdx.x * (128 / LG) + threadIdx.x / LG;
    // groups past the last one stay for the shuffles, with nothing to load or store
    const bool live = g < a.groups;
    const int t = live ? g / a.runs : 0;
    const int row0 = live ? (g - t * a.runs) * HU : a.rows;

    Place pl;
    pl.u = threadIdx.x % LG;
    pl.rot = a.rot_units;
    pl.R = r.rotary_dim;
    pl.D = r.head_dim;
    pl.rotated = pl.u < a.rot_units;
    pl.any = pl.u < a.units;

    Half8 x[HU];
    const int nq = r.q_heads, nk = r.q_heads + r.kv_heads;
#pragma unroll
    for (int j = 0; j < HU; ++j) {
        const int row = row0 + j;
        if (row >= a.rows) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j].a[e] = x[j].b[e] = 0.0f;
        } else if (row < nq) {
            load_head<VEC, ADJ, F32>(r.q, t * r.q_token + row * r.q_head, pl, x[j]);
        } else if (row < nk) {
            load_head<VEC, ADJ, F32>(r.k, t * r.k_token + (row - nq) * r.k_head, pl, x[j]);
        } else {
            load_head<VEC, ADJ, F32>(r.v, t * r.v_token + (row - nk) * r.v_head, pl, x[j]);
        }
    }

    // the lane's four turns
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        cs[e] = 1.0f;
        sn[e] = 0.0f;
    }
    if (pl.rotated && row0 < nk) {
        int pos[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pos[i] = i < r.axes ? r.positions[i * r.axis_stride + t] : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = 4 * pl.u + e;
            if (2 * p < pl.R) {
                const unsigned long long f = r.table[p];
                const int axis = (int)(f & 3);
                const int at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
                const unsigned long long turn = (unsigned long long)(long long)at * (f & ~3ull);
                sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn[e], &cs[e]);
            }
        }
    }

    long long cache_off = -1;
    if (r.with_cache && live) {
        const unsigned slot = (unsigned)r.slots[t];
        if (slot < (unsigned)r.cache.pages * (unsigned)r.cache.page_size) {
            const unsigned page = slot / (unsigned)r.cache.page_size;
            cache_off = page * r.cache.page_stride + (slot - page * (unsigned)r.cache.page_size) * r.cache.slot_stride;
        }
    }

    if (r.norm != WQ_HEAD_NORM_NONE) {
        if (r.norm == WQ_HEAD_NORM_LAYER) {
            float m[HU];
#pragma unroll
            for (int j = 0; j < HU; ++j) m[j] = sum8(x[j]);
#pragma unroll
            for (int j = 0; j < HU; ++j) m[j] = group_sum<LG>(m[j]) * a.inv_d;
#pragma unroll
            for (int j = 0; j < HU; ++j) {
                if (row0 + j >= nk) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // places without an element keep their zero
                    if (VEC ? pl.any : pl.elem<ADJ>(0, e) >= 0) x[j].a[e] -= m[j];
                    if (VEC ? pl.any : pl.elem<ADJ>(1, e) >= 0) x[j].b[e] -= m[j];
                }
            }
        }
        float s[HU];
#pragma unroll
        for (int j = 0; j < HU; ++j) s[j] = squares8(x[j]);
#pragma unroll
        for (int j = 0; j < HU; ++j) s[j] = group_sum<LG>(s[j]);
#pragma unroll
        for (int j = 0; j < HU; ++j) {
            const int row = row0 + j;
            if (row >= nk) continue;
            // one Newton step on rsqrtf (off by two units in the last place) makes
            // it good to fp32 outputs, and the same whatever the outputs' type is
            const float v = s[j] * a.inv_d + r.eps, r0 = rsqrtf(v);
            const float f = fmaf(0.5f * r0, fmaf(-v * r0, r0, 1.0f), r0);
            const void* w = row < nq ? r.q_weight : r.k_weight;
            const void* c = row < nq ? r.q_bias : r.k_bias;
            Half8 h;
            if (w) load_head<VEC, ADJ, false>(w, 0, pl, h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[j].a[e] *= w ? f * h.a[e] : f;
                x[j].b[e] *= w ? f * h.b[e] : f;
            }
            if (c) {
                load_head<VEC, ADJ, false>(c, 0, pl, h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[j].a[e] += h.a[e];
                    x[j].b[e] += h.b[e];
                }
            }
        }
    }

#pragma unroll
    for (int j = 0; j < HU; ++j) {
        const int row = row0 + j;
        if (row >= a.rows) continue;
        if (row >= nk) {
            if (cache_off >= 0)
                store_head<VEC, ADJ>(r.cache.v, false, cache_off + (row - nk) * r.cache.head_stride, pl, x[j]);
            continue;
        }
        Half8 y = x[j];
        if (pl.rotated) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y.a[e] = fmaf(x[j].a[e], cs[e], -(x[j].b[e] * sn[e]));
                y.b[e] = fmaf(x[j].b[e], cs[e], x[j].a[e] * sn[e]);
            }
        }
        const bool f32 = r.out_type == WQ_TYPE_F32;
        if (row < nq) {
            store_head<VEC, ADJ>(r.q_out, f32, t * r.q_out_token + row * r.q_out_head, pl, y);
        } else {
            if (r.k_out) store_head<VEC, ADJ>(r.k_out, f32, t * r.k_out_token + (row - nq) * r.k_out_head, pl, y);
            if (cache_off >= 0)
                store_head<VEC, ADJ>(r.cache.k, false, cache_off + (row - nq) * r.cache.head_stride, pl, y);
        }
    }
}

template <int LG, int HU>
cudaError_t launch_as(const RopeArgs& a, bool vec, bool adj, bool f32, cudaStream_t stream) {
    const unsigned per = 128 / LG, grid = ((unsigned)a.groups + per - 1) / per;
    auto go = [&](auto kern) { return launch_dependent(kern, grid, 128, 1, 0, stream, a); };
    if (f32)
        return vec ? (adj ? go(rope_kernel<LG, HU, true, true, true>) : go(rope_kernel<LG, HU, true, false, true>))
                   : (adj ? go(rope_kernel<LG, HU, false, true, true>) : go(rope_kernel<LG, HU, false, false, true>));
    return vec ? (adj ? go(rope_kernel<LG, HU, true, true, false>) : go(rope_kernel<LG, HU, true, false, false>))
               : (adj ? go(rope_kernel<LG, HU, false, true, false>) : go(rope_kernel<LG, HU, false, false, false>));
}

template <int HU>
cudaError_t launch_heads(RopeArgs& a, bool vec, bool adj, bool f32, cudaStream_t stream) {
    a.runs = (a.rows + HU - 1) / HU;
    a.groups = a.r.tokens * a.runs;
    return a.units <= 8    ? launch_as<8, HU>(a, vec, adj, f32, stream)
           : a.units <= 16 ? launch_as<16, HU>(a, vec, adj, f32, stream)
                           : launch_as<32, HU>(a, vec, adj, f32, stream);
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
    const cudaError_t e = many ? launch_heads<4>(a, vec, adj, f32, stream) : launch_heads<1>(a, vec, adj, f32, stream);
    return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

}  // namespace wq
