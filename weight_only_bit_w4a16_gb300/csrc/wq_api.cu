// wq_api.cu -- the C ABI (include/wq.h): argument validation and kernel
// selection.  Nothing here computes; every step of the product runs in the
// kernels of wq_dequant.cu, wq_gemv.cu, wq_gemv_tma.cu, wq_tc.cu,
// wq_prepack.cu, wq_gemv_pre.cu, wq_fp4_quant.cu, wq_fp4_mm.cu, wq_norm.cu,
// wq_rope.cu and wq_attn.cu.
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "wq_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Shared checks of the weight description.  Returns WQ_OK or an error code.
int check_weights(const uint8_t* packed, const void* scales, const uint8_t* zeros, int N, int K,
                  int fmt, int group) {
    if (N < 0 || K < 0) return WQ_ERR_INVALID_ARG;
    if (fmt != WQ_NVFP4 && fmt != WQ_MXFP4 && fmt != WQ_INT4) return WQ_ERR_INVALID_ARG;
    if (group <= 0) return WQ_ERR_INVALID_ARG;
    if (fmt == WQ_NVFP4 && group != 16) return WQ_ERR_UNSUPPORTED;
    if (fmt == WQ_MXFP4 && group != 32) return WQ_ERR_UNSUPPORTED;
    if (fmt == WQ_INT4 && group % 32 != 0) return WQ_ERR_UNSUPPORTED;
    if (K % 32 != 0 || K % group != 0) return WQ_ERR_UNSUPPORTED;
    if (N > 0 && K > 0) {
        if (!packed || !scales) return WQ_ERR_INVALID_ARG;
        if (fmt == WQ_INT4 && !zeros) return WQ_ERR_INVALID_ARG;
        if (fmt != WQ_INT4 && zeros) return WQ_ERR_INVALID_ARG;
        if (!aligned(packed, 16)) return WQ_ERR_ALIGN;
        if (fmt == WQ_INT4 && !aligned(scales, 2)) return WQ_ERR_ALIGN;
    }
    return WQ_OK;
}

}  // namespace

#define WQ_EXPORT __attribute__((visibility("default")))

namespace {

int gemm_impl(const void* A, const uint8_t* packed, const void* scales, const uint8_t* zeros, void* C, int M,
              int N, int K, int format, int group, void* workspace, size_t workspace_bytes, void* stream,
              int path, const wq_epilogue* epi_in = nullptr) {
    if (format & ~(0xFF | WQ_OUT_F32)) return WQ_ERR_INVALID_ARG;
    const int fmt = format & 0xFF;
    const bool out_f32 = (format & WQ_OUT_F32) != 0;
    if (M < 0) return WQ_ERR_INVALID_ARG;
    if (path & ~(0xFF | WQ_LAUNCH_OVERLAP | WQ_LAUNCH_INPUTS_READY)) return WQ_ERR_INVALID_ARG;
    const bool inputs_ready = (path & WQ_LAUNCH_INPUTS_READY) != 0;
    const bool overlap = (path & WQ_LAUNCH_OVERLAP) != 0 || inputs_ready;
    path &= 0xFF;
    if (path != WQ_PATH_AUTO && path != WQ_PATH_GEMV && path != WQ_PATH_TC) return WQ_ERR_INVALID_ARG;
    if (workspace_bytes > 0 && !workspace) return WQ_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return WQ_ERR_ALIGN;
    int st = check_weights(packed, scales, zeros, N, K, fmt, group);
    if (st != WQ_OK) return st;
    if (M == 0 || N == 0) return WQ_OK;
    if (!C || (K > 0 && !A)) return WQ_ERR_INVALID_ARG;
    if (!aligned(C, 16) || (K > 0 && !aligned(A, 16))) return WQ_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (workspace_bytes == 0) workspace = nullptr;
    wq::Epilogue epi{nullptr, nullptr, 0};
    if (epi_in) {
        if (epi_in->gated != 0 && epi_in->gated != 1) return WQ_ERR_INVALID_ARG;
        if (epi_in->gated && N % 16 != 0) return WQ_ERR_UNSUPPORTED;
        if (!aligned(epi_in->bias, 2) || !aligned(epi_in->residual, 2)) return WQ_ERR_ALIGN;
        epi.bias = static_cast<const uint16_t*>(epi_in->bias);
        epi.residual = static_cast<const uint16_t*>(epi_in->residual);
        epi.gated = epi_in->gated;
    }

    if (path == WQ_PATH_TC)
        return wq::launch_tc(A, packed, scales, zeros, C, M, N, K, fmt, group, out_f32, workspace, workspace_bytes,
                             epi, overlap, s);
    if (path == WQ_PATH_AUTO && M > 16 && K > 0) {
        st = wq::launch_tc(A, packed, scales, zeros, C, M, N, K, fmt, group, out_f32, workspace, workspace_bytes,
                           epi, overlap, s);
        if (st != WQ_ERR_UNSUPPORTED) return st;
        // shapes the tensor-core kernel does not take run on the GEMV kernel
    }
    return wq::launch_gemv(A, packed, scales, zeros, C, M, N, K, fmt, group, out_f32, overlap, inputs_ready, epi, s);
}

}  // namespace

extern "C" {

WQ_EXPORT int wq_gemm_ex(const void* A, const uint8_t* packed, const void* scales, const uint8_t* zeros, void* C,
               int M, int N, int K, int format, int group, void* stream, int path) {
    return gemm_impl(A, packed, scales, zeros, C, M, N, K, format, group, nullptr, 0, stream, path);
}

WQ_EXPORT int wq_gemm_ws(const void* A, const uint8_t* packed, const void* scales, const uint8_t* zeros, void* C,
               int M, int N, int K, int format, int group, void* workspace, size_t workspace_bytes, void* stream,
               int path) {
    return gemm_impl(A, packed, scales, zeros, C, M, N, K, format, group, workspace, workspace_bytes, stream, path);
}

WQ_EXPORT int wq_gemm_static(const void* A, const uint8_t* packed, const void* scales, const uint8_t* zeros,
                             void* C, int M, int N, int K, int format, int group, void* stream, int path) {
    // the description first, as every entry point checks it
    if (format & ~(0xFF | WQ_OUT_F32)) return WQ_ERR_INVALID_ARG;
    if (M < 0) return WQ_ERR_INVALID_ARG;
    if (path & ~(0xFF | WQ_LAUNCH_OVERLAP | WQ_LAUNCH_INPUTS_READY)) return WQ_ERR_INVALID_ARG;
    const int route = path & 0xFF;
    if (route != WQ_PATH_AUTO && route != WQ_PATH_GEMV && route != WQ_PATH_TC) return WQ_ERR_INVALID_ARG;
    int st = check_weights(packed, scales, zeros, N, K, format & 0xFF, group);
    if (st != WQ_OK) return st;
    size_t cap = 0;
    void* ws = wq::static_workspace(&cap, static_cast<cudaStream_t>(stream), &st);
    if (!ws) return st != WQ_OK ? st : WQ_ERR_CUDA;
    if (const char* e = getenv("WQ_STATIC_WS_CAP")) {   // tests: a smaller usable part
        const size_t v = (size_t)strtoull(e, nullptr, 10);
        if (v < cap) cap = v;
    }
    // the scratch matters only where the tensor-core kernel runs
    const bool tc = route == WQ_PATH_TC || (route == WQ_PATH_AUTO && M > 16);
    const size_t need = (tc && N > 0 && K > 0 && K % 64 == 0) ? wq::tc_workspace_bytes(M, N, K, format & 0xFF) : 0;
    if (need > cap) return WQ_ERR_UNSUPPORTED;
    return gemm_impl(A, packed, scales, zeros, C, M, N, K, format, group, ws, cap, stream, path);
}

WQ_EXPORT int wq_gemm_fused(const void* A, const uint8_t* packed, const void* scales, const uint8_t* zeros, void* C,
                            int M, int N, int K, int format, int group, const wq_epilogue* epilogue,
                            void* workspace, size_t workspace_bytes, void* stream, int path) {
    return gemm_impl(A, packed, scales, zeros, C, M, N, K, format, group, workspace, workspace_bytes, stream, path,
                     epilogue);
}

WQ_EXPORT size_t wq_gemm_workspace_size(int M, int N, int K, int format, int group) {
    if (M <= 16 || N <= 0 || K <= 0) return 0;
    if (check_weights(reinterpret_cast<const uint8_t*>(16), reinterpret_cast<const void*>(16),
                      (format & 0xFF) == WQ_INT4 ? reinterpret_cast<const uint8_t*>(16) : nullptr, N, K,
                      format & 0xFF, group) != WQ_OK)
        return 0;
    return wq::tc_workspace_bytes(M, N, K, format & 0xFF);
}

WQ_EXPORT size_t wq_workspace_bytes(int M, int N, int K, int format, int group) {
    return wq_gemm_workspace_size(M, N, K, format, group);
}

WQ_EXPORT int wq_gemm(const void* A, const uint8_t* packed, const void* scales, const uint8_t* zeros, void* C, int M,
            int N, int K, int format, int group) {
    return wq_gemm_ex(A, packed, scales, zeros, C, M, N, K, format, group, nullptr, WQ_PATH_AUTO);
}

// prepack takes int4 g128, NVFP4 g16, MXFP4 g32 and positive N, K (K a
// multiple of 32 and of the group, as everywhere)
static bool prepack_desc_ok(int N, int K, int fmt, int group) {
    if (N <= 0 || K <= 0) return false;
    if (check_weights(reinterpret_cast<const uint8_t*>(16), reinterpret_cast<const void*>(16),
                      fmt == WQ_INT4 ? reinterpret_cast<const uint8_t*>(16) : nullptr, N, K, fmt, group) != WQ_OK)
        return false;
    return fmt != WQ_INT4 || group == 128;
}

WQ_EXPORT size_t wq_prepack_bytes(int N, int K, int format, int group) {
    if (format & ~0xFF) return 0;
    return prepack_desc_ok(N, K, format, group) ? wq::prepack_bytes(N, K, format) : 0;
}

WQ_EXPORT int wq_prepack(const uint8_t* packed, const void* scales, const uint8_t* zeros, void* prepacked,
                         size_t prepacked_bytes, int N, int K, int format, int group, void* stream) {
    if (format & ~0xFF) return WQ_ERR_INVALID_ARG;
    int st = check_weights(packed, scales, zeros, N, K, format, group);
    if (st != WQ_OK) return st;
    if (!prepack_desc_ok(N, K, format, group)) return WQ_ERR_UNSUPPORTED;
    if (!prepacked) return WQ_ERR_INVALID_ARG;
    if (prepacked_bytes < wq::prepack_bytes(N, K, format)) return WQ_ERR_INVALID_ARG;
    if (!aligned(prepacked, 16)) return WQ_ERR_ALIGN;
    return wq::launch_prepack(packed, scales, zeros, prepacked, N, K, format, static_cast<cudaStream_t>(stream));
}

WQ_EXPORT int wq_gemm_prepacked(const void* A, const void* prepacked, void* C, int M, int N, int K, int format,
                                int group, const wq_epilogue* epilogue, void* workspace, size_t workspace_bytes,
                                void* stream, int path) {
    if (format & ~(0xFF | WQ_OUT_F32)) return WQ_ERR_INVALID_ARG;
    const int fmt = format & 0xFF;
    if (M < 0 || N < 0 || K < 0) return WQ_ERR_INVALID_ARG;
    if (path & ~(0xFF | WQ_LAUNCH_OVERLAP | WQ_LAUNCH_INPUTS_READY)) return WQ_ERR_INVALID_ARG;
    const bool inputs_ready = (path & WQ_LAUNCH_INPUTS_READY) != 0;
    const bool overlap = (path & WQ_LAUNCH_OVERLAP) != 0 || inputs_ready;
    const int route = path & 0xFF;
    if (route != WQ_PATH_AUTO && route != WQ_PATH_GEMV && route != WQ_PATH_TC) return WQ_ERR_INVALID_ARG;
    if (workspace_bytes > 0 && !workspace) return WQ_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return WQ_ERR_ALIGN;
    if (workspace_bytes == 0) workspace = nullptr;
    if (fmt != WQ_NVFP4 && fmt != WQ_MXFP4 && fmt != WQ_INT4) return WQ_ERR_INVALID_ARG;
    if (group <= 0) return WQ_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return WQ_OK;
    if (!prepack_desc_ok(N, K, fmt, group)) return WQ_ERR_UNSUPPORTED;
    if (!A || !prepacked || !C) return WQ_ERR_INVALID_ARG;
    if (!aligned(A, 16) || !aligned(C, 16) || !aligned(prepacked, 16)) return WQ_ERR_ALIGN;
    wq::Epilogue epi{nullptr, nullptr, 0};
    if (epilogue) {
        if (epilogue->gated != 0 && epilogue->gated != 1) return WQ_ERR_INVALID_ARG;
        if (epilogue->gated && N % 16 != 0) return WQ_ERR_UNSUPPORTED;
        if (!aligned(epilogue->bias, 2) || !aligned(epilogue->residual, 2)) return WQ_ERR_ALIGN;
        epi.bias = static_cast<const uint16_t*>(epilogue->bias);
        epi.residual = static_cast<const uint16_t*>(epilogue->residual);
        epi.gated = epilogue->gated;
    }
    const bool out_f32 = (format & WQ_OUT_F32) != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (route == WQ_PATH_TC)
        return wq::launch_tc_prepacked(A, prepacked, C, M, N, K, fmt, group, out_f32, workspace, workspace_bytes,
                                       epi, overlap, s);
    if (route == WQ_PATH_AUTO && M > 16) {
        const int st = wq::launch_tc_prepacked(A, prepacked, C, M, N, K, fmt, group, out_f32, workspace,
                                               workspace_bytes, epi, overlap, s);
        if (st != WQ_ERR_UNSUPPORTED) return st;
    }
    return wq::launch_gemv_prepacked(A, prepacked, C, M, N, K, fmt, out_f32, overlap, inputs_ready, epi, s);
}

WQ_EXPORT int wq_dequant(const uint8_t* packed, const void* scales, const uint8_t* zeros, void* W, int N, int K,
               int format, int group, void* stream) {
    if (format & ~0xFF) return WQ_ERR_INVALID_ARG;
    const int st = check_weights(packed, scales, zeros, N, K, format, group);
    if (st != WQ_OK) return st;
    if (N == 0 || K == 0) return WQ_OK;
    if (!W) return WQ_ERR_INVALID_ARG;
    if (!aligned(W, 16)) return WQ_ERR_ALIGN;
    return wq::launch_dequant(packed, scales, zeros, W, N, K, format, group, static_cast<cudaStream_t>(stream));
}

// Sizes past this are refused by the product and the norms: their kernels step
// through tiles, blocks of rows and pieces of a row with 32-bit indices, the
// last of which ends up to 16383 past the size.
constexpr int kMaxSize = 0x7FFF0000;

// what the 4-bit calls take: an fp4 format, K a multiple of 32
static int check_fp4(int rows, int K, int format, int layout) {
    if (rows < 0 || K < 0) return WQ_ERR_INVALID_ARG;
    if (format != WQ_NVFP4 && format != WQ_MXFP4) return format == WQ_INT4 ? WQ_ERR_UNSUPPORTED : WQ_ERR_INVALID_ARG;
    if (layout != WQ_SCALES_ROWS && layout != WQ_SCALES_TILED) return WQ_ERR_INVALID_ARG;
    return K % 32 == 0 ? WQ_OK : WQ_ERR_UNSUPPORTED;
}

WQ_EXPORT size_t wq_fp4_scale_bytes(int rows, int K, int format, int layout) {
    if (check_fp4(rows, K, format, layout) != WQ_OK || rows == 0 || K == 0) return 0;
    return wq::fp4_scale_bytes(rows, K, format, layout == WQ_SCALES_TILED);
}

WQ_EXPORT int wq_fp4_quantize(const wq_fp4_quant* args, void* stream) {
    if (!args) return WQ_ERR_INVALID_ARG;
    const wq_fp4_quant& q = *args;
    const int st = check_fp4(q.rows, q.K, q.format, q.layout);
    if (st != WQ_OK) return st;
    if (q.x_type != WQ_TYPE_BF16 && q.x_type != WQ_TYPE_F32) return WQ_ERR_INVALID_ARG;
    if (q.tensor_scale && q.format != WQ_NVFP4) return WQ_ERR_UNSUPPORTED;
    if (q.rows == 0 || q.K == 0) return WQ_OK;
    if (!q.x || !q.packed || !q.scales || (q.rows > 1 && q.ldx < q.K)) return WQ_ERR_INVALID_ARG;
    if (!aligned(q.packed, 16) || !aligned(q.values, 16) || !aligned(q.tensor_scale, 4) ||
        !aligned(q.x, q.x_type == WQ_TYPE_F32 ? 4 : 2) || (q.layout == WQ_SCALES_TILED && !aligned(q.scales, 16)))
        return WQ_ERR_ALIGN;
    return wq::launch_fp4_quantize(q.x, q.x_type == WQ_TYPE_F32, q.ldx, q.rows, q.K, q.format, q.tensor_scale, q.packed,
                                   q.scales, q.layout == WQ_SCALES_TILED, q.values, static_cast<cudaStream_t>(stream));
}

WQ_EXPORT int wq_fp4_tile_scales(const uint8_t* scales, uint8_t* tiled, int rows, int K, int format, void* stream) {
    const int st = check_fp4(rows, K, format, WQ_SCALES_TILED);
    if (st != WQ_OK) return st;
    if (rows == 0 || K == 0) return WQ_OK;
    if (!scales || !tiled) return WQ_ERR_INVALID_ARG;
    if (!aligned(tiled, 16)) return WQ_ERR_ALIGN;
    return wq::launch_fp4_tile_scales(scales, tiled, rows, K, format, static_cast<cudaStream_t>(stream));
}

WQ_EXPORT int wq_block_norm(const wq_norm* args, void* stream) {
    if (!args) return WQ_ERR_INVALID_ARG;
    const wq_norm& n = *args;
    auto type_ok = [](int t) { return t == WQ_TYPE_BF16 || t == WQ_TYPE_F32; };
    auto elem = [](int t) { return (uintptr_t)(t == WQ_TYPE_F32 ? 4 : 2); };
    const bool fp4 = n.out_type == WQ_NORM_OUT_NVFP4 || n.out_type == WQ_NORM_OUT_MXFP4;
    if (n.rows < 0 || n.d < 0 || (n.kind != WQ_NORM_RMS && n.kind != WQ_NORM_LAYER)) return WQ_ERR_INVALID_ARG;
    if (n.post != 0 && n.post != 1) return WQ_ERR_INVALID_ARG;
    if (!type_ok(n.x_type) || !type_ok(n.branch_type)) return WQ_ERR_INVALID_ARG;
    if (n.out_type < WQ_NORM_OUT_NONE || n.out_type > WQ_NORM_OUT_MXFP4) return WQ_ERR_INVALID_ARG;
    if (!n.branch && (n.post || n.gate)) return WQ_ERR_INVALID_ARG;
    if (!n.post && (n.post_weight || n.post_bias)) return WQ_ERR_INVALID_ARG;
    if (n.gate && (n.gate_rows <= 0 || n.rows % n.gate_rows != 0)) return WQ_ERR_INVALID_ARG;
    if (fp4) {
        const int format = n.out_type == WQ_NORM_OUT_NVFP4 ? WQ_NVFP4 : WQ_MXFP4;
        const int st = check_fp4(n.rows, n.d, format, n.out_scale_layout);
        if (st != WQ_OK) return st;
        if (n.out_tensor_scale && format != WQ_NVFP4) return WQ_ERR_UNSUPPORTED;
    }
    if (n.rows > kMaxSize || n.d > kMaxSize) return WQ_ERR_UNSUPPORTED;
    if (n.rows == 0 || n.d == 0) return WQ_OK;
    if (!n.x || (n.out_type == WQ_NORM_OUT_NONE ? !n.x_out : !n.out)) return WQ_ERR_INVALID_ARG;
    if (fp4 && !n.out_scales) return WQ_ERR_INVALID_ARG;
    if (n.rows > 1 && (n.ldx < n.d || (n.branch && n.ldb < n.d) || (n.x_out && n.ldxo < n.d) ||
                       (n.out_type != WQ_NORM_OUT_NONE && !fp4 && n.ldo < n.d)))
        return WQ_ERR_INVALID_ARG;
    if (!aligned(n.x, elem(n.x_type)) || !aligned(n.x_out, elem(n.x_type)) ||
        !aligned(n.branch, elem(n.branch_type)) || !aligned(n.gate, 2) || !aligned(n.weight, 2) ||
        !aligned(n.bias, 2) || !aligned(n.post_weight, 2) || !aligned(n.post_bias, 2))
        return WQ_ERR_ALIGN;
    if (fp4 ? !aligned(n.out, 16) || !aligned(n.out_tensor_scale, 4) ||
                  (n.out_scale_layout == WQ_SCALES_TILED && !aligned(n.out_scales, 16))
            : !aligned(n.out, n.out_type == WQ_NORM_OUT_F32 ? 4 : 2))
        return WQ_ERR_ALIGN;
    return wq::launch_block_norm(n, static_cast<cudaStream_t>(stream));
}

WQ_EXPORT int wq_gemm_fp4(const wq_fp4_gemm* args, void* stream) {
    if (!args) return WQ_ERR_INVALID_ARG;
    const wq_fp4_gemm& g = *args;
    if (g.format & ~(0xFF | WQ_OUT_F32)) return WQ_ERR_INVALID_ARG;
    const int fmt = g.format & 0xFF;
    if (g.M < 0 || g.N < 0) return WQ_ERR_INVALID_ARG;
    if (g.path & ~(0xFF | WQ_LAUNCH_OVERLAP | WQ_LAUNCH_INPUTS_READY)) return WQ_ERR_INVALID_ARG;
    const int route = g.path & 0xFF;
    if (route == WQ_PATH_GEMV) return WQ_ERR_UNSUPPORTED;
    if (route != WQ_PATH_AUTO && route != WQ_PATH_TC) return WQ_ERR_INVALID_ARG;
    const int st = check_fp4(g.M, g.K, fmt, WQ_SCALES_TILED);
    if (st != WQ_OK) return st;
    if (g.M > kMaxSize || g.N > kMaxSize || g.K > kMaxSize) return WQ_ERR_UNSUPPORTED;
    if ((g.a_tensor_scale || g.b_tensor_scale) && fmt != WQ_NVFP4) return WQ_ERR_UNSUPPORTED;
    if (g.epilogue.gated != 0 && g.epilogue.gated != 1) return WQ_ERR_INVALID_ARG;
    if (g.epilogue.gated && g.N % 16 != 0) return WQ_ERR_UNSUPPORTED;
    if (!aligned(g.epilogue.bias, 2) || !aligned(g.epilogue.residual, 2)) return WQ_ERR_ALIGN;
    const wq::Epilogue epi{static_cast<const uint16_t*>(g.epilogue.bias),
                           static_cast<const uint16_t*>(g.epilogue.residual), g.epilogue.gated};
    if (g.M == 0 || g.N == 0) return WQ_OK;
    if (!g.C || (g.K > 0 && (!g.a_packed || !g.a_scales || !g.b_packed || !g.b_scales))) return WQ_ERR_INVALID_ARG;
    if (!aligned(g.C, 16) || !aligned(g.a_tensor_scale, 4) || !aligned(g.b_tensor_scale, 4)) return WQ_ERR_ALIGN;
    if (g.K > 0 && (!aligned(g.a_packed, 16) || !aligned(g.b_packed, 16) || !aligned(g.a_scales, 16) ||
                    !aligned(g.b_scales, 16)))
        return WQ_ERR_ALIGN;
    return wq::launch_gemm_fp4({g.a_packed, g.a_scales, g.a_tensor_scale}, {g.b_packed, g.b_scales, g.b_tensor_scale},
                               g.C, g.M, g.N, g.K, fmt, (g.format & WQ_OUT_F32) != 0, epi,
                               (g.path & (WQ_LAUNCH_OVERLAP | WQ_LAUNCH_INPUTS_READY)) != 0,
                               static_cast<cudaStream_t>(stream));
}

WQ_EXPORT int wq_rope_table(const double* inv_freq, const int* axis, int pairs, unsigned long long* table) {
    if (pairs < 0) return WQ_ERR_INVALID_ARG;
    if (pairs == 0) return WQ_OK;
    if (!inv_freq || !table) return WQ_ERR_INVALID_ARG;
    // 1 / (2 pi) as the sum of two doubles
    constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    for (int i = 0; i < pairs; ++i) {
        const double f = inv_freq[i];
        const int ax = axis ? axis[i] : 0;
        if (!std::isfinite(f) || ax < 0 || ax > 3) return WQ_ERR_INVALID_ARG;
        // |f| / (2 pi) modulo 1 in units of 2^-62, from a product of twice the
        // precision: its leading part's fraction is exact, the rest is small
        const double m = std::fabs(f), p = m * hi, e = std::fma(m, hi, -p) + m * lo;
        const unsigned long long turn =
            (unsigned long long)std::nearbyint((p - std::floor(p)) * 0x1p62) +
            (unsigned long long)(long long)std::nearbyint((e - std::trunc(e)) * 0x1p62);
        const unsigned long long n = f < 0.0 ? 0ull - turn : turn;
        table[i] = (n << 2) | (unsigned)ax;
    }
    return WQ_OK;
}

// the cache of the calls below, as a description
static int check_cache(const wq_kv_cache& c) {
    if (c.pages < 0 || c.page_size <= 0) return WQ_ERR_INVALID_ARG;
    if ((long long)c.pages * c.page_size > 0x7FFFFFFFLL) return WQ_ERR_UNSUPPORTED;
    return WQ_OK;
}

WQ_EXPORT int wq_head_rope(const wq_rope* args, void* stream) {
    if (!args) return WQ_ERR_INVALID_ARG;
    const wq_rope& r = *args;
    auto type_ok = [](int t) { return t == WQ_TYPE_BF16 || t == WQ_TYPE_F32; };
    auto elem = [](int t) { return (uintptr_t)(t == WQ_TYPE_F32 ? 4 : 2); };
    if (r.tokens < 0 || r.q_heads < 0 || r.kv_heads < 0 || r.head_dim < 0) return WQ_ERR_INVALID_ARG;
    if (!type_ok(r.type) || !type_ok(r.out_type)) return WQ_ERR_INVALID_ARG;
    if (r.norm < WQ_HEAD_NORM_NONE || r.norm > WQ_HEAD_NORM_LAYER) return WQ_ERR_INVALID_ARG;
    if (r.pairs != WQ_PAIRS_HALVES && r.pairs != WQ_PAIRS_ADJACENT) return WQ_ERR_INVALID_ARG;
    if (r.rotary_dim < 0 || r.rotary_dim > r.head_dim || r.rotary_dim % 2 != 0) return WQ_ERR_INVALID_ARG;
    if (r.with_cache != 0 && r.with_cache != 1) return WQ_ERR_INVALID_ARG;
    if (r.norm == WQ_HEAD_NORM_NONE && (r.q_weight || r.q_bias || r.k_weight || r.k_bias)) return WQ_ERR_INVALID_ARG;
    if (r.rotary_dim > 0 && (r.axes < 1 || r.axes > 4)) return WQ_ERR_INVALID_ARG;
    if (r.with_cache) {
        const int st = check_cache(r.cache);
        if (st != WQ_OK) return st;
    }
    if (r.tokens == 0 || r.head_dim == 0 || (r.q_heads == 0 && r.kv_heads == 0)) return WQ_OK;
    if (r.head_dim > 256 || wq::rope_units(r.head_dim, r.rotary_dim) > 32) return WQ_ERR_UNSUPPORTED;
    if ((long long)r.tokens * ((long long)r.q_heads + 2LL * r.kv_heads) > kMaxSize) return WQ_ERR_UNSUPPORTED;
    if (r.q_heads > 0 && (!r.q || !r.q_out)) return WQ_ERR_INVALID_ARG;
    if (r.kv_heads > 0 && (!r.k || (!r.k_out && !r.with_cache))) return WQ_ERR_INVALID_ARG;
    if (r.rotary_dim > 0 && (!r.table || !r.positions)) return WQ_ERR_INVALID_ARG;
    if (r.with_cache && r.kv_heads > 0 && (!r.v || !r.slots)) return WQ_ERR_INVALID_ARG;
    if (r.with_cache && r.kv_heads > 0 && r.cache.pages > 0 && (!r.cache.k || !r.cache.v)) return WQ_ERR_INVALID_ARG;
    if (!aligned(r.q, elem(r.type)) || !aligned(r.k, elem(r.type)) || !aligned(r.v, elem(r.type)) ||
        !aligned(r.q_out, elem(r.out_type)) || !aligned(r.k_out, elem(r.out_type)) || !aligned(r.q_weight, 2) ||
        !aligned(r.q_bias, 2) || !aligned(r.k_weight, 2) || !aligned(r.k_bias, 2) || !aligned(r.table, 8) ||
        !aligned(r.positions, 4) || !aligned(r.slots, 4) ||
        (r.with_cache && (!aligned(r.cache.k, 2) || !aligned(r.cache.v, 2))))
        return WQ_ERR_ALIGN;
    return wq::launch_rope(r, static_cast<cudaStream_t>(stream));
}

constexpr int kMaxSequences = 1024;   // their plan is held in shared memory

static bool attention_shape_ok(int tokens, int sequences, int q_heads, int kv_heads, int head_dim) {
    return head_dim % 8 == 0 && head_dim >= 8 && head_dim <= 128 && kv_heads > 0 && q_heads % kv_heads == 0 &&
           sequences <= kMaxSequences && (long long)tokens * q_heads <= kMaxSize / 128;
}

WQ_EXPORT size_t wq_prefix_attention_workspace(int tokens, int sequences, int q_heads, int kv_heads, int head_dim) {
    if (tokens <= 0 || sequences <= 0 || q_heads <= 0 ||
        !attention_shape_ok(tokens, sequences, q_heads, kv_heads, head_dim))
        return 0;
    return wq::attn_workspace_bytes(tokens, sequences, q_heads, kv_heads, head_dim);
}

WQ_EXPORT int wq_prefix_attention(const wq_attention* args, void* stream) {
    if (!args) return WQ_ERR_INVALID_ARG;
    const wq_attention& t = *args;
    if (t.tokens < 0 || t.sequences < 0 || t.q_heads < 0 || t.kv_heads < 0 || t.head_dim < 0 || t.prefix_len < 0 ||
        t.prefix_table_pages < 0 || t.table_pages < 0)
        return WQ_ERR_INVALID_ARG;
    if (!(t.scale > 0.0f) || !std::isfinite(t.scale)) return WQ_ERR_INVALID_ARG;
    int st = check_cache(t.cache);
    if (st != WQ_OK) return st;
    if (t.tokens == 0 || t.q_heads == 0 || t.head_dim == 0) return WQ_OK;
    if (t.sequences == 0) return t.q_start ? WQ_OK : WQ_ERR_INVALID_ARG;
    if (!t.q_start && t.tokens % t.sequences != 0) return WQ_ERR_INVALID_ARG;
    if (!attention_shape_ok(t.tokens, t.sequences, t.q_heads, t.kv_heads, t.head_dim)) return WQ_ERR_UNSUPPORTED;
    if (t.cache.page_size % 16 != 0) return WQ_ERR_UNSUPPORTED;
    if ((long long)t.table_pages * t.cache.page_size > 0x7FFF0000LL || t.prefix_len > 0x7FFF0000)
        return WQ_ERR_UNSUPPORTED;
    if (!t.q || !t.out || !t.seq_lens || (t.table_pages > 0 && !t.tables)) return WQ_ERR_INVALID_ARG;
    if (t.prefix_len > 0 && (!t.prefix_pages || (long long)t.prefix_table_pages * t.cache.page_size < t.prefix_len))
        return WQ_ERR_INVALID_ARG;
    if (t.table_pages > 0 && t.sequences > 1 && t.table_stride < t.table_pages) return WQ_ERR_INVALID_ARG;
    if ((t.table_pages > 0 || t.prefix_len > 0) && (t.cache.pages == 0 || !t.cache.k || !t.cache.v))
        return WQ_ERR_INVALID_ARG;
    if (!aligned(t.q, 16) || !aligned(t.out, 16) || t.q_token % 8 || t.q_head % 8 || t.out_token % 8 ||
        t.out_head % 8 || !aligned(t.cache.k, 16) || !aligned(t.cache.v, 16) || t.cache.page_stride % 8 ||
        t.cache.slot_stride % 8 || t.cache.head_stride % 8 || !aligned(t.lse, 4) || !aligned(t.q_start, 4) ||
        !aligned(t.seq_lens, 4) || !aligned(t.tables, 4) || !aligned(t.prefix_pages, 4) || !aligned(t.workspace, 256))
        return WQ_ERR_ALIGN;
    if (!t.workspace ||
        t.workspace_bytes < wq::attn_workspace_bytes(t.tokens, t.sequences, t.q_heads, t.kv_heads, t.head_dim))
        return WQ_ERR_INVALID_ARG;
    return wq::launch_prefix_attention(t, static_cast<cudaStream_t>(stream));
}

WQ_EXPORT int wq_get_device_error(void) {
    const int a = wq::read_and_clear_device_status();
    const int b = wq::read_and_clear_gemv_status();
    const int c = wq::read_and_clear_pre_status();
    const int d = wq::read_and_clear_staged_status();
    const int e = wq::read_and_clear_fp4_status();
    const int f = wq::read_and_clear_attn_status();
    return a != 0 ? a : (b != 0 ? b : (c != 0 ? c : (d != 0 ? d : (e != 0 ? e : f))));
}

WQ_EXPORT int wq_selftest_timeout(void* stream) {
    return wq::launch_timeout_selftest(static_cast<cudaStream_t>(stream));
}

WQ_EXPORT const char* wq_status_string(int status) {
    switch (status) {
        case WQ_OK: return "WQ_OK";
        case WQ_ERR_INVALID_ARG: return "WQ_ERR_INVALID_ARG: null pointer, negative size or bad format/path";
        case WQ_ERR_UNSUPPORTED: return "WQ_ERR_UNSUPPORTED: shape or group not handled by the kernels";
        case WQ_ERR_ALIGN: return "WQ_ERR_ALIGN: pointer not aligned as required";
        case WQ_ERR_CUDA: return "WQ_ERR_CUDA: a CUDA runtime call or kernel launch failed";
        case WQ_ERR_DEVICE_TIMEOUT: return "WQ_ERR_DEVICE_TIMEOUT: a bounded device-side wait ran out";
        default: return "unknown wq status";
    }
}

WQ_EXPORT int wq_version(void) { return 100; }

}  // extern "C"
