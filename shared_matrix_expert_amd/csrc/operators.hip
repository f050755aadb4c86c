// C-ABI entry points of the MX-matrix operators: validation and launches.
#include <hip/hip_runtime.h>

#include "edge_moe.h"
#include "operators.h"

namespace {

bool aligned(const void* p, size_t a) { return p && ((uintptr_t)p % a) == 0; }

// M matrices of N rows x K in the MX layouts.
int mx_shape_status(int32_t M, int32_t N, int32_t K) {
    if (M < 1 || N < 1 || K < 1) return EDGE_MOE_EINVAL;
    if (K % 128 || K > 32768 || (int64_t)M * N > (1ll << 30)) return EDGE_MOE_EUNSUPPORTED;
    return EDGE_MOE_OK;
}

int mx_rows_status(int32_t M, int32_t N, int32_t K, int32_t format, int32_t type, const void* dense, int64_t stride,
                   const uint8_t* codes, const uint8_t* scales, em::MxRows* r) {
    if ((format != EDGE_MOE_MX_FP4 && format != EDGE_MOE_MX_FP8) || (type != EDGE_MOE_BF16 && type != EDGE_MOE_FLOAT))
        return EDGE_MOE_EINVAL;
    const int st = mx_shape_status(M, N, K);
    if (st != EDGE_MOE_OK) return st;
    if (!aligned(dense, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return EDGE_MOE_EINVAL;
    if (stride < K || stride > (1ll << 32) || stride * (type == EDGE_MOE_FLOAT ? 4 : 2) % 16) return EDGE_MOE_EINVAL;
    *r = em::MxRows{(int64_t)M * N, N, K, stride, format, type == EDGE_MOE_FLOAT};
    return em::device_status();
}

// Shape checks of the MX product: EDGE_MOE_*.
int mx_product_status(const edge_moe_mx_dims* d) {
    if (!d || d->T < 1 || d->R < 0 || d->M < 1 || (d->x_format != EDGE_MOE_MX_FP4 && d->x_format != EDGE_MOE_MX_FP8))
        return EDGE_MOE_EINVAL;
    const int st = mx_shape_status(d->M, d->N, d->K);
    if (st != EDGE_MOE_OK) return st;
    if (d->T > (1 << 20) || d->R > (1 << 25) || d->M > 1024 || d->N > 32768) return EDGE_MOE_EUNSUPPORTED;
    return EDGE_MOE_OK;
}

em::MxProduct mx_product_args(const edge_moe_mx_dims& d) {
    em::MxProduct a{};
    a.T = d.T; a.R = d.R; a.M = d.M; a.N = d.N; a.K = d.K; a.fmt = d.x_format;
    return a;
}

int hip_status(hipError_t e) { return e == hipSuccess ? EDGE_MOE_OK : EDGE_MOE_EHIP; }

}  // namespace

extern "C" {

int edge_moe_mx_quantize(int32_t M, int32_t N, int32_t K, int32_t format, int32_t src_type, const void* src,
                         int64_t src_stride, uint8_t* codes, uint8_t* scales, void* stream) {
    em::MxRows r;
    const int st = mx_rows_status(M, N, K, format, src_type, src, src_stride, codes, scales, &r);
    if (st != EDGE_MOE_OK) return st;
    return hip_status(em::launch_mx_quantize(r, src, codes, scales, (hipStream_t)stream));
}

int edge_moe_mx_dequantize(int32_t M, int32_t N, int32_t K, int32_t format, int32_t dst_type, const uint8_t* codes,
                           const uint8_t* scales, void* dst, int64_t dst_stride, void* stream) {
    em::MxRows r;
    const int st = mx_rows_status(M, N, K, format, dst_type, dst, dst_stride, codes, scales, &r);
    if (st != EDGE_MOE_OK) return st;
    return hip_status(em::launch_mx_dequantize(r, codes, scales, dst, (hipStream_t)stream));
}

size_t edge_moe_mx_product_ws_bytes(const edge_moe_mx_dims* dims) {
    if (mx_product_status(dims) != EDGE_MOE_OK) return 0;
    return em::mx_product_ws_bytes(mx_product_args(*dims));
}

int edge_moe_mx_product(const edge_moe_mx_dims* dims, const uint16_t* x, int64_t x_stride, const int32_t* row_src,
                        const int32_t* offsets, const uint8_t* codes, const uint8_t* scales, uint16_t* y,
                        int64_t y_stride, void* ws, size_t ws_bytes, void* stream) {
    int st = mx_product_status(dims);
    if (st != EDGE_MOE_OK) return st;
    const edge_moe_mx_dims& d = *dims;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || (d.R > 0 && !aligned(y, 2))) return EDGE_MOE_EINVAL;
    if ((row_src && !aligned(row_src, 4)) || (offsets && !aligned(offsets, 4))) return EDGE_MOE_EINVAL;
    if (x_stride < d.K || x_stride % 8 || x_stride > (1ll << 32) || y_stride < d.N || y_stride > (1ll << 32))
        return EDGE_MOE_EINVAL;
    if ((!offsets && d.M != 1) || (!row_src && d.R > d.T)) return EDGE_MOE_EINVAL;
    if (!ws) return EDGE_MOE_EWORKSPACE;
    if (!aligned(ws, 256)) return EDGE_MOE_EINVAL;
    em::MxProduct a = mx_product_args(d);
    if (ws_bytes < em::mx_product_ws_bytes(a)) return EDGE_MOE_EWORKSPACE;
    st = em::device_status();
    if (st != EDGE_MOE_OK) return st;
    if (d.R == 0) return EDGE_MOE_OK;
    a.x = x; a.x_stride = x_stride; a.row_src = row_src; a.offsets = offsets; a.codes = codes; a.scales = scales;
    a.y = y; a.y_stride = y_stride;
    a.vec = y_stride % 4 == 0 && aligned(y, 8);
    return hip_status(em::launch_mx_product(a, ws, (hipStream_t)stream));
}

}  // extern "C"
