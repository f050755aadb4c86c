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

}  // extern "C"
