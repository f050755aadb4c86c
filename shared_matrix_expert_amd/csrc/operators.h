// Internal launch interface of the MX-matrix and router-training operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct edge_moe_dims;

namespace em {

// kernel timing hooks and host checks (api.hip)
void prof_begin(hipStream_t s);
void prof_end(hipStream_t s, const char* name);
int layer_dims_status(const edge_moe_dims* d);   // the layer's shape checks: EDGE_MOE_*
int device_status();                             // EDGE_MOE_OK on a gfx950 device

// ---- MX quantiser (mx_quant.hip): `rows` rows of K elements, N rows a matrix
struct MxRows {
    int64_t rows;        // M * N
    int N, K;
    int64_t stride;      // elements between rows of the dense side
    int fmt;             // kMxFp4, kMxFp8
    int f32;             // dense side float32 (else bf16)
};
hipError_t launch_mx_quantize(const MxRows& r, const void* src, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const MxRows& r, const uint8_t* codes, const uint8_t* scales, void* dst, hipStream_t s);

}  // namespace em
