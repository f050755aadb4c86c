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
    const int32_t* row_src = nullptr;   // (quantise, bf16) the src row of each row, of src_rows
    int src_rows = 0;
};
hipError_t launch_mx_quantize(const MxRows& r, const void* src, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const MxRows& r, const uint8_t* codes, const uint8_t* scales, void* dst, hipStream_t s);


// ---- MX product (mx_product.hip)
struct MxProduct {
    int T, R, M, N, K, fmt;
    const uint16_t* x;          // [T] rows of K bf16, x_stride elements apart
    int64_t x_stride;
    const int32_t* row_src;     // [R] x row of each y row, or null (row r reads x row r)
    const int32_t* offsets;     // [M + 1] first y row of each matrix, or null (M = 1)
    const uint8_t* codes;       // [M][N][K/2] E2M1
    const uint8_t* scales;      // [M][K/128][N][4] E8M0
    uint16_t* y;                // [R] rows of N bf16, y_stride elements apart
    int64_t y_stride;
    int vec;                    // y rows take 4-, 8- or 16-byte stores (1, 2, 3) at every second, fourth or eighth column
    int xrows, gathered;        // rows of x in the workspace; gathered: row r is y row r's, else x row r
    uint8_t* xq;                // workspace: x's codes [xrows][K] or [xrows][K/2] ...
    uint8_t* xs;                // ... and scales [K/128][xrows][4]
};
size_t mx_product_ws_bytes(const MxProduct& a);
hipError_t launch_mx_product(MxProduct a, void* ws, hipStream_t s);

// ---- router load and losses (router_train.hip)
struct RouterLoad {
    int T, E, k, S, vec;            // vec: logit rows take 16-byte accesses
    int chunk;                      // tokens per workgroup
    const float* logits;            // [T][E]
    const int32_t* topk_idx;        // [T][k]
    const int32_t* seq_offsets;     // [S + 1] or null (S = 1: every token)
    int32_t* counts;                // [S][E]
    float* probs;                   // [S][E]
    float* loss;                    // [2]
    // workspace
    float* part_p; int32_t* part_c; // [chunks + S][E]
    double* part_z;                 // [chunks + S]
    double* dots;                   // [S * E / 64][2]
    uint32_t* done;
};
size_t router_load_ws_bytes(const RouterLoad& a);
hipError_t launch_router_load(RouterLoad a, void* ws, hipStream_t s);

// ---- router backward (router_train.hip)
struct RouterGrad {
    int T, E, k, S, d, vec;
    int Tp, Ep;                     // T and E up to multiples of 32
    int bi, slices, xslices;        // tile rows of the products, token slices of dW_r, expert slices of dx
    int chunk;                      // tokens per workgroup of rt_dlogits
    const float* logits; const int32_t* topk_idx; const float* topk_w;
    const float* d_topk_w;          // [T][k] or null
    const float* d_loss;            // [2] or null
    const int32_t* counts; const int32_t* seq_offsets;
    const uint16_t* x; const uint16_t* w_router;
    float* dlogits; float* dx; float* dw_router; float* dbias;   // each may be null
    // workspace
    uint16_t* planes;               // [3][Tp][Ep] bf16: dz = their sum
    float* part_w; float* part_x;   // [slices][E][d]; [xslices][T][d] (unless 1)
    float* part_b;                  // [Tp / chunk][E]
};
size_t router_grad_ws_bytes(RouterGrad a);
hipError_t launch_router_grad(RouterGrad a, void* ws, hipStream_t s);

}  // namespace em
