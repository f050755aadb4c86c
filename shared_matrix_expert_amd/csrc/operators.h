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
    const uint8_t* xq;          // workspace: x's codes [xrows][K] or [xrows][K/2] ...
    const uint8_t* xs;          // ... and scales [K/128][xrows][4]
};
size_t mx_product_ws_bytes(const MxProduct& a);
hipError_t launch_mx_product(MxProduct a, void* ws, hipStream_t s);
hipError_t launch_mx_product_coded(MxProduct a, hipStream_t s);   // xq, xs: the caller's, [T] rows

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

// ---- norm (norm.hip)
struct NormFwd {
    int T, d;
    float eps;
    const uint16_t* x; int64_t x_stride;                 // strides in elements
    const void* add; int64_t add_stride; int add_f32;    // null: nothing to add
    const void* gain; int gain_f32;
    uint16_t* x_out; int64_t xo_stride;                  // each output may be null
    uint16_t* y; int64_t y_stride;
    uint8_t* codes; uint8_t* scales;                     // [T][d] E4M3, [d/128][T][4] E8M0
    float* rstd;
    double per_d;                                        // 1 / d
    int t0;                                              // a launch's first row
};
hipError_t launch_norm_forward(NormFwd a, hipStream_t s);
struct NormBwd {
    int T, d;
    const uint16_t* x; int64_t x_stride;
    const void* gain; int gain_f32;
    const float* rstd;
    const void* dy; int64_t dy_stride;
    const void* dres; int64_t dres_stride;               // null: nothing
    void* dx; int64_t dx_stride;                         // null: not computed
    float* dgain;                                        // null: not computed
    int f32;                                             // dy, dres, dx
    int chunk; double per_d;                             // rows a workgroup, 1 / d
    float* part;                                         // workspace: [workgroups or runs of rows][d]
};
size_t norm_backward_ws_bytes(int T, int d);
hipError_t launch_norm_backward(NormBwd a, void* ws, hipStream_t s);

// ---- products with bf16 matrices and their gradients (dense_product.hip)
struct DenseProduct {
    int T, R, M, N, K;
    const uint16_t* x; int64_t x_stride;
    const int32_t* row_src;     // [R] x row of each y row, or null (row r reads x row r)
    const int32_t* offsets;     // [M + 1] first y row of each matrix, or null (M = 1)
    const uint16_t* w;          // [M][N][K]
    const uint16_t* dy; int64_t dy_stride;
    void* out; int64_t out_stride; int out_f32;
    int slices, row_tiles, to_part;
    int col0, cols;             // columns of out that a launch makes
    const int32_t* map; const int32_t* passes; int pass_steps;   // dx of tokens in one sum: rows by token and matrix
    float* part;                // workspace: [slices][rows][columns] of out
};
struct DenseGrad {
    DenseProduct p;
    void* dx; int64_t dx_stride; int dx_f32;
    const int32_t* token_rows; int per_token;            // [T][per_token] rows of each token, or null: dx by rows
    void* dw; int dw_f32;
};
// Sums of the slices of `rows` rows, in order: out row i from row i, or from the rows of
// token i (dense_product.hip).
struct RowJoin {
    const float* part;              // [slices][rows][cols up to a multiple of 4]
    int slices;
    int64_t rows;
    int cols;
    void* out; int64_t out_stride; int out_f32;
    int whole;                      // out rows take four columns at once
    int64_t out_rows;
    const int32_t* offsets; int M;  // rows offsets[0] .. offsets[M] - 1 are written; null: all
    const int32_t* token_rows; int per_token;
};
hipError_t launch_join(const RowJoin& j, hipStream_t s);
size_t dense_product_ws_bytes(const DenseProduct& a);
hipError_t launch_dense_product(DenseProduct a, void* ws, hipStream_t s);
size_t dense_backward_ws_bytes(const DenseProduct& a);
hipError_t launch_dense_backward(const DenseGrad& g, void* ws, hipStream_t s);

// ---- product with int4 matrices (int4_product.hip)
struct Int4Product {
    int T, R, M, N, K, gq;      // gq: elements of a scale, at most K
    const uint16_t* x; int64_t x_stride;
    const int32_t* row_src;     // [R] x row of each y row, or null (row r reads x row r)
    const int32_t* offsets;     // [M + 1] first y row of each matrix, or null (M = 1)
    const uint8_t* codes;       // [M][N][K/2]
    const uint16_t* scales;     // [M][N][K/gq] fp16
    void* y; int64_t y_stride; int y_f32;
    int vec;                    // y rows take 16-byte stores (8 bf16, 4 float32) at every eighth or fourth column
    int slices, row_tiles;
    int tile0;                  // a launch's first row tile
    float* part;                // workspace: [slices][R][N up to a multiple of 4]
};
size_t int4_product_ws_bytes(const Int4Product& a);
hipError_t launch_int4_product(Int4Product a, void* ws, hipStream_t s);

}  // namespace em
