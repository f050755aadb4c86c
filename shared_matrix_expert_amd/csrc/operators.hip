// C-ABI entry points of the operators around the expert layer (MX matrices, router
// training, norm, dense and int4 matrices): validation and launches.
#include <hip/hip_runtime.h>

#include "edge_moe.h"
#include "operators.h"

namespace {

bool aligned(const void* p, size_t a) { return p && ((uintptr_t)p % a) == 0; }

// M matrices of N rows x K in the MX layouts.  2^27 rows are 2^31 threads of the
// quantiser; a launch holds fewer than 2^32.
int mx_shape_status(int32_t M, int32_t N, int32_t K) {
    if (M < 1 || N < 1 || K < 1) return EDGE_MOE_EINVAL;
    if (K % 128 || K > 32768 || (int64_t)M * N > (1ll << 27)) return EDGE_MOE_EUNSUPPORTED;
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

// n_seq sequences of the batch's tokens: EDGE_MOE_*.
int seqs_status(const int32_t* seq_offsets, int32_t n_seq) {
    if (n_seq < 1 || (!seq_offsets && n_seq != 1) || (seq_offsets && !aligned(seq_offsets, 4))) return EDGE_MOE_EINVAL;
    return n_seq > 4095 ? EDGE_MOE_EUNSUPPORTED : EDGE_MOE_OK;
}

int ws_status(const void* ws, size_t ws_bytes, size_t need) {
    if (!ws) return EDGE_MOE_EWORKSPACE;
    if (!aligned(ws, 256)) return EDGE_MOE_EINVAL;
    return ws_bytes < need ? EDGE_MOE_EWORKSPACE : EDGE_MOE_OK;
}

em::RouterGrad grad_args(const edge_moe_dims& d) {
    em::RouterGrad a{};
    a.T = d.T; a.E = d.n_experts; a.k = d.top_k; a.d = d.d; a.S = 1;
    return a;
}

bool type_ok(int32_t t) { return t == EDGE_MOE_BF16 || t == EDGE_MOE_FLOAT; }
int type_bytes(int32_t t) { return t == EDGE_MOE_FLOAT ? 4 : 2; }

// Rows of `cols` elements at 16 bytes each, `stride` elements apart.
bool rows_ok(const void* p, int64_t stride, int64_t cols, int elem) {
    return aligned(p, 16) && stride >= cols && stride <= (1ll << 32) && stride * elem % 16 == 0;
}

int norm_shape_status(int32_t T, int32_t d) {
    if (T < 0 || d < 8 || d % 8) return EDGE_MOE_EINVAL;
    return T > (1 << 25) || d > 32768 ? EDGE_MOE_EUNSUPPORTED : EDGE_MOE_OK;
}

// Shape checks of the products with bf16 matrices: EDGE_MOE_*.
int dense_status(const edge_moe_dense_dims* d) {
    if (!d || d->T < 1 || d->R < 0 || d->M < 1 || d->N < 8 || d->K < 8 || d->N % 8 || d->K % 8) return EDGE_MOE_EINVAL;
    if (d->T > (1 << 20) || d->R > (1 << 25) || d->M > 1024 || d->N > 32768 || d->K > 32768) return EDGE_MOE_EUNSUPPORTED;
    return EDGE_MOE_OK;
}

em::DenseProduct dense_args(const edge_moe_dense_dims& d) {
    em::DenseProduct a{};
    a.T = d.T; a.R = d.R; a.M = d.M; a.N = d.N; a.K = d.K;
    return a;
}

// Shape checks of the product with int4 matrices: EDGE_MOE_*.
int int4_status(const edge_moe_packed_dims* d) {
    if (!d || d->T < 1 || d->R < 0 || d->M < 1 || d->N < 1 || d->K < 32 || d->K % 32) return EDGE_MOE_EINVAL;
    const int32_t q = d->quant_group;
    if (q < 32 || q > 4096 || (q & (q - 1)) || (q < d->K && d->K % q)) return EDGE_MOE_EINVAL;
    if (d->T > (1 << 20) || d->R > (1 << 25) || d->M > 1024 || d->N > 32768 || d->K > 32768) return EDGE_MOE_EUNSUPPORTED;
    return EDGE_MOE_OK;
}

em::Int4Product int4_args(const edge_moe_packed_dims& d) {
    em::Int4Product a{};
    a.T = d.T; a.R = d.R; a.M = d.M; a.N = d.N; a.K = d.K; a.gq = d.quant_group < d.K ? d.quant_group : d.K;
    return a;
}

// The batch's row lists: EDGE_MOE_*.
int lists_status(const int32_t* row_src, const int32_t* offsets, int T, int R, int M) {
    if ((row_src && !aligned(row_src, 4)) || (offsets && !aligned(offsets, 4))) return EDGE_MOE_EINVAL;
    return (!offsets && M != 1) || (!row_src && R > T) ? EDGE_MOE_EINVAL : EDGE_MOE_OK;
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
    em::MxProduct a = mx_product_args(d);
    st = ws_status(ws, ws_bytes, em::mx_product_ws_bytes(a));
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK) return st;
    if (d.R == 0) return EDGE_MOE_OK;
    a.x = x; a.x_stride = x_stride; a.row_src = row_src; a.offsets = offsets; a.codes = codes; a.scales = scales;
    a.y = y; a.y_stride = y_stride;
    a.vec = y_stride % 8 == 0 && aligned(y, 16) ? 3 : y_stride % 4 == 0 && aligned(y, 8) ? 2 : y_stride % 2 == 0 && aligned(y, 4) ? 1 : 0;
    return hip_status(em::launch_mx_product(a, ws, (hipStream_t)stream));
}

int edge_moe_mx_product_coded(const edge_moe_mx_dims* dims, const uint8_t* x_codes, const uint8_t* x_scales, const int32_t* row_src,
                              const int32_t* offsets, const uint8_t* codes, const uint8_t* scales, uint16_t* y,
                              int64_t y_stride, void* stream) {
    int st = mx_product_status(dims);
    if (st != EDGE_MOE_OK) return st;
    em::MxProduct a = mx_product_args(*dims);
    if (!aligned(x_codes, 16) || !aligned(x_scales, 4) || !aligned(codes, 16) || !aligned(scales, 4) || (a.R > 0 && !aligned(y, 2)))
        return EDGE_MOE_EINVAL;
    if (y_stride < a.N || y_stride > (1ll << 32)) return EDGE_MOE_EINVAL;
    st = lists_status(row_src, offsets, a.T, a.R, a.M);
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK || a.R == 0) return st;
    a.xq = x_codes; a.xs = x_scales; a.row_src = row_src; a.offsets = offsets; a.codes = codes; a.scales = scales;
    a.y = y; a.y_stride = y_stride;
    a.vec = y_stride % 8 == 0 && aligned(y, 16) ? 3 : y_stride % 4 == 0 && aligned(y, 8) ? 2 : y_stride % 2 == 0 && aligned(y, 4) ? 1 : 0;
    return hip_status(em::launch_mx_product_coded(a, (hipStream_t)stream));
}

size_t edge_moe_balance_ws_bytes(const edge_moe_dims* dims, int32_t n_seq) {
    if (em::layer_dims_status(dims) != EDGE_MOE_OK || n_seq < 1 || n_seq > 4095) return 0;
    em::RouterLoad a{};
    a.T = dims->T; a.E = dims->n_experts; a.k = dims->top_k; a.S = n_seq;
    return em::router_load_ws_bytes(a);
}

int edge_moe_balance(const edge_moe_dims* dims, const float* logits, const int32_t* topk_idx,
                     const int32_t* seq_offsets, int32_t n_seq, int32_t* counts, float* probs, float* loss, void* ws,
                     size_t ws_bytes, void* stream) {
    int st = em::layer_dims_status(dims);
    if (st != EDGE_MOE_OK) return st;
    if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(counts, 4) || !aligned(probs, 4) || !aligned(loss, 4))
        return EDGE_MOE_EINVAL;
    st = seqs_status(seq_offsets, n_seq);
    if (st != EDGE_MOE_OK) return st;
    em::RouterLoad a{};
    a.T = dims->T; a.E = dims->n_experts; a.k = dims->top_k; a.S = n_seq;
    st = ws_status(ws, ws_bytes, em::router_load_ws_bytes(a));
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK) return st;
    a.vec = a.E % 4 == 0 && aligned(logits, 16);
    a.logits = logits; a.topk_idx = topk_idx; a.seq_offsets = seq_offsets;
    a.counts = counts; a.probs = probs; a.loss = loss;
    return hip_status(em::launch_router_load(a, ws, (hipStream_t)stream));
}

size_t edge_moe_route_backward_ws_bytes(const edge_moe_dims* dims) {
    if (em::layer_dims_status(dims) != EDGE_MOE_OK) return 0;
    return em::router_grad_ws_bytes(grad_args(*dims));
}

int edge_moe_route_backward(const edge_moe_dims* dims, const edge_moe_route_grad* g, void* ws, size_t ws_bytes,
                            void* stream) {
    int st = em::layer_dims_status(dims);
    if (st != EDGE_MOE_OK) return st;
    if (!g || !aligned(g->logits, 4)) return EDGE_MOE_EINVAL;
    if (!g->d_topk_w && !g->d_loss) return EDGE_MOE_EINVAL;
    if (g->d_topk_w && (!aligned(g->d_topk_w, 4) || !aligned(g->topk_idx, 4) || !aligned(g->topk_w, 4))) return EDGE_MOE_EINVAL;
    if (g->d_loss) {
        if (!aligned(g->d_loss, 4) || !aligned(g->counts, 4)) return EDGE_MOE_EINVAL;
        st = seqs_status(g->seq_offsets, g->n_seq);
        if (st != EDGE_MOE_OK) return st;
    }
    if (!g->dlogits && !g->dx && !g->dw_router && !g->dbias) return EDGE_MOE_EINVAL;
    if ((g->dlogits && !aligned(g->dlogits, 4)) || (g->dbias && !aligned(g->dbias, 4))) return EDGE_MOE_EINVAL;
    if (g->dx && (!aligned(g->dx, 16) || !aligned(g->w_router, 16))) return EDGE_MOE_EINVAL;
    if (g->dw_router && (!aligned(g->dw_router, 16) || !aligned(g->x, 16))) return EDGE_MOE_EINVAL;
    em::RouterGrad a = grad_args(*dims);
    st = ws_status(ws, ws_bytes, em::router_grad_ws_bytes(a));
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK) return st;
    a.S = g->d_loss ? g->n_seq : 1;
    a.vec = a.E % 4 == 0 && aligned(g->logits, 16) && (!g->dlogits || aligned(g->dlogits, 16));
    a.logits = g->logits; a.topk_idx = g->topk_idx; a.topk_w = g->topk_w; a.d_topk_w = g->d_topk_w;
    a.d_loss = g->d_loss; a.counts = g->counts; a.seq_offsets = g->d_loss ? g->seq_offsets : nullptr;
    a.x = g->x; a.w_router = g->w_router;
    a.dlogits = g->dlogits; a.dx = g->dx; a.dw_router = g->dw_router; a.dbias = g->dbias;
    return hip_status(em::launch_router_grad(a, ws, (hipStream_t)stream));
}

int edge_moe_norm(const edge_moe_norm_args* g, void* stream) {
    if (!g) return EDGE_MOE_EINVAL;
    const int T = g->T, d = g->d;
    int st = norm_shape_status(T, d);
    if (st != EDGE_MOE_OK) return st;
    if (!(g->eps > 0.f) || !(g->eps < 3.4e38f) || !type_ok(g->gain_type) || !aligned(g->gain, 16)) return EDGE_MOE_EINVAL;
    if (!g->x_out && !g->y && !g->codes && !g->scales && !g->rstd && T > 0) return EDGE_MOE_EINVAL;
    if (T > 0 && !rows_ok(g->x, g->x_stride, d, 2)) return EDGE_MOE_EINVAL;
    if (g->add && (!type_ok(g->add_type) || !rows_ok(g->add, g->add_stride, d, type_bytes(g->add_type)))) return EDGE_MOE_EINVAL;
    if ((g->x_out && !rows_ok(g->x_out, g->x_out_stride, d, 2)) || (g->y && !rows_ok(g->y, g->y_stride, d, 2)))
        return EDGE_MOE_EINVAL;
    if (!g->codes != !g->scales || (g->codes && (!aligned(g->codes, 16) || !aligned(g->scales, 4)))) return EDGE_MOE_EINVAL;
    if (g->rstd && !aligned(g->rstd, 4)) return EDGE_MOE_EINVAL;
    if (g->codes && d % 128) return EDGE_MOE_EUNSUPPORTED;
    st = em::device_status();
    if (st != EDGE_MOE_OK || T == 0) return st;
    em::NormFwd a{};
    a.T = T; a.d = d; a.eps = g->eps;
    a.x = g->x; a.x_stride = g->x_stride;
    a.add = g->add; a.add_stride = g->add_stride; a.add_f32 = g->add_type == EDGE_MOE_FLOAT;
    a.gain = g->gain; a.gain_f32 = g->gain_type == EDGE_MOE_FLOAT;
    a.x_out = g->x_out; a.xo_stride = g->x_out_stride; a.y = g->y; a.y_stride = g->y_stride;
    a.codes = g->codes; a.scales = g->scales; a.rstd = g->rstd;
    return hip_status(em::launch_norm_forward(a, (hipStream_t)stream));
}

size_t edge_moe_norm_backward_ws_bytes(int32_t T, int32_t d) {
    return norm_shape_status(T, d) == EDGE_MOE_OK ? em::norm_backward_ws_bytes(T, d) : 0;
}

int edge_moe_norm_backward(const edge_moe_norm_grad* g, void* ws, size_t ws_bytes, void* stream) {
    if (!g) return EDGE_MOE_EINVAL;
    const int T = g->T, d = g->d;
    int st = norm_shape_status(T, d);
    if (st != EDGE_MOE_OK) return st;
    if (!type_ok(g->gain_type) || !type_ok(g->grad_type) || !aligned(g->gain, 16)) return EDGE_MOE_EINVAL;
    const int gb = type_bytes(g->grad_type);
    if (T > 0 && (!aligned(g->rstd, 4) || !rows_ok(g->x, g->x_stride, d, 2) || !rows_ok(g->dy, g->dy_stride, d, gb)))
        return EDGE_MOE_EINVAL;
    if ((g->dres && !rows_ok(g->dres, g->dres_stride, d, gb)) || (g->dx && !rows_ok(g->dx, g->dx_stride, d, gb)))
        return EDGE_MOE_EINVAL;
    if ((!g->dx && !g->dgain && T > 0) || (g->dgain && !aligned(g->dgain, 4))) return EDGE_MOE_EINVAL;
    st = ws_status(ws, ws_bytes, em::norm_backward_ws_bytes(T, d));
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK) return st;
    em::NormBwd a{};
    a.T = T; a.d = d;
    a.x = g->x; a.x_stride = g->x_stride; a.gain = g->gain; a.gain_f32 = g->gain_type == EDGE_MOE_FLOAT; a.rstd = g->rstd;
    a.dy = g->dy; a.dy_stride = g->dy_stride; a.dres = g->dres; a.dres_stride = g->dres_stride;
    a.dx = g->dx; a.dx_stride = g->dx_stride; a.dgain = g->dgain; a.f32 = gb == 4;
    return hip_status(em::launch_norm_backward(a, ws, (hipStream_t)stream));
}

size_t edge_moe_dense_product_ws_bytes(const edge_moe_dense_dims* dims) {
    return dense_status(dims) == EDGE_MOE_OK ? em::dense_product_ws_bytes(dense_args(*dims)) : 0;
}

int edge_moe_dense_product(const edge_moe_dense_dims* dims, const uint16_t* x, int64_t x_stride, const int32_t* row_src,
                           const int32_t* offsets, const uint16_t* w, int32_t y_type, void* y, int64_t y_stride, void* ws,
                           size_t ws_bytes, void* stream) {
    int st = dense_status(dims);
    if (st != EDGE_MOE_OK) return st;
    em::DenseProduct a = dense_args(*dims);
    if (!rows_ok(x, x_stride, a.K, 2) || !aligned(w, 16) || !type_ok(y_type)) return EDGE_MOE_EINVAL;
    if (a.R > 0 && !rows_ok(y, y_stride, a.N, type_bytes(y_type))) return EDGE_MOE_EINVAL;
    st = lists_status(row_src, offsets, a.T, a.R, a.M);
    if (st == EDGE_MOE_OK) st = ws_status(ws, ws_bytes, em::dense_product_ws_bytes(a));
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK || a.R == 0) return st;
    a.x = x; a.x_stride = x_stride; a.row_src = row_src; a.offsets = offsets; a.w = w;
    a.out = y; a.out_stride = y_stride; a.out_f32 = y_type == EDGE_MOE_FLOAT;
    return hip_status(em::launch_dense_product(a, ws, (hipStream_t)stream));
}

size_t edge_moe_dense_product_backward_ws_bytes(const edge_moe_dense_dims* dims) {
    return dense_status(dims) == EDGE_MOE_OK ? em::dense_backward_ws_bytes(dense_args(*dims)) : 0;
}

int edge_moe_dense_product_backward(const edge_moe_dense_dims* dims, const edge_moe_dense_grad* g, void* ws, size_t ws_bytes,
                                    void* stream) {
    int st = dense_status(dims);
    if (st != EDGE_MOE_OK) return st;
    if (!g || (!g->dx && !g->dw)) return EDGE_MOE_EINVAL;
    em::DenseGrad a{};
    a.p = dense_args(*dims);
    em::DenseProduct& p = a.p;
    if (p.R > 0 && !rows_ok(g->dy, g->dy_stride, p.N, 2)) return EDGE_MOE_EINVAL;
    if (g->dw && (!rows_ok(g->x, g->x_stride, p.K, 2) || !type_ok(g->dw_type) || !aligned(g->dw, 16))) return EDGE_MOE_EINVAL;
    if (g->dx && (!aligned(g->w, 16) || !type_ok(g->dx_type) || !rows_ok(g->dx, g->dx_stride, p.K, type_bytes(g->dx_type))))
        return EDGE_MOE_EINVAL;
    if (g->dx && g->token_rows && (!aligned(g->token_rows, 4) || g->per_token < 1)) return EDGE_MOE_EINVAL;
    if (g->dx && g->token_rows && g->per_token > 1024) return EDGE_MOE_EUNSUPPORTED;
    st = lists_status(g->row_src, g->offsets, g->dw ? p.T : p.R, p.R, p.M);
    if (st == EDGE_MOE_OK) st = ws_status(ws, ws_bytes, em::dense_backward_ws_bytes(p));
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK) return st;
    p.x = g->x; p.x_stride = g->x_stride; p.row_src = g->row_src; p.offsets = g->offsets; p.w = g->w;
    p.dy = g->dy; p.dy_stride = g->dy_stride;
    a.dx = g->dx; a.dx_stride = g->dx_stride; a.dx_f32 = g->dx_type == EDGE_MOE_FLOAT;
    a.token_rows = g->dx ? g->token_rows : nullptr; a.per_token = g->per_token;
    a.dw = g->dw; a.dw_f32 = g->dw_type == EDGE_MOE_FLOAT;
    return hip_status(em::launch_dense_backward(a, ws, (hipStream_t)stream));
}

size_t edge_moe_packed_product_ws_bytes(const edge_moe_packed_dims* dims) {
    return int4_status(dims) == EDGE_MOE_OK ? em::int4_product_ws_bytes(int4_args(*dims)) : 0;
}

int edge_moe_packed_product(const edge_moe_packed_dims* dims, const uint16_t* x, int64_t x_stride, const int32_t* row_src,
                          const int32_t* offsets, const uint8_t* codes, const uint16_t* scales, int32_t y_type, void* y,
                          int64_t y_stride, void* ws, size_t ws_bytes, void* stream) {
    int st = int4_status(dims);
    if (st != EDGE_MOE_OK) return st;
    em::Int4Product a = int4_args(*dims);
    if (!rows_ok(x, x_stride, a.K, 2) || !aligned(codes, 16) || !aligned(scales, 4) || !type_ok(y_type)) return EDGE_MOE_EINVAL;
    if (a.R > 0 && (!aligned(y, type_bytes(y_type)) || y_stride < a.N || y_stride > (1ll << 32))) return EDGE_MOE_EINVAL;
    st = lists_status(row_src, offsets, a.T, a.R, a.M);
    if (st == EDGE_MOE_OK) st = ws_status(ws, ws_bytes, em::int4_product_ws_bytes(a));
    if (st == EDGE_MOE_OK) st = em::device_status();
    if (st != EDGE_MOE_OK || a.R == 0) return st;
    a.x = x; a.x_stride = x_stride; a.row_src = row_src; a.offsets = offsets; a.codes = codes; a.scales = scales;
    a.y = y; a.y_stride = y_stride; a.y_f32 = y_type == EDGE_MOE_FLOAT;
    a.vec = aligned(y, 16) && y_stride % (a.y_f32 ? 4 : 8) == 0;
    return hip_status(em::launch_int4_product(a, ws, (hipStream_t)stream));
}

}  // extern "C"
