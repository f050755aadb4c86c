// C-ABI entry points of the MX-matrix and router-training operators: validation
// and launches.
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

}  // extern "C"
