// Product of token rows with int4 matrices in the layer's storage:
//   y[r][n] = sum over groups q of K of s_m[n][q] sum_{k in q} x[src(r)][k] c_m[n][k]
// with c the signed codes and s the fp16 scales of Gq elements each.  Codes become bf16
// exactly (dequant8), x is bf16, a group's products are summed in float32 on the matrix
// cores and the sum is scaled by a float32 fused multiply-add: every weight is exactly
// c s, as in the layer.
//
//   ip_stream  four waves split K and stream the codes straight into operand registers.
#include <type_traits>

#include "common.h"
#include "mfma_ops.h"
#include "operators.h"
#include "row_tile.h"

namespace em {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// x row of y row r, -1 where row_src names none.
EM_DEV int x_row(const Int4Product& a, int r) {
    if (!a.row_src) return r;
    const int s = a.row_src[r];
    return (unsigned)s < (unsigned)a.T ? s : -1;
}

EM_DEV void store1(void* out, int f32, int64_t at, float v) {
    if (f32) {
        static_cast<float*>(out)[at] = v;
    } else {
        const f32x2 p = {v, v};
        static_cast<uint16_t*>(out)[at] = (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
    }
}

// A lane's 16 bytes are 32 neighbouring codes (lane group g those of 32 g): word i of the
// lane groups exchanged so that word s holds codes 32 s + 8 g .. + 7, one scale group an
// instruction.
EM_DEV uint4 by_group(uint4 v) {
    auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
    auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return make_uint4(c[0], c[1], d[0], d[1]);
}

}  // namespace

// GPC: scale groups in 128 elements of K (1: groups of 128 and more).  A workgroup takes
// one row tile (16 NS rows of one matrix) and 16 NC columns.  The last 32, 64 or 96
// elements of a K that is no multiple of 128 are a chunk whose missing codes are zero.
template <int GPC, int NS, int NC>
__global__ void __launch_bounds__(256)
ip_stream(Int4Product a) {
    constexpr int WD = NS == 4 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) float red[4][NS * NC][256];
    const RowTile t = row_tile<16 * NS>(a.offsets, a.M, a.R, [](int) { return (int)blockIdx.y; });
    if (t.r1 == 0) return;
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
    const int n0 = blockIdx.x * (16 * NC);
    const int chunks = (a.K + KC - 1) / KC;
    const int s0 = chunks * wv / 4, s1 = chunks * (wv + 1) / 4;
    const int ng = a.K / a.gq;

    const uint8_t* wp[NC];
    const uint16_t* sp[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t row = (int64_t)t.m * a.N + min(n0 + 16 * c + m, a.N - 1);
        wp[c] = a.codes + row * (a.K / 2);
        sp[c] = a.scales + row * ng;
    }
    uint4 w[WD][NC];
    uint16_t sc[WD][NC][GPC];
    auto load_w = [&](int d, int ch) {
        const int k = KC * ch + 32 * g;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            w[d][c] = ld16(wp[c] + min(k, a.K - 32) / 2);
#pragma unroll
            for (int q = 0; q < GPC; ++q) sc[d][c][q] = sp[c][min((KC * ch + KC / GPC * q) / a.gq, ng - 1)];
        }
    };
    if (s0 < s1) {
#pragma unroll
        for (int d = 0; d < WD; ++d) load_w(d, min(s0 + d, s1 - 1));
    }
    bool live[NS];
    const uint16_t* xp[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const int r = t.r0 + 16 * s + m, src = x_row(a, min(r, t.r1 - 1));
        live[s] = src >= 0;
        xp[s] = a.x + (int64_t)max(src, 0) * a.x_stride;
    }
    floatx4 acc[NS][NC];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[s][c] = zero4();
    for (int ch = s0; ch < s1; ch += WD) {
#pragma unroll
        for (int d = 0; d < WD; ++d) {
            if (ch + d < s1) {
                const int k0 = KC * (ch + d), left = a.K - k0;
                uint4 x[NS][4];
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = GPC == 1 ? 32 * g + 8 * i : 32 * i + 8 * g;
                        const uint4 v = ld16(xp[s] + k0 + (at < left ? at : 0));
                        x[s][i] = at < left && live[s] ? v : zero_u4();
                    }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    uint4 raw = 32 * g < left ? w[d][c] : zero_u4();
                    if constexpr (GPC > 1) raw = by_group(raw);
                    uint4 b[4];
                    dequant_b(raw, b);
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int q = 0; q < GPC; ++q) {
                            floatx4 u = zero4();
#pragma unroll
                            for (int i = 4 / GPC * q; i < 4 / GPC * (q + 1); ++i) u = mfma_bf16(x[s][i], b[i], u);
                            acc[s][c] = fma4(16.0f * fp16_bits_to_f32(sc[d][c][q]), u, acc[s][c]);
                        }
                }
                load_w(d, min(ch + d + WD, s1 - 1));
            }
        }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c) *reinterpret_cast<floatx4*>(&red[wv][s * NC + c][4 * lane]) = acc[s][c];
    __syncthreads();
    // tile i = (subtile s, column tile c) is summed by wave i % 4; lane (g, m) holds rows
    // 4 g .. 4 g + 3 of column m
#pragma unroll
    for (int i = 0; i < NS * NC; ++i) {
        if ((i & 3) != wv) continue;
        floatx4 v = *reinterpret_cast<const floatx4*>(&red[0][i][4 * lane]);
#pragma unroll
        for (int q = 1; q < 4; ++q) v += *reinterpret_cast<const floatx4*>(&red[q][i][4 * lane]);
        const int n = n0 + 16 * (i % NC) + m, r = t.r0 + 16 * (i / NC) + 4 * g;
        if (n >= a.N) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r + j < t.r1) store1(a.y, a.y_f32, (int64_t)(r + j) * a.y_stride + n, v[j]);
    }
}

// ------------------------------------------------------------------ host side ----
namespace {

int64_t max_row_tiles(const Int4Product& a, int BT) {
    const int live = a.M < a.R ? a.M : a.R;
    return a.M > 1 ? a.R / BT + live : (a.R + BT - 1) / BT;
}

template <int GPC, int NS>
hipError_t launch_stream(const Int4Product& a, hipStream_t s) {
    const int64_t tiles = max_row_tiles(a, 16 * NS);
    prof_begin(s);
    if (tiles * ((a.N + 31) / 32) <= 128) ip_stream<GPC, NS, 1><<<dim3((a.N + 15) / 16, (unsigned)tiles), 256, 0, s>>>(a);
    else ip_stream<GPC, NS, 2><<<dim3((a.N + 31) / 32, (unsigned)tiles), 256, 0, s>>>(a);
    prof_end(s, "ip_stream");
    return hipGetLastError();
}

// How many times 16 rows of a matrix ip_stream takes at once.
int stream_rows(const Int4Product& a) {
    const int live = a.M < a.R ? a.M : a.R;
    const int64_t avg = ((int64_t)a.R + live - 1) / live, cols = (a.N + 31) / 32;
    for (int ns = 1; ns < 4; ns *= 2)
        if (max_row_tiles(a, 16 * ns) * cols <= 256 || avg <= 16 * ns) return ns;
    return 4;
}

template <int GPC>
hipError_t launch_product(const Int4Product& a, hipStream_t s) {
    switch (stream_rows(a)) {
        case 1: return launch_stream<GPC, 1>(a, s);
        case 2: return launch_stream<GPC, 2>(a, s);
        default: return launch_stream<GPC, 4>(a, s);
    }
}

}  // namespace

size_t int4_product_ws_bytes(const Int4Product&) { return 256; }

hipError_t launch_int4_product(Int4Product a, void* ws, hipStream_t s) {
    (void)ws;
    if (a.gq >= KC || a.gq == a.K) return launch_product<1>(a, s);    // (a narrower group is the whole of a K below 128)
    return a.gq == 64 ? launch_product<2>(a, s) : launch_product<4>(a, s);
}

}  // namespace em
