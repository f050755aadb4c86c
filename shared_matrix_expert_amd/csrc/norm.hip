// Root-mean-square norm between layers, forward and backward.
//
//   forward   r = bf16(x + add);  rstd = 1 / sqrt(mean r^2 + eps)
//             y = bf16(r rstd gain);  codes, scales = MXFP8 of y (mx_quant.hip's rule)
//   backward  v = r rstd, dv = dy gain:  dr = rstd (dv - v mean(dv v))
//             dx = dres + dr,  dgain = sum_t dy v
//
// Each row is read once, kept in registers over the reduction and written once, so
// both directions are bound by HBM (measured: a large copy passes 5.1 TB/s).  W waves
// share a row, each lane NV runs of eight neighbours; an MX block is then four
// neighbouring lanes.  The squares are summed in float64: no bf16 row overflows there,
// and the sum's order does not show.
//
// Forward: a workgroup a row, or four rows of 1024 and less.  16384 rows of 4096, float32
// added, codes out, 606 MB: 103 us, 5.9 TB/s; runs of rows a workgroup, the next row asked
// for ahead, 116 us (4096 workgroups) and 126 us (2048).  bf16 added, bf16 out, 537 MB: 80,
// 82 and 110 us.
//
// Backward: a workgroup takes a run of neighbouring rows and asks for the next one before it
// reduces the present one; the gain and its gradient stay in registers, so that dgain passes
// through memory once a workgroup.  dgain is summed in float64, exact products included: its
// error does not grow with the rows, and no time shows (a float32 sum lost up to half a unit a
// row).  16384 rows of 4096, bf16, 537 MB: 109 us with dgain's launch, 5 us of it; 1024
// workgroups 122, 256 117.
#include <type_traits>

#include "mx_format.h"
#include "operators.h"

namespace em {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

EM_DEV uint4 ldv(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// Eight neighbouring elements as loaded: bf16 in one word, float32 in two.
template <bool F32> struct Raw8 { uint4 v[F32 ? 2 : 1]; };

template <bool F32>
EM_DEV void load8(Raw8<F32>& o, const void* row, int e) {
    if constexpr (F32) {
        const float* p = static_cast<const float*>(row) + e;
        o.v[0] = ldv(p);
        o.v[1] = ldv(p + 4);
    } else {
        o.v[0] = ldv(static_cast<const uint16_t*>(row) + e);
    }
}

template <bool F32>
EM_DEV void widen8(const Raw8<F32>& r, float (&f)[8]) {
    if constexpr (F32) {
        f[0] = __uint_as_float(r.v[0].x); f[1] = __uint_as_float(r.v[0].y);
        f[2] = __uint_as_float(r.v[0].z); f[3] = __uint_as_float(r.v[0].w);
        f[4] = __uint_as_float(r.v[1].x); f[5] = __uint_as_float(r.v[1].y);
        f[6] = __uint_as_float(r.v[1].z); f[7] = __uint_as_float(r.v[1].w);
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// Eight elements of a gain of either type.
EM_DEV void load_gain(float (&f)[8], const void* gain, int f32, int e) {
    if (f32) {
        Raw8<true> r;
        load8(r, gain, e);
        widen8(r, f);
    } else {
        Raw8<false> r;
        load8(r, gain, e);
        widen8(r, f);
    }
}

EM_DEV uint32_t pack2(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
EM_DEV uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// x + a on its way to bf16: the float32 sum, moved one unit towards the exact one
// where it lies on the middle of two bf16 values, so that rounding it gives the
// exact sum's bf16 (edge_moe_residual's).
EM_DEV float sum_for_bf16(float x, float a) {
    const float s = x + a;
    const float xs = s - a, as = s - xs;
    const float lost = (x - xs) + (a - as);                 // s + lost = x + a exactly
    int32_t b = __float_as_int(s);
    if ((b & 0xFFFF) == 0x8000 && lost != 0.f) b += (lost > 0.f) == (s > 0.f) ? 1 : -1;
    return __int_as_float(b);
}

template <int CTRL, int ROWS>
EM_DEV double dpp_add_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over the wave's lanes, the same in every lane (a fixed order).
EM_DEV double wave_sum_f64(double v) {
    v = dpp_add_f64<0x111, 0xF>(v);       // row_shr:1, 2, 4, 8, then row_bcast:15 and :31
    v = dpp_add_f64<0x112, 0xF>(v);
    v = dpp_add_f64<0x114, 0xF>(v);
    v = dpp_add_f64<0x118, 0xF>(v);
    v = dpp_add_f64<0x142, 0xA>(v);
    v = dpp_add_f64<0x143, 0xC>(v);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the row's W waves; `turn` alternates, so that one barrier a row is enough.
template <int W, int N>
EM_DEV double row_sum(double v, double (&slots)[N][W], int turn) {
    v = wave_sum_f64(v);
    if constexpr (W == 1) return v;
    const int wv = wave_id();
    if (lane_id() == 0) slots[turn][wv] = v;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) s += slots[turn][i];
    return s;
}

// 1 / sqrt(m) in float64: the hardware's estimate and two steps towards the root (of an
// infinity, zero, as it is: a step would multiply the two).
EM_DEV double rsqrt_f64(double m) {
    const double e = __builtin_amdgcn_rsq(m);
    double r = e * fma(-0.5 * m * e, e, 1.5);
    r = r * fma(-0.5 * m * r, r, 1.5);
    return m == __builtin_inf() ? 0.0 : r;
}

// Stored past the caches, where the rows read next would take their place.
EM_DEV void past_caches(void* to, const uint4& v) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, static_cast<u32x4*>(to));
}
EM_DEV void past_caches(void* to, const uint2& v) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(u32x2{v.x, v.y}, static_cast<u32x2*>(to));
}

// Rows of a workgroup: W > 1 one at a time, W = 1 one a wave.
template <int W> constexpr int rows_at_once() { return W == 1 ? 4 : 1; }
template <int W> constexpr int norm_threads() { return W == 1 ? 256 : 64 * W; }

}  // namespace

// ADD: nothing, bf16 or float32 to add (0, 1, 2).
template <int W, int NV, int ADD>
__global__ void __launch_bounds__(norm_threads<W>())
norm_forward(NormFwd a) {
    __shared__ double slots[1][W];
    const int in_row = W == 1 ? lane_id() : (int)threadIdx.x;
    const int t = a.t0 + (W == 1 ? 4 * (int)blockIdx.x + wave_id() : (int)blockIdx.x);
    if (t >= a.T) return;                                      // W = 1 only: a wave without a row (no barrier there)
    bool live[NV];
    int at[NV];                                                // lanes past the row read its first elements again
    float gain[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 8 * (in_row + 64 * W * i);
        live[i] = e < a.d;
        at[i] = live[i] ? e : 0;
        load_gain(gain[i], a.gain, a.gain_f32, at[i]);
    }
    Raw8<false> xr[NV];
    Raw8<ADD == 2> ar[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load8(xr[i], a.x + t * a.x_stride, at[i]);
        if constexpr (ADD == 2) load8(ar[i], static_cast<const float*>(a.add) + t * a.add_stride, at[i]);
        if constexpr (ADD == 1) load8(ar[i], static_cast<const uint16_t*>(a.add) + t * a.add_stride, at[i]);
    }
    uint4 r[NV];                                           // the row in bf16
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[8];
        widen8(xr[i], f);
        if constexpr (ADD != 0) {
            float g[8];
            widen8(ar[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = sum_for_bf16(f[j], g[j]);
            r[i] = pack8(f);
            Raw8<false> back;
            back.v[0] = r[i];
            widen8(back, f);
        } else {
            r[i] = xr[i].v[0];
        }
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fma((double)f[j], (double)f[j], s);
        sum += live[i] ? s : 0.0;
    }
    sum = row_sum<W>(sum, slots, 0);
    const float rstd = (float)rsqrt_f64(sum * a.per_d + (double)a.eps);
    if (a.rstd && in_row == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (a.x_out && live[i]) past_caches(a.x_out + t * a.xo_stride + at[i], r[i]);
        if (!a.y && !a.codes) continue;
        float f[8];
        Raw8<false> rr;
        rr.v[0] = r[i];
        widen8(rr, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * gain[i][j];
        const uint4 y = pack8(f);
        if (a.y && live[i]) past_caches(a.y + t * a.y_stride + at[i], y);
        if (a.codes) {                                     // d a multiple of 128: a block's four lanes are live together
            uint32_t m = amax8_bf16(y);
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0xB1, 0xF, 0xF, false));
            m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x4E, 0xF, 0xF, false));
            const int X = e8m0_of<kMxFp8>(m);
            const bool bad = X == 255;
            const float sc = e8m0_f32(bad ? 127 : X);
            const uint32_t lim = e4m3_limit(bad ? 127 : X);
            const uint32_t q0 = fp8x4_bf16(y.x, y.y, sc, lim), q1 = fp8x4_bf16(y.z, y.w, sc, lim);
            if (live[i]) {
                past_caches(a.codes + (int64_t)t * a.d + at[i], bad ? make_uint2(0u, 0u) : make_uint2(q0, q1));
                if (!(lane_id() & 3)) a.scales[((int64_t)(at[i] >> 7) * a.T + t) * 4 + (at[i] >> 5 & 3)] = (uint8_t)X;
            }
        }
    }
}

// Rows of sixteen waves (more than 8192) leave a lane 128 registers: dgain's sums are then made
// in a pass of their own (norm_gain_sums), and rows of more than 16384 are not asked for ahead.
// 4096 rows of 16384, bf16 130 us (the sums beside the rows 311), float32 261 (595); 2048 of
// 32768 248 (771) and 395 (1049).
template <int W> constexpr bool sums_beside_rows() { return W < 16; }

// F32: dy, dres and dx are float32 (else bf16).
template <int W, int NV, bool F32>
__global__ void __launch_bounds__(norm_threads<W>())
norm_backward(NormBwd a) {
    __shared__ double slots[2][W];
    constexpr bool SUMS = sums_beside_rows<W>(), AHEAD = NV < 4;
    __shared__ __attribute__((aligned(16))) double part[W == 1 ? 4 : 1][W == 1 ? 512 * NV : 2];
    const int in_row = W == 1 ? lane_id() : (int)threadIdx.x;
    const int first = blockIdx.x * a.chunk + (W == 1 ? wave_id() : 0);
    const int last = min(a.T, (int)(blockIdx.x + 1) * a.chunk);
    constexpr int STEP = rows_at_once<W>();
    using G = Raw8<F32>;
    bool live[NV];
    int at[NV];
    float gain[NV][8];
    double dg[SUMS ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = 8 * (in_row + 64 * W * i);
        live[i] = e < a.d;
        at[i] = live[i] ? e : 0;
        load_gain(gain[i], a.gain, a.gain_f32, at[i]);
#pragma unroll
        for (int j = 0; SUMS && j < 8; ++j) dg[i][j] = 0.0;
    }
    constexpr int64_t ES = F32 ? 4 : 2;
    Raw8<false> xr[NV];
    G yr[NV], rr[NV];
    float rs = 0.f;
    auto fetch = [&](int t) {
        rs = a.rstd[t];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load8(xr[i], a.x + t * a.x_stride, at[i]);
            load8(yr[i], static_cast<const char*>(a.dy) + t * a.dy_stride * ES, at[i]);
            if (a.dres) load8(rr[i], static_cast<const char*>(a.dres) + t * a.dres_stride * ES, at[i]);
        }
    };
    if (AHEAD && first < last) fetch(first);
    int turn = 0;
    for (int t = first; t < last; t += STEP) {
        if (!AHEAD) fetch(t);
        const float rstd = rs;
        float v[NV][8], dv[NV][8], res[NV][8];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            widen8(xr[i], v[i]);
            widen8(yr[i], dv[i]);
            if (a.dres) widen8(rr[i], res[i]);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= rstd;
                if constexpr (SUMS) dg[i][j] = fma((double)dv[i][j], (double)v[i][j], dg[i][j]);
                dv[i][j] *= gain[i][j];
                s = fmaf(dv[i][j], v[i][j], s);
            }
            sum += live[i] ? s : 0.f;
        }
        if (AHEAD && t + STEP < last) fetch(t + STEP);
        if (a.dx) {
            const float mean = (float)(row_sum<W>((double)sum, slots, turn) * a.per_d);
            turn ^= 1;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dr = rstd * fmaf(-v[i][j], mean, dv[i][j]);
                    dv[i][j] = a.dres ? res[i][j] + dr : dr;
                }
                if (!live[i]) continue;
                char* o = static_cast<char*>(a.dx) + (t * a.dx_stride + at[i]) * ES;
                if constexpr (F32) {
                    *reinterpret_cast<float4*>(o) = make_float4(dv[i][0], dv[i][1], dv[i][2], dv[i][3]);
                    *reinterpret_cast<float4*>(o + 16) = make_float4(dv[i][4], dv[i][5], dv[i][6], dv[i][7]);
                } else {
                    past_caches(o, pack8(dv[i]));         // (pairs of float4 half a line apart: 16384 x 512 22.6 us, past the caches 24.6)
                }
            }
        }
    }
    if (!SUMS || !a.part) return;
    float* out = a.part + (int64_t)blockIdx.x * a.d;
    if constexpr (W == 1) {                                    // the four waves' rows, added in wave order
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) part[wave_id()][8 * (in_row + 64 * i) + j] = dg[i][j];
        __syncthreads();
        for (int e = threadIdx.x; e < a.d; e += 256) out[e] = (float)((part[0][e] + part[1][e]) + (part[2][e] + part[3][e]));
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!live[i]) continue;
            *reinterpret_cast<float4*>(out + at[i]) = make_float4((float)dg[i][0], (float)dg[i][1], (float)dg[i][2], (float)dg[i][3]);
            *reinterpret_cast<float4*>(out + at[i] + 4) = make_float4((float)dg[i][4], (float)dg[i][5], (float)dg[i][6], (float)dg[i][7]);
        }
    }
}

// Sums of dgain's terms over a run of rows, where they have no place beside the rows: a
// workgroup takes 512 columns, its sixteen waves four rows each at once, added in wave order.
// The only run's sums are dgain.
template <bool F32>
__global__ void __launch_bounds__(1024)
norm_gain_sums(NormBwd a, int run) {
    __shared__ double sp[16][512];
    constexpr int64_t ES = F32 ? 4 : 2;
    constexpr int ROWS = 4;
    const int wv = wave_id(), col = 8 * lane_id(), e = min(512 * (int)blockIdx.x + col, a.d - 8);
    const int first = blockIdx.y * run, last = min(a.T, first + run);
    double dg[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = 0.0;
    for (int t = first + ROWS * wv; t < last; t += 16 * ROWS) {
        Raw8<false> x[ROWS];
        Raw8<F32> dy[ROWS];
        float rstd[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int at = min(t + i, last - 1);
            rstd[i] = a.rstd[at];
            load8(x[i], a.x + at * a.x_stride, e);
            load8(dy[i], static_cast<const char*>(a.dy) + at * a.dy_stride * ES, e);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (t + i >= last) break;
            float v[8], g[8];
            widen8(x[i], v);
            widen8(dy[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) dg[j] = fma((double)g[j], (double)(v[j] * rstd[i]), dg[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sp[wv][col + j] = dg[j];
    __syncthreads();
    const int out = 512 * blockIdx.x + threadIdx.x;
    if (threadIdx.x >= 512 || out >= a.d) return;
    double s = sp[0][threadIdx.x];
    for (int r = 1; r < 16; ++r) s += sp[r][threadIdx.x];
    if (gridDim.y == 1) a.dgain[out] = (float)s;
    else a.part[(int64_t)blockIdx.y * a.d + out] = (float)s;
}

// dgain from the workgroups' partial sums: 16 rows of 64 threads over interleaved
// workgroups in float64, then the rows in order.
__global__ void __launch_bounds__(1024)
norm_dgain(const float* __restrict__ part, int blocks, int d, float* __restrict__ dgain) {
    __shared__ double sp[16][64];
    const int col = threadIdx.x & 63, row = threadIdx.x >> 6, e = blockIdx.x * 64 + col;
    double s = 0.0;
    if (e < d) {
#pragma unroll 8
        for (int b = row; b < blocks; b += 16) s += (double)part[(int64_t)b * d + e];
    }
    sp[row][col] = s;
    __syncthreads();
    if (row || e >= d) return;
    for (int r = 1; r < 16; ++r) s += sp[r][col];
    dgain[e] = (float)s;
}

// ------------------------------------------------------------------ host side ----
namespace {

struct NormPlan { int w, nv, chunk, blocks; };

constexpr int kBwdBlocks = 512, kSumBlocks = 512;

// Waves a row, runs of 512 elements a wave; backward, rows a workgroup and workgroups: at most
// kBwdBlocks, or half as many of more than four waves.  4096 rows of 8192: 256 of eight waves
// 45.9 us, 512 52; dx of 4096 rows of 16384, float32, 256 of sixteen waves 189 us, 512 196,
// 4096 212.
NormPlan norm_plan(int T, int d) {
    NormPlan p{};
    const int runs = (d + 511) / 512;
    p.nv = runs <= 1 ? 1 : runs <= 32 ? 2 : 4;
    p.w = 1;
    while (p.w * p.nv < runs) p.w *= 2;
    const int at_once = p.w == 1 ? 4 : 1;
    const int groups = (T + at_once - 1) / at_once;
    if (!T) return p;
    const int most = p.w > 4 ? kBwdBlocks / 2 : kBwdBlocks;
    p.chunk = (groups + most - 1) / most * at_once;
    p.blocks = (T + p.chunk - 1) / p.chunk;
    return p;
}

// Rows of dgain's partial sums: a workgroup of norm_backward each, or a run of `run` rows
// each (norm_gain_sums, two workgroups a compute unit; 256 rows and fewer in one run spare
// norm_dgain's launch).
struct GainPlan { int run, parts; };
GainPlan gain_plan(const NormPlan& p, int T, int d) {
    if (p.w < 16 || !T) return GainPlan{0, p.blocks};
    const int most = kSumBlocks / ((d + 511) / 512), even = ((T + most - 1) / most + 3) / 4 * 4;
    const int run = even < 256 ? 256 : even;
    return GainPlan{run, (T + run - 1) / run};
}

// A launch holds fewer than 2^32 threads: rows of more than 2^31 of them take several.
template <int W, int NV>
void launch_fwd(NormFwd a, hipStream_t s) {
    constexpr int kRows = (int)((1ll << 31) / norm_threads<W>()) * rows_at_once<W>();
    for (a.t0 = 0; a.t0 < a.T; a.t0 += kRows) {
        const int rows = a.T - a.t0 < kRows ? a.T - a.t0 : kRows, blocks = (rows + rows_at_once<W>() - 1) / rows_at_once<W>();
        if (!a.add) norm_forward<W, NV, 0><<<blocks, norm_threads<W>(), 0, s>>>(a);
        else if (!a.add_f32) norm_forward<W, NV, 1><<<blocks, norm_threads<W>(), 0, s>>>(a);
        else norm_forward<W, NV, 2><<<blocks, norm_threads<W>(), 0, s>>>(a);
    }
}

template <int W, int NV>
void launch_bwd(const NormBwd& a, const NormPlan& p, hipStream_t s) {
    if (a.f32) norm_backward<W, NV, true><<<p.blocks, norm_threads<W>(), 0, s>>>(a);
    else norm_backward<W, NV, false><<<p.blocks, norm_threads<W>(), 0, s>>>(a);
}

template <class F>
void by_plan(const NormPlan& p, F launch) {
    using std::integral_constant;
    const integral_constant<int, 2> two{};
    if (p.nv == 1) launch(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (p.nv == 4) launch(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (p.w == 1) launch(integral_constant<int, 1>{}, two);
    else if (p.w == 2) launch(two, two);
    else if (p.w == 4) launch(integral_constant<int, 4>{}, two);
    else if (p.w == 8) launch(integral_constant<int, 8>{}, two);
    else launch(integral_constant<int, 16>{}, two);
}

}  // namespace

hipError_t launch_norm_forward(NormFwd a, hipStream_t s) {
    const NormPlan p = norm_plan(a.T, a.d);
    a.per_d = 1.0 / a.d;
    prof_begin(s);
    by_plan(p, [&](auto w, auto nv) { launch_fwd<decltype(w)::value, decltype(nv)::value>(a, s); });
    prof_end(s, "norm_forward");
    return hipGetLastError();
}

size_t norm_backward_ws_bytes(int T, int d) {
    const size_t n = (size_t)gain_plan(norm_plan(T, d), T, d).parts * d * 4;
    return n > 256 ? n : 256;
}

hipError_t launch_norm_backward(NormBwd a, void* ws, hipStream_t s) {
    const NormPlan p = norm_plan(a.T, a.d);
    const GainPlan sums = gain_plan(p, a.T, a.d);
    a.chunk = p.chunk;
    a.per_d = 1.0 / a.d;
    a.part = a.dgain ? static_cast<float*>(ws) : nullptr;
    if (sums.run && a.dgain) {                                    // first: dx may lie on dy
        const dim3 grid((a.d + 511) / 512, sums.parts);
        prof_begin(s);
        if (a.f32) norm_gain_sums<true><<<grid, 1024, 0, s>>>(a, sums.run);
        else norm_gain_sums<false><<<grid, 1024, 0, s>>>(a, sums.run);
        prof_end(s, "norm_gain_sums");
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (p.blocks && (a.dx || !sums.run)) {
        prof_begin(s);
        by_plan(p, [&](auto w, auto nv) { launch_bwd<decltype(w)::value, decltype(nv)::value>(a, p, s); });
        prof_end(s, "norm_backward");
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.dgain || (sums.run && sums.parts == 1)) return hipSuccess;
    prof_begin(s);
    norm_dgain<<<(a.d + 63) / 64, 1024, 0, s>>>(a.part, sums.parts, a.d, a.dgain);
    prof_end(s, "norm_dgain");
    return hipGetLastError();
}

}  // namespace em
