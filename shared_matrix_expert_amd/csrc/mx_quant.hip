// MX quantiser: dense rows (bf16 or float32) to microscaling codes and E8M0
// scales, and back.  Layouts are the MX layer's: codes row-major (E2M1 two per
// byte, element 2i in the low nibble; E4M3 one per byte), scales K-step-major
// [K/128][N][4] for each matrix of N rows.
//
// Both directions read each input once and write each output once with a
// handful of conversions per element, so they are bound by HBM.  Sixteen lanes
// take one 128-element step of a row.  bf16: 8 elements in a row each, a scale
// block four neighbouring lanes, its maximum two quad permutes.  float32: 4
// elements in each half of the step, a block eight lanes; every access of the
// sixteen lanes is then 256 bytes in a row (with 8 neighbours each, two accesses
// of half the bytes of every line, 65536 x 4096 back from FP4 took 526 us, 203
// here).  A workgroup takes 16 rows x 4 steps: the four steps' loads are in flight
// together, and the scale words of its 16 rows fall in one 64-byte run per step.
// The dense side is read and written past the caches: 8 matrices of 8192 x 4096
// (537 MB dense, 143 packed) there and back 321 -> 288 us (4.7 TB/s), 16384 rows of
// 4096 in FP8 92 -> 72 us (39 there, 5.2 TB/s).  Eight steps a workgroup measured
// no faster.
#include "mx_format.h"
#include "operators.h"

namespace em {

namespace {

constexpr int QR = 16;    // rows per workgroup
constexpr int QS = 4;     // K steps per workgroup

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The dense side passes once, so its accesses leave the caches to the codes.
EM_DEV uint4 ld16_once(const uint4* p) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

// Value of the lane's quad neighbours under an xor of 1 (0xB1) or 2 (0x4E).
template <int CTRL>
EM_DEV uint32_t quad(uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false); }

EM_DEV uint32_t quad_max(uint32_t v) {
    v = max(v, quad<0xB1>(v));
    return max(v, quad<0x4E>(v));
}
EM_DEV uint32_t oct_max(uint32_t v) {
    v = quad_max(v);
    return max(v, quad<0x141>(v));                              // row_half_mirror: the other quad of the eight lanes
}

// A lane's first float32 element in half h of a 128-element step: four neighbours
// each, so that an access of the sixteen lanes is 256 bytes in a row.
EM_DEV int f32_at(int l16, int h) { return 64 * h + 4 * l16; }

}  // namespace

// GATHER: row r of the result is src row row_src[r] (row 0 for one outside
// 0..src_rows - 1).
template <int FMT, bool F32, bool GATHER>
__global__ void __launch_bounds__(256)
mxq_quantize(const void* __restrict__ src, int64_t stride, int64_t rows, int N, int K, uint8_t* __restrict__ codes,
             uint8_t* __restrict__ scales, const int32_t* __restrict__ row_src, int src_rows) {
    const int l16 = threadIdx.x & 15;
    const int64_t row = (int64_t)blockIdx.x * QR + (threadIdx.x >> 4);
    if (row >= rows) return;
    const int steps = K / kMxStep, s0 = blockIdx.y * QS;
    const int64_t m = row / N, n = row - m * N;
    uint8_t* srow = scales + (m * steps * N + n) * 4;          // + step * N * 4 + block
    int64_t from = row;
    if constexpr (GATHER) {
        const int r = row_src[row];
        from = (unsigned)r < (unsigned)src_rows ? r : 0;
    }
    uint4 v[QS][F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        const int64_t k = (int64_t)min(s0 + i, steps - 1) * kMxStep;
        if constexpr (F32) {
            const float* p = static_cast<const float*>(src) + from * stride + k;
            v[i][0] = ld16_once(reinterpret_cast<const uint4*>(p + f32_at(l16, 0)));
            v[i][1] = ld16_once(reinterpret_cast<const uint4*>(p + f32_at(l16, 1)));
        } else {
            v[i][0] = ld16_once(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + from * stride + k + 8 * l16));
        }
    }
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        if (s0 + i >= steps) break;
        uint8_t* sc_out = srow + (int64_t)(s0 + i) * N * 4;
        const int64_t at = row * K + (int64_t)(s0 + i) * kMxStep;
        if constexpr (F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
                float f[4];
                uint32_t a = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a = max(a, w[j] & 0x7FFFFFFFu);
                    f[j] = __uint_as_float(w[j]);
                }
                const int X = e8m0_of<FMT>(oct_max(a) >> 16);
                const bool bad = X == 255;
                const float sc = e8m0_f32(bad ? 127 : X);
                const int64_t c = at + f32_at(l16, h);
                if constexpr (FMT == kMxFp4) *reinterpret_cast<uint16_t*>(codes + (c >> 1)) = bad ? 0 : fp4x4_f32(f, sc);
                else *reinterpret_cast<uint32_t*>(codes + c) = bad ? 0u : fp8x4_f32(f, sc);
                if ((l16 & 7) == 0) sc_out[2 * h + (l16 >> 3)] = (uint8_t)X;
            }
        } else {
            const int X = e8m0_of<FMT>(quad_max(amax8_bf16(v[i][0])));
            const bool bad = X == 255;
            const float sc = e8m0_f32(bad ? 127 : X);
            const int64_t c = at + 8 * l16;
            if constexpr (FMT == kMxFp4) {
                const uint32_t q = fp4x8_bf16(v[i][0], sc);
                *reinterpret_cast<uint32_t*>(codes + (c >> 1)) = bad ? 0u : q;
            } else {
                const uint32_t lim = e4m3_limit(bad ? 127 : X);
                const uint32_t q0 = fp8x4_bf16(v[i][0].x, v[i][0].y, sc, lim), q1 = fp8x4_bf16(v[i][0].z, v[i][0].w, sc, lim);
                *reinterpret_cast<uint2*>(codes + c) = bad ? make_uint2(0u, 0u) : make_uint2(q0, q1);
            }
            if ((l16 & 3) == 0) sc_out[l16 >> 2] = (uint8_t)X;
        }
    }
}

// Codes 2 I and 2 I + 1 of a word as floats, and a block's scale (X = 255: NaN).
template <int FMT, int I>
EM_DEV f32x2 mx_pair(uint32_t q) {
    if constexpr (FMT == kMxFp4) return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, I);
    else return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, 1.0f, I == 1);
}
EM_DEV float mx_scale(int X) { return X == 255 ? __uint_as_float(0x7FC00000u) : e8m0_f32(X); }

// Back: value(code) * 2^(X - 127), exact in float32, then rounded once to the
// dense type (a code has at most four significant bits, so bf16 rounds only
// below its smallest subnormal; past the type's range an infinity).  X = 255
// and the E4M3 NaN code give NaN.
template <int FMT, bool F32>
__global__ void __launch_bounds__(256)
mxq_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t stride, int64_t rows, int N,
               int K, void* __restrict__ dst) {
    const int l16 = threadIdx.x & 15;
    const int64_t row = (int64_t)blockIdx.x * QR + (threadIdx.x >> 4);
    if (row >= rows) return;
    const int steps = K / kMxStep, s0 = blockIdx.y * QS;
    const int64_t m = row / N, n = row - m * N;
    const uint8_t* srow = scales + (m * steps * N + n) * 4;
    if constexpr (F32) {                                        // four codes in each half of a step
        uint32_t q[QS][2];
        int X[QS][2];
#pragma unroll
        for (int i = 0; i < QS; ++i) {
            const int st = min(s0 + i, steps - 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t c = row * K + (int64_t)st * kMxStep + f32_at(l16, h);
                if constexpr (FMT == kMxFp4) q[i][h] = *reinterpret_cast<const uint16_t*>(codes + (c >> 1));
                else q[i][h] = *reinterpret_cast<const uint32_t*>(codes + c);
                X[i][h] = srow[(int64_t)st * N * 4 + 2 * h + (l16 >> 3)];
            }
        }
#pragma unroll
        for (int i = 0; i < QS; ++i) {
            if (s0 + i >= steps) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float sc = mx_scale(X[i][h]);
                const f32x2 lo = mx_pair<FMT, 0>(q[i][h]), hi = mx_pair<FMT, 1>(q[i][h]);
                const f32x4 o = {lo.x * sc, lo.y * sc, hi.x * sc, hi.y * sc};
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o),
                                            reinterpret_cast<u32x4*>(static_cast<float*>(dst) + row * stride + (int64_t)(s0 + i) * kMxStep + f32_at(l16, h)));
            }
        }
        return;
    }
    uint32_t q[QS][FMT == kMxFp4 ? 1 : 2];                      // bf16: eight codes in a row
    int X[QS];
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        const int st = min(s0 + i, steps - 1);
        const int64_t at = row * K + (int64_t)st * kMxStep + 8 * l16;
        if constexpr (FMT == kMxFp4) {
            q[i][0] = *reinterpret_cast<const uint32_t*>(codes + (at >> 1));
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(codes + at);
            q[i][0] = w.x;
            q[i][1] = w.y;
        }
        X[i] = srow[(int64_t)st * N * 4 + (l16 >> 2)];
    }
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        if (s0 + i >= steps) break;
        const float sc = mx_scale(X[i]);
        f32x2 f[4];
        if constexpr (FMT == kMxFp4) {
            f[0] = mx_pair<FMT, 0>(q[i][0]); f[1] = mx_pair<FMT, 1>(q[i][0]);
            f[2] = mx_pair<FMT, 2>(q[i][0]); f[3] = mx_pair<FMT, 3>(q[i][0]);
        } else {
            f[0] = mx_pair<FMT, 0>(q[i][0]); f[1] = mx_pair<FMT, 1>(q[i][0]);
            f[2] = mx_pair<FMT, 0>(q[i][1]); f[3] = mx_pair<FMT, 1>(q[i][1]);
        }
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 v = {f[j].x * sc, f[j].y * sc};
            w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
        }
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dst) + row * stride + (int64_t)(s0 + i) * kMxStep + 8 * l16));
    }
}

namespace {
dim3 quant_grid(const MxRows& r) {
    return dim3((unsigned)((r.rows + QR - 1) / QR), (unsigned)((r.K / kMxStep + QS - 1) / QS));
}
}  // namespace

hipError_t launch_mx_quantize(const MxRows& r, const void* src, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    const dim3 g = quant_grid(r);
    const auto launch = [&](auto kernel) {
        kernel<<<g, 256, 0, s>>>(src, r.stride, r.rows, r.N, r.K, codes, scales, r.row_src, r.src_rows);
    };
    prof_begin(s);
    if (r.row_src) {                                            // bf16 (the product's x)
        if (r.fmt == kMxFp4) launch(mxq_quantize<kMxFp4, false, true>);
        else launch(mxq_quantize<kMxFp8, false, true>);
    } else if (r.fmt == kMxFp4) {
        if (r.f32) launch(mxq_quantize<kMxFp4, true, false>);
        else launch(mxq_quantize<kMxFp4, false, false>);
    } else {
        if (r.f32) launch(mxq_quantize<kMxFp8, true, false>);
        else launch(mxq_quantize<kMxFp8, false, false>);
    }
    prof_end(s, "mxq_quantize");
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxRows& r, const uint8_t* codes, const uint8_t* scales, void* dst, hipStream_t s) {
    const dim3 g = quant_grid(r);
    prof_begin(s);
    if (r.fmt == kMxFp4) {
        if (r.f32) mxq_dequantize<kMxFp4, true><<<g, 256, 0, s>>>(codes, scales, r.stride, r.rows, r.N, r.K, dst);
        else mxq_dequantize<kMxFp4, false><<<g, 256, 0, s>>>(codes, scales, r.stride, r.rows, r.N, r.K, dst);
    } else {
        if (r.f32) mxq_dequantize<kMxFp8, true><<<g, 256, 0, s>>>(codes, scales, r.stride, r.rows, r.N, r.K, dst);
        else mxq_dequantize<kMxFp8, false><<<g, 256, 0, s>>>(codes, scales, r.stride, r.rows, r.N, r.K, dst);
    }
    prof_end(s, "mxq_dequantize");
    return hipGetLastError();
}

}  // namespace em
