// Product of token rows with int4 matrices in the layer's storage:
//   y[r][n] = sum over groups q of K of s_m[n][q] sum_{k in q} x[src(r)][k] c_m[n][k]
// with c the signed codes and s the fp16 scales of Gq elements each.  Codes become bf16
// exactly (dequant8), x is bf16, a group's products are summed in float32 on the matrix
// cores and the sum is scaled by a float32 fused multiply-add: every weight is exactly
// c s, as in the layer.
//
//   ip_rows    few rows a matrix: bound by the code bytes.  Four or eight waves split K, ask
//              for their codes all at once in operand registers and keep the x rows in the LDS.
//   ip_stream  the same for 17 to 32 rows, and where a tile's scales or rows lie too oddly:
//              x straight from memory.
//   ip_tile    many rows: LDS tiles by direct global -> LDS loads, counted by hand.
#include <type_traits>

#include "common.h"
#include "lds_load.h"
#include "mfma_ops.h"
#include "operators.h"
#include "row_tile.h"

namespace em {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

EM_DEV uint32_t pack2(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

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
        static_cast<uint16_t*>(out)[at] = (uint16_t)pack2(v, v);
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

// What lanes without an element read: x past K.
__device__ const uint4 ip_zero = {0u, 0u, 0u, 0u};

// The W waves' sums of 16 NS rows x 16 NC columns, added in wave order and stored: tile
// i = (subtile s, column tile c) by wave i % W; lane (g, m) holds rows 4 g .. 4 g + 3 of
// column m.  Bit r of named[s]: row_src names an x row for row 16 s + r; without one the row is
// zeros, whatever the scales that met its zeros of x.
template <int W, int NS, int NC>
EM_DEV void join_waves(const Int4Product& a, const floatx4 (&acc)[NS][NC], const uint32_t (&named)[NS], float (&red)[W][NS * NC][256],
                       int r0, int r1, int n0) {
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c) *reinterpret_cast<floatx4*>(&red[wv][s * NC + c][4 * lane]) = acc[s][c];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS * NC; ++i) {
        if (i % W != wv) continue;
        floatx4 v = *reinterpret_cast<const floatx4*>(&red[0][i][4 * lane]);
#pragma unroll
        for (int q = 1; q < W; ++q) v += *reinterpret_cast<const floatx4*>(&red[q][i][4 * lane]);
        const int n = n0 + 16 * (i % NC) + m, r = r0 + 16 * (i / NC) + 4 * g;
        if (n >= a.N) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r + j < r1) store1(a.y, a.y_f32, (int64_t)(r + j) * a.y_stride + n, named[i / NC] >> (4 * g + j) & 1 ? v[j] : 0.f);
    }
}

}  // namespace

// GPC: scale groups in 128 elements of K (1: groups of 128 and more).  The last 32, 64 or 96
// elements of a K that is no multiple of 128 are a chunk whose missing x is zero.
//
// ------------------------------------------------------------------ few rows -----
// A workgroup takes up to 16 rows of one matrix and 16 NC columns, each of its W waves a part
// of K, 4096 / W elements at a time: all of their codes and scales are asked for at once, then
// the x rows into the wave's own part of the LDS, and one wait covers both.  Bound by that
// one trip to memory and what follows it: one token through 8192 x 4096, 18 MB, 7.6 us; 80
// rows over 512 of 128 x 4096, 22 MB, 12.4.
// VEC: a wave's scales of such a block are 8 or 16 bytes (GPC 1: groups of 128, K a multiple
// of 4096), those of a chunk 4 or 8 (GPC 2, 4: K a multiple of 128).  One row through 8192 x 5120,
// whose scales are loaded one by one, takes 10.0 us, 4096 of K 7.8, 3968 7.0.
// Four waves with four groups in 128 of K spill 22 registers: the 80 rows take 17 us with
// groups of 32, 16 with groups of 64, 12.9 with groups of 128.
template <int W, int GPC, int NC, bool VEC>
__global__ void __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2)))
ip_rows(Int4Product a) {
    constexpr int WD = 32 / W, XR = 8, RS = 2 * KC * WD + 16;     // chunks and x rows at once, bytes of an x row in the LDS
    static_assert(XR * RS >= NC * 1024, "");
    __shared__ __attribute__((aligned(16))) uint8_t xl[W][XR * RS];
    const RowTile t = row_tile<16>(a.offsets, a.M, a.R, [&](int) { return a.tile0 + (int)blockIdx.y; });
    if (t.r1 == 0) return;
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
    const int n0 = blockIdx.x * (16 * NC);
    const int chunks = (a.K + KC - 1) / KC;
    const int s0 = chunks * wv / W, s1 = chunks * (wv + 1) / W;
    const int ng = a.K / a.gq, rows = t.r1 - t.r0;

    const uint8_t* wp[NC];
    const uint16_t* sp[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t row = (int64_t)t.m * a.N + min(n0 + 16 * c + m, a.N - 1);
        wp[c] = a.codes + row * (a.K / 2);
        sp[c] = a.scales + row * ng;
    }
    uint4 w[WD][NC];
    constexpr bool BLOCK = VEC && GPC == 1;                       // scales by blocks
    uint4 sb[NC];
    uint2 sc[BLOCK ? 1 : WD][NC];                                 // a chunk's scales, two a word
    auto load_w = [&](int d, int ch) {
        const int k = KC * ch + 32 * g;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            w[d][c] = ld16(wp[c] + min(k, a.K - 32) / 2);
            if constexpr (BLOCK) continue;
            if constexpr (VEC && GPC == 4) {
                sc[d][c] = *reinterpret_cast<const uint2*>(sp[c] + 4 * ch);
            } else if constexpr (VEC && GPC == 2) {
                sc[d][c] = make_uint2(*reinterpret_cast<const uint32_t*>(sp[c] + 2 * ch), 0u);
            } else {
                uint32_t h[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int q = 0; q < GPC; ++q) {
                    const int i = (KC * ch + KC / GPC * q) / a.gq;
                    h[q] = i < ng ? sp[c][min(i, ng - 1)] : 0u;   // past K: nothing, whatever the last scale is
                }
                sc[d][c] = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
            }
        }
    };
    auto scale = [&](int d, int c, int q) {
        uint32_t v;
        if constexpr (BLOCK) v = (d / 2 == 0 ? sb[c].x : d / 2 == 1 ? sb[c].y : d / 2 == 2 ? sb[c].z : sb[c].w) >> (16 * (d & 1));
        else v = (q < 2 ? sc[d][c].x : sc[d][c].y) >> (16 * (q & 1));
        return 16.0f * fp16_bits_to_f32((uint16_t)v);
    };
    auto load_scales_of = [&](int c, int ch) {                    // (BLOCK)
        if constexpr (WD == 8) return ld16(sp[c] + ch);
        const uint2 v = *reinterpret_cast<const uint2*>(sp[c] + ch);
        return make_uint4(v.x, v.y, 0u, 0u);
    };
    auto load_block = [&](int ch) {
        if constexpr (BLOCK) {
#pragma unroll
            for (int c = 0; c < NC; ++c) sb[c] = load_scales_of(c, ch);
        }
#pragma unroll
        for (int d = 0; d < WD; ++d) load_w(d, min(ch + d, s1 - 1));
    };
    if (s0 < s1) load_block(s0);
    const int src = x_row(a, t.r0 + min(m, rows - 1));
    const uint16_t* xp = a.x + (int64_t)max(src, 0) * a.x_stride;  // (more than XR rows) this lane's row
    const bool few = rows <= XR;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&xl[wv][0];
    const uint8_t* xrow = &xl[wv][min(m, rows - 1) * RS];
    floatx4 acc[1][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[0][c] = zero4();
    // One chunk of a block, and two at once: their conversions and products then interleave.
    // (More at once cost registers, and with them waves: whole blocks without a branch took
    // 7.6 us on one token through 8192 x 4096 with four waves, pairs 7.9, single chunks 9.0; 80
    // rows over 512 of 128 x 4096 15.6, 12.4, 13.4.)
    auto chunk = [&](int ch, int d, auto in_lds) {
        constexpr bool LDS = decltype(in_lds)::value;
        const int k0 = KC * (ch + d), left = a.K - k0;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = GPC == 1 ? 32 * g + 8 * i : 32 * i + 8 * g;
            if constexpr (LDS) {
                x[i] = ld16(xrow + 2 * (KC * d + at));
            } else {
                const uint4 v = ld16(xp + k0 + (at < left ? at : 0));
                x[i] = at < left && src >= 0 ? v : zero_u4();
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            uint4 raw = w[d][c];
            if constexpr (GPC > 1) raw = by_group(raw);
            uint4 b[4];
            dequant_b(raw, b);
#pragma unroll
            for (int q = 0; q < GPC; ++q) {
                floatx4 u = zero4();
#pragma unroll
                for (int i = 4 / GPC * q; i < 4 / GPC * (q + 1); ++i) u = mfma_bf16(x[i], b[i], u);
                acc[0][c] = fma4(scale(d, c, q), u, acc[0][c]);
            }
        }
    };
    auto run = [&](auto in_lds) {
        for (int ch = s0; ch < s1; ch += WD) {
            if constexpr (decltype(in_lds)::value) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // the rows before have been read
                for (int r = 0; r < rows; ++r) {
                    const int from = __builtin_amdgcn_readlane(src, r);
                    const uint16_t* p = a.x + (int64_t)max(from, 0) * a.x_stride;
#pragma unroll
                    for (int h = 0; h < WD / 4; ++h) {
                        const int k = KC * ch + 512 * h + 8 * lane;
                        const void* at = from >= 0 && k < a.K ? static_cast<const void*>(p + k) : static_cast<const void*>(&ip_zero);
                        lds_load16(at, __builtin_amdgcn_readfirstlane(base + r * RS + 1024 * h));
                    }
                }
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
            const bool more = ch + WD < s1;
            uint4 sn[NC];
            if constexpr (BLOCK) {
#pragma unroll
                for (int c = 0; c < NC; ++c) sn[c] = load_scales_of(c, min(ch + WD, s1 - WD));
            }
#pragma unroll
            for (int d = 0; d < WD; d += 2) {
                if (ch + d + 1 < s1) {
                    chunk(ch, d, in_lds);
                    chunk(ch, d + 1, in_lds);
                } else if (ch + d < s1) {
                    chunk(ch, d, in_lds);
                }
                if (more) {
                    load_w(d, min(ch + d + WD, s1 - 1));
                    load_w(d + 1, min(ch + d + 1 + WD, s1 - 1));
                }
            }
            if constexpr (BLOCK) {
#pragma unroll
                for (int c = 0; c < NC; ++c) sb[c] = sn[c];
            }
        }
    };
    if (few) run(std::true_type{});
    else run(std::false_type{});
    __syncthreads();                                              // the x rows have been read: their place takes the sums
    const uint32_t named[1] = {(uint32_t)__ballot(src >= 0)};     // (lanes 0 .. 15: rows 0 .. 15)
    join_waves<W, 1, NC>(a, acc, named, *reinterpret_cast<float(*)[W][NC][256]>(&xl[0][0]), t.r0, t.r1, n0);
}

// ------------------------------------------------------------------ 17 to 32 rows ----
template <int GPC, int NS, int NC>
__global__ void __launch_bounds__(256)
ip_stream(Int4Product a) {
    constexpr int WD = NS == 4 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) float red[4][NS * NC][256];
    const RowTile t = row_tile<16 * NS>(a.offsets, a.M, a.R, [&](int) { return a.tile0 + (int)blockIdx.y; });
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
            for (int q = 0; q < GPC; ++q) {
                const int i = (KC * ch + KC / GPC * q) / a.gq;
                sc[d][c][q] = i < ng ? sp[c][min(i, ng - 1)] : (uint16_t)0;     // past K: nothing, whatever the last scale is
            }
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
    uint32_t named[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) named[s] = (uint32_t)__ballot(live[s]);      // (lanes 0 .. 15: rows 16 s .. 16 s + 15)
    join_waves<4, NS, NC>(a, acc, named, red, t.r0, t.r1, n0);
}

// ------------------------------------------------------------------ many rows ----
// A workgroup takes BT rows x BN columns, each wave all rows of 32 columns, so that no code
// is converted twice; 128 of K a step.  x, codes and scales arrive by direct global -> LDS
// loads two steps ahead in three stages, every wave as many loads a step.  A scale comes as
// the aligned word that holds it.  256-byte x rows, 16-byte segments XOR-swizzled by the row
// (with groups of 128 and more the segments that lane groups 0 .. 3 read together are kept
// side by side); 64-byte code rows as mx_product.hip's.  Bound by the matrix cores and, of
// the same order, the conversion of the codes: 4096 rows in 8 groups through 8192 x 4096
// 308 us, 0.89 PFLOP/s, 1001 through 4096 x 8192 114 (groups of 32 179); waves of 64 rows x
// 64 columns, which read half as much of x from the LDS and convert each code twice, 364 and
// 141.
namespace {

template <int GPC, int BT_, int BN_>
struct IpCfg {
    static constexpr int BT = BT_, BN = BN_, NW = BN / 32, NJ = BT / 16;
    static constexpr int X_B = BT * 256, W_B = BN * 64, S_B = BN * 4 * GPC, STAGE = X_B + W_B + S_B;
    static constexpr int X_L = X_B / 1024 / NW, W_L = W_B / 1024 / NW, S_P = S_B / 256, S_L = (S_P + NW - 1) / NW;
    static constexpr int LOADS = X_L + W_L + S_L;
    static constexpr int RS = BN + 4;                             // floats of an out row in the LDS
    static constexpr int LDS_B = 3 * STAGE > BT * RS * 4 ? 3 * STAGE : BT * RS * 4;
    static_assert(LDS_B <= 160 * 1024, "");
};

// Slot of x segment s (eight elements) of row r; of code segment s (32 codes) of column r.
template <int GPC>
EM_DEV int x_slot(int r, int s) { return (GPC == 1 ? s >> 2 | (s & 3) << 2 : s) ^ (r & 15); }
EM_DEV int w_slot(int r, int s) { return s ^ (-(r >> 2) & 3); }

}  // namespace

template <int GPC, int BT, int BN>
__global__ void __launch_bounds__((IpCfg<GPC, BT, BN>::NW * 64))
ip_tile(Int4Product a) {
    using C = IpCfg<GPC, BT, BN>;
    constexpr int NJ = C::NJ;
    __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS_B];
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
    const int nn = (a.N + BN - 1) / BN;
    int tn = 0, z = 0;
    const RowTile t = row_tile<BT>(a.offsets, a.M, a.R, [&](int rows) {
        rows = min(rows, a.row_tiles);                            // more only where offsets descend
        const int each = rows * nn, total = each * a.slices, per = (total + 7) >> 3, at = blockIdx.x >> 3;
        int b = (blockIdx.x & 7) * per + at;                      // XCD x takes neighbouring tiles
        if (at >= per || b >= total) return -1;
        z = b / each;
        b -= z * each;
        const int grp = b / (8 * nn), left = min(8, rows - 8 * grp), in = b - grp * 8 * nn;
        tn = in / left;
        return 8 * grp + in % left;
    });
    if (t.r1 == 0) return;
    const int n0 = tn * BN, rows = t.r1 - t.r0, ng = a.K / a.gq;
    uint64_t named[BT / 64];                                      // rows whose x row row_src names
#pragma unroll
    for (int h = 0; h < BT / 64; ++h) named[h] = __ballot(x_row(a, t.r0 + min(64 * h + lane, rows - 1)) >= 0);
    auto has_x = [&](int r) { return (BT == 64 || r < 64 ? named[0] : named[BT / 64 - 1]) >> (r & 63) & 1; };
    const int steps = (a.K + KC - 1) / KC, whole_steps = a.K / KC;
    const int s0 = (int)((int64_t)steps * z / a.slices), s1 = (int)((int64_t)steps * (z + 1) / a.slices);

    // ---- loads: load u of a wave brings piece u NW + wv of x, of the codes, of the scales
    const char* xbase = reinterpret_cast<const char*>(a.row_src ? a.x : a.x + (int64_t)t.r0 * a.x_stride);
    const uint8_t* wbase = a.codes + ((int64_t)t.m * a.N + n0) * (a.K / 2);
    uint32_t xoff[C::X_L], woff[C::W_L], soff[C::S_L];
    // The lane's first element of K within a step: of an x load, of a code load.
    auto x_k = [&](int u) {
        const int row = (u * C::NW + wv) * 4 + lane / 16, slot = (lane & 15) ^ (row & 15);
        return 8 * (GPC == 1 ? slot >> 2 | (slot & 3) << 2 : slot);
    };
    auto w_k = [&](int u) { return 32 * w_slot((u * C::NW + wv) * 16 + lane / 4, lane & 3); };
#pragma unroll
    for (int u = 0; u < C::X_L; ++u) {
        const int r = min((u * C::NW + wv) * 4 + lane / 16, rows - 1);
        xoff[u] = (uint32_t)(2 * ((a.row_src ? max(x_row(a, t.r0 + r), 0) : r) * a.x_stride + x_k(u)));
    }
#pragma unroll
    for (int u = 0; u < C::W_L; ++u) woff[u] = min((u * C::NW + wv) * 16 + lane / 4, a.N - 1 - n0) * (a.K / 2) + w_k(u) / 2;
    // where the scales' pieces run out before the waves, the first again
    auto s_piece = [&](int u) { return (u * C::NW + wv) % C::S_P; };
#pragma unroll
    for (int u = 0; u < C::S_L; ++u) soff[u] = min(64 * (s_piece(u) % (BN / 64)) + lane, a.N - 1 - n0) * ng;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int64_t srow0 = ((int64_t)t.m * a.N + n0) * ng;         // index of the first column's first scale
    const uint16_t* sbase = a.scales + (srow0 & ~1ll);
    const int sodd = (int)srow0 & 1;
    // index of scale group q of step st, the last one past K
    auto group_of = [&](int st, int q) { return min((KC * st + KC / GPC * q) / a.gq, ng - 1); };
    auto fetch = [&](int st, int u, auto fast) {
        constexpr bool FAST = decltype(fast)::value;              // all of the step's K exists
        const uint32_t stage = base + (uint32_t)(st % 3) * C::STAGE;
        if (u < C::X_L) {
            const uint32_t dst = __builtin_amdgcn_readfirstlane(stage + 1024 * (u * C::NW + wv));
            const char* from = xbase + (int64_t)st * 256;
            if constexpr (FAST) lds_load16(from, xoff[u], dst);
            else lds_load16(KC * st + x_k(u) < a.K ? from + xoff[u] : reinterpret_cast<const char*>(&ip_zero), dst);
        } else if (u < C::X_L + C::W_L) {
            const int v = u - C::X_L;
            const uint32_t dst = __builtin_amdgcn_readfirstlane(stage + C::X_B + 1024 * (v * C::NW + wv));
            if constexpr (FAST) lds_load16(wbase + (int64_t)st * 64, woff[v], dst);
            else lds_load16(wbase, woff[v] - w_k(v) / 2 + min(KC * st + w_k(v), a.K - 32) / 2, dst);      // codes past K meet zeros
        } else {
            const int v = u - C::X_L - C::W_L, piece = s_piece(v);
            const uint32_t i = (uint32_t)sodd + soff[v] + group_of(st, piece / (BN / 64));
            lds_load4(sbase, 2u * (i & ~1u), __builtin_amdgcn_readfirstlane(stage + C::X_B + C::W_B + 256 * piece));
        }
    };

    floatx4 acc[2][NJ];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[p][j] = zero4();
    int odd[2];                                                   // parity of a column's first scale index
#pragma unroll
    for (int p = 0; p < 2; ++p) odd[p] = (sodd + min(32 * wv + 16 * p + m, a.N - 1 - n0) * ng) & 1;
    auto step = [&](int st, auto fast) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(C::LOADS) : "memory");   // this step landed, the one before is read
        const uint8_t* X = lds + (st % 3) * C::STAGE;
        const uint8_t* W = X + C::X_B;
        const uint32_t* S = reinterpret_cast<const uint32_t*>(W + C::W_B);
        uint4 raw[2];
        float sc[2][GPC];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int col = 32 * wv + 16 * p + m;
            raw[p] = *reinterpret_cast<const uint4*>(W + col * 64 + 16 * w_slot(m, g));
            if constexpr (GPC > 1) raw[p] = by_group(raw[p]);
#pragma unroll
            for (int q = 0; q < GPC; ++q) {
                const uint32_t v = S[q * BN + col] >> (16 * ((odd[p] + group_of(st, q)) & 1));
                const bool in = KC * st + KC / GPC * q < a.K;     // past K: nothing, whatever the last scale is
                sc[p][q] = in ? 16.0f * fp16_bits_to_f32((uint16_t)v) : 0.f;
            }
        }
        floatx4 u[2][NJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 x[NJ], b[2];                                    // converted 32 of K at a time, under the other wave's products
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                x[j] = *reinterpret_cast<const uint4*>(X + (16 * j + m) * 256 + 16 * x_slot<GPC>(m, GPC == 1 ? 4 * g + i : 4 * i + g));
#pragma unroll
            for (int v = i * C::LOADS / 4; v < (i + 1) * C::LOADS / 4; ++v) fetch(st + 2, v, fast);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t q[4];
                dequant8(i == 0 ? raw[p].x : i == 1 ? raw[p].y : i == 2 ? raw[p].z : raw[p].w, q);
                b[p] = make_uint4(q[0], q[1], q[2], q[3]);
            }
            const bool first = i % (4 / GPC) == 0, last = (i + 1) % (4 / GPC) == 0;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int j = 0; j < NJ; ++j) u[p][j] = mfma_bf16(x[j], b[p], first ? zero4() : u[p][j]);
            if (last) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) acc[p][j] = fma4(sc[p][i * GPC / 4], u[p][j], acc[p][j]);
            }
        }
    };
    if (s0 < s1) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int u = 0; u < C::LOADS; ++u) fetch(s0 + st, u, std::false_type{});
        int st = s0;
        for (; st < s1 && st + 2 < whole_steps; ++st) step(st, std::true_type{});
        for (; st < s1; ++st) step(st, std::false_type{});
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");        // nothing more lands in the stages

    // ---- out through the LDS, whole rows: lane (g, m) holds rows 4 g .. 4 g + 3 of column m
    float* o = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int v = 0; v < 4; ++v) o[(16 * j + 4 * g + v) * C::RS + 32 * wv + 16 * p + m] = acc[p][j][v];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int cols = min(BN, a.N - n0);
    if (a.slices > 1) {
        const int Np = (a.N + 3) & ~3;
        for (int i = threadIdx.x; i < rows * (BN / 4); i += C::NW * 64) {
            const int r = i / (BN / 4), c = 4 * (i % (BN / 4));
            if (c < cols)                                         // (the join knows no row_src)
                *reinterpret_cast<floatx4*>(a.part + ((int64_t)z * a.R + t.r0 + r) * Np + n0 + c) =
                    has_x(r) ? *reinterpret_cast<const floatx4*>(o + r * C::RS + c) : zero4();
        }
        return;
    }
    const int each = a.y_f32 ? 4 : 8, per = BN / each;            // columns of a store, stores of a row
    for (int i = threadIdx.x; i < rows * per; i += C::NW * 64) {
        const int r = i / per, c = each * (i % per);
        if (c >= cols) continue;
        const bool live = has_x(r);
        const floatx4 lo = live ? *reinterpret_cast<const floatx4*>(o + r * C::RS + c) : zero4();
        const int64_t at = (int64_t)(t.r0 + r) * a.y_stride + n0 + c;
        if (a.y_f32) {
            if (a.vec && c + 4 <= cols) {
                __builtin_nontemporal_store(lo, reinterpret_cast<floatx4*>(static_cast<float*>(a.y) + at));
            } else {
                for (int k = 0; k < 4 && c + k < cols; ++k) static_cast<float*>(a.y)[at + k] = lo[k];
            }
            continue;
        }
        const floatx4 hi = live ? *reinterpret_cast<const floatx4*>(o + r * C::RS + c + 4) : zero4();
        const u32x4 v = {pack2(lo.x, lo.y), pack2(lo.z, lo.w), pack2(hi.x, hi.y), pack2(hi.z, hi.w)};
        uint16_t* y = static_cast<uint16_t*>(a.y) + at;
        if (a.vec && c + 8 <= cols) {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y));
        } else {
            for (int k = 0; k < 8 && c + k < cols; ++k) y[k] = (uint16_t)(v[k / 2] >> (16 * (k & 1)));
        }
    }
}

// ------------------------------------------------------------------ host side ----
namespace {

int64_t max_row_tiles(const Int4Product& a, int BT) {
    const int live = a.M < a.R ? a.M : a.R;
    return a.M > 1 ? a.R / BT + live : (a.R + BT - 1) / BT;
}

// Launches of `tiles` row tiles: a grid takes up to 65536 of them in its second dimension.
template <class F>
hipError_t launch_row_tiles(Int4Product a, int64_t tiles, const char* name, hipStream_t s, F launch) {
    prof_begin(s);
    for (; a.tile0 < tiles; a.tile0 += 65536) launch(a, (unsigned)(tiles - a.tile0 < 65536 ? tiles - a.tile0 : 65536));
    prof_end(s, name);
    return hipGetLastError();
}

template <int GPC, int NS>
hipError_t launch_stream(const Int4Product& a, hipStream_t s) {
    return launch_row_tiles(a, max_row_tiles(a, 16 * NS), "ip_stream", s, [&](const Int4Product& b, unsigned tiles) {
        ip_stream<GPC, NS, 2><<<dim3((a.N + 31) / 32, tiles), 256, 0, s>>>(b);
    });
}

template <int W, int GPC, int NC>
hipError_t launch_rows(const Int4Product& a, hipStream_t s) {
    const bool vec = GPC == 1 ? a.gq == KC && a.K % 4096 == 0 : a.K % KC == 0;
    return launch_row_tiles(a, max_row_tiles(a, 16), "ip_rows", s, [&](const Int4Product& b, unsigned tiles) {
        const dim3 grid((a.N + 16 * NC - 1) / (16 * NC), tiles);
        if (vec) ip_rows<W, GPC, NC, true><<<grid, 64 * W, 0, s>>>(b);
        else ip_rows<W, GPC, NC, false><<<grid, 64 * W, 0, s>>>(b);
    });
}

struct IpPlan { int bt, bn, slices; };                            // bn 0: ip_rows (bt 16) or ip_stream (32, 64)

// The least of an estimate in us from measured times.  Few rows: K / 4096 times a part of
// its own and one a workgroup.  Tiles: a step of 128 of K alone on a compute unit or with it
// full, 1.25 and 1.6 times that with two and four scale groups a step; slices of K are
// joined by a launch more.  Measured (us, inputs in the memory-side cache, rows through M x N x
// K; 16, 32: rows a workgroup, tiles rows x columns / slices): 20 through 4096 x 4096 16 8.9, 32
// 13.0, 64x128/8 12.5; 64 through 1024 x 4096 16 8.1, 32 14.8; 32 through 8192 x 4096 16 14.9, 32
// 15.6, 64x128/4 16.3; 256 through 4096 x 4096 64x256/4 26.5, 64x128/2 24.2, 128x256/8 27.6, 64x128
// 33.6; 4096 through 4096 x 4096 128x256 128, 64x128 181; 4096 routed over 64 of 128 x 4096 64x128/4
// 22.3, 128x256/4 27.4.
IpPlan plan(const Int4Product& a) {
    struct Cost { int bt, bn, fit; float fixed, alone, full; };
    static constexpr Cost kTiles[3] = {{64, 128, 2, 3.0f, 0.98f, 1.33f}, {64, 256, 1, 3.0f, 1.25f, 1.30f}, {128, 256, 1, 4.0f, 1.70f, 2.00f}};
    const int live = a.M < a.R ? a.M : (a.R ? a.R : 1);
    const float each = (float)a.R / live, k = a.K / 4096.0f;
    // row tiles of a matrix: among few matrices the last one is half empty on average; many
    // (routed experts) have about as many rows each
    const auto row_tiles = [&](int bt) {
        const float q = each / bt, up = (float)(int)(q + 0.9f);
        return a.M == 1 ? (float)((a.R + bt - 1) / bt) : (float)live * (a.M < 64 && q > 0.5f ? q + 0.5f : up > q + 0.25f ? up : q + 0.25f);
    };
    const auto few = [&](int bt, float own, float one, int fit) {  // workgroups past `fit` cost 0.055 each
        const float n = row_tiles(bt) * ((a.N + 31) / 32);
        return 4 + k * (own + one * (n < fit ? n : fit) + 0.055f * (n > fit ? n - fit : 0));
    };
    IpPlan best{16, 0, 1};
    float least = few(16, 3.4f, 0.0234f, 512);
    const auto take = [&](float us, IpPlan p) {
        if (us < least) {
            least = us;
            best = p;
        }
    };
    take(few(32, 9.8f, 0.0115f, 256), IpPlan{32, 0, 1});
    // a tile takes scales by words, and the last word would end past them where a matrix has an odd
    // number (1001 rows through 1025 x 4224, 33 groups a column, 52 us; through 1024 columns 25)
    if ((int64_t)a.N * (a.K / a.gq) % 2) {
        take(each > 64 ? 0.f : least, IpPlan{64, 0, 1});
        return best;
    }
    const int steps = (a.K + KC - 1) / KC;
    const float groups = a.gq >= KC || a.gq == a.K ? 1.f : a.gq == 64 ? 1.25f : 1.6f;
    for (const Cost& t : kTiles) {
        const float tiles = row_tiles(t.bt) * ((a.N + t.bn - 1) / t.bn);
        for (int z = 1; z <= 8 && (z == 1 || (steps >= 2 * z && tiles * z < 2048)); z *= 2) {
            const float n = tiles * z / 256, part = (float)((steps + z - 1) / z) * groups;
            const int rounds = (int)(n / t.fit);
            const float rest = n - rounds * t.fit;                // tiles a compute unit in the last round
            float us = 4 + rounds * (t.fixed + part * t.full);
            if (rest > 0) {
                const float share = t.fit == 1 ? (rounds ? 1.f : rest) : (rest < 1 ? 0.f : rest - 1);
                us += t.fixed + part * (t.alone + (t.full - t.alone) * (share < 1 ? share : 1.f));
            }
            if (z > 1) us += 4 + 0.15f * z + (float)((double)a.R * a.N * (8 * z + 2) / 5e6);
            take(us, IpPlan{t.bt, t.bn, z});
        }
    }
    return best;
}

template <int GPC, int BT, int BN>
hipError_t launch_tile(Int4Product a, const IpPlan& p, hipStream_t s) {
    a.slices = p.slices;
    a.row_tiles = (int)max_row_tiles(a, BT);
    const int64_t blocks = (int64_t)a.row_tiles * ((a.N + BN - 1) / BN) * p.slices;
    prof_begin(s);
    ip_tile<GPC, BT, BN><<<(unsigned)((blocks + 7) & ~7ll), IpCfg<GPC, BT, BN>::NW * 64, 0, s>>>(a);
    prof_end(s, "ip_tile");
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.slices == 1) return e;
    return launch_join(RowJoin{a.part, p.slices, a.R, a.N, a.y, a.y_stride, a.y_f32, a.vec && a.N % 4 == 0, a.R, a.offsets, a.M,
                               nullptr, 0}, s);
}

template <int GPC>
hipError_t launch_product(const Int4Product& a, hipStream_t s) {
    IpPlan p = plan(a);
    // lane offsets of a tile's x rows have 32 bits (600 gathered rows through 4096 x 4096, x rows 2^22
    // elements apart: 105 us, close together in tiles 49)
    const int64_t rows = a.row_src ? a.T : 128;
    if (p.bn && rows * a.x_stride >= (1ll << 31)) p = IpPlan{64, 0, 1};
    if (p.bn == 0) {
        if (p.bt == 64) return launch_stream<GPC, 4>(a, s);
        if (p.bt == 32) return launch_stream<GPC, 2>(a, s);
        // 32 columns a workgroup, 16 where that leaves half of the compute units idle; eight
        // waves a workgroup while each has a compute unit to itself, four where two share one
        // (one token through 8192 x 4096 with four 7.9 us, with eight 7.7, 12 tokens 10.5 and
        // 8.9; 80 rows over 512 of 128 x 4096, 340 workgroups, 12.4 and 14.8)
        const int64_t wgs = max_row_tiles(a, 16) * ((a.N + 31) / 32);
        return wgs <= 128 ? launch_rows<8, GPC, 1>(a, s) : wgs <= 256 ? launch_rows<8, GPC, 2>(a, s) : launch_rows<4, GPC, 2>(a, s);
    }
    if (p.bn == 128) return launch_tile<GPC, 64, 128>(a, p, s);
    return p.bt == 64 ? launch_tile<GPC, 64, 256>(a, p, s) : launch_tile<GPC, 128, 256>(a, p, s);
}

}  // namespace

size_t int4_product_ws_bytes(const Int4Product& a) {
    const IpPlan p = plan(a);
    return p.slices > 1 ? ((size_t)p.slices * a.R * ((a.N + 3) & ~3) * 4 + 255) & ~(size_t)255 : 256;
}

hipError_t launch_int4_product(Int4Product a, void* ws, hipStream_t s) {
    a.part = static_cast<float*>(ws);
    if (a.gq >= KC || a.gq == a.K) return launch_product<1>(a, s);    // (a narrower group is the whole of a K below 128)
    return a.gq == 64 ? launch_product<2>(a, s) : launch_product<4>(a, s);
}

}  // namespace em
