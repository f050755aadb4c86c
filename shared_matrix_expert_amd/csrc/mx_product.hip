// MX product: y[r] = bf16(sum_k Q(x[src(r)])[k] * W_m[k]), W_m an MXFP4 matrix
// [N][K], m the matrix that row r belongs to, Q the rounding of x to MXFP8 or
// MXFP4 along K (mx_quant.hip's rule).
//
// The matrix cores multiply the stored codes and apply both operands' block
// scales (v_mfma_scale_f32_16x16x128_f8f6f4), so no code is converted.  W is the
// instruction's row operand and x its column operand: a lane then holds four
// consecutive columns of one y row.  Operand layout (lane l = 16 g + m):
//   E2M1: row / column m, nibbles K 32 g .. 32 g + 31
//   E4M3: bytes 0-15 K 16 g .. 16 g + 15, bytes 16-31 K 64 + 16 g .. + 15
//   scale byte: K block g of row / column m;  D: W rows 4 g .. 4 g + 3, x row m.
// An instruction sums its 128 products to about 2^-13.5 of their magnitude sum;
// y is rounded to bf16 (2^-8), which is what keeps that invisible.
//
//   mxp_stream  few rows per matrix: bound by the weight bytes.  Each wave
//               streams its part of K from HBM straight into operand registers
//               and rounds the x rows it needs on the way.
//   mxp_gemm    many rows: x rounded once (mxq_quantize into the workspace),
//               LDS-tiled.  An instruction takes 32 cycles with x in E4M3, 16 with
//               x in E2M1; the matrix cores are busy 61% and 47% of the cycles.
#include "lds_load.h"
#include "mx_format.h"
#include "operators.h"
#include "row_tile.h"

namespace em {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

EM_DEV uint4 ldg16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

template <int FMT> constexpr int mx_code() { return FMT == kMxFp4 ? 4 : 0; }   // the instruction's format field

// acc += W (E2M1) . x (FMT) over 128 elements of K.
template <int FMT>
EM_DEV floatx4 mfma_mx(const uint4& w, int ws, const i32x8& x, int xs, const floatx4& acc) {
    const i32x8 a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, acc, 4, mx_code<FMT>(), 0, ws, 0, xs);
}

// An x fragment's registers.
template <int FMT> struct XOp { typedef int type __attribute__((ext_vector_type(FMT == kMxFp4 ? 4 : 8))); };

// ---- rows ------------------------------------------------------------------
// x row of y row r, -1 where row_src names none.
EM_DEV int x_row(const MxProduct& a, int r) {
    if (!a.row_src) return r;
    const int s = a.row_src[r];
    return (unsigned)s < (unsigned)a.T ? s : -1;
}

// Row of the rounded x in the workspace for y row r (row 0 where row_src names none).
EM_DEV int xq_row(const MxProduct& a, int r) { return a.gathered ? r : max(x_row(a, r), 0); }

// Four consecutive columns of a y row (`whole`: all four exist and take one store).
EM_DEV void store4(const MxProduct& a, int64_t r, int n, const floatx4& v, bool whole) {
    uint16_t* p = a.y + r * a.y_stride + n;
    const f32x2 lo = {v.x, v.y}, hi = {v.z, v.w};
    const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2));
    const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2));
    if (whole) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w0, w1);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.N) p[i] = (uint16_t)((i < 2 ? w0 : w1) >> (16 * (i & 1)));
}

// ---- x rounded by a wave ------------------------------------------------------
// Codes of 16 neighbouring bf16 elements (a lane and its neighbour share a
// block) and the block's scale byte.
template <int FMT>
EM_DEV void round16(const uint4 (&v)[2], uint32_t (&q)[4], int& X) {
    const uint32_t mine = max(amax8_bf16(v[0]), amax8_bf16(v[1]));
    const uint32_t a = max(mine, (uint32_t)__builtin_amdgcn_update_dpp((int)mine, (int)mine, 0xB1, 0xF, 0xF, false));
    X = e8m0_of<FMT>(a);
    const bool bad = X == 255;
    const float sc = e8m0_f32(bad ? 127 : X);
    if constexpr (FMT == kMxFp4) {
        q[0] = fp4x8_bf16(v[0], sc);
        q[1] = fp4x8_bf16(v[1], sc);
        q[2] = q[3] = 0;
    } else {
        const uint32_t lim = e4m3_limit(bad ? 127 : X);
        q[0] = fp8x4_bf16(v[0].x, v[0].y, sc, lim);
        q[1] = fp8x4_bf16(v[0].z, v[0].w, sc, lim);
        q[2] = fp8x4_bf16(v[1].x, v[1].y, sc, lim);
        q[3] = fp8x4_bf16(v[1].z, v[1].w, sc, lim);
    }
    if (bad) q[0] = q[1] = q[2] = q[3] = 0;
}

}  // namespace

// ------------------------------------------------------------------ few rows -----
// A workgroup takes one row tile (16 NS rows of one matrix) and 16 NC columns;
// its four waves split K into contiguous quarters and their partial sums are
// added through LDS in wave order.  The weights run WD steps ahead in
// registers: at K = 4096 and WD = 8 a wave's whole share is asked for at once.
// x comes rounded from the workspace, or (FUSED, 16 rows) the wave rounds the
// rows it has, 1024 elements of K at a time, into its own part of the LDS while
// its weights are in flight.  (Rounding in operand registers instead, every lane
// its own row's elements, costs 16 rows' work whatever their number: one token
// through 8192 x 4096 took 9.4 us that way.)
// One row through 8192 x 4096: 6.3 us for 17.8 MB, the launch, one trip to memory (W
// and x are asked for together) and the chain behind it (rounding, products, the
// sum of four waves); through 8192 x 32768: 27 us a call, 5.2 TB/s.  80 rows over 512
// matrices of 128 x 4096: 10 us, three trips in turn: the offsets; W and then the row
// list, which comes back behind all of W since loads return in order; x.
template <int FMT, int NS, int NC, bool FUSED>
__global__ void __launch_bounds__(256)
mxp_stream(MxProduct a) {
    constexpr int WD = NS == 4 ? 4 : 8, XD = NS == 4 ? 1 : 2;
    constexpr int XB = FMT == kMxFp4 ? 64 : 128;                  // bytes of an x row per step
    constexpr int RS = 8 * XB + 16, SS = 36;                      // LDS row strides: codes of 8 steps, scale bytes
    constexpr int XL = FUSED ? 16 * (RS + SS) : 16;
    __shared__ __attribute__((aligned(16))) uint8_t xl[4][XL];
    __shared__ __attribute__((aligned(16))) float red[4][NS * NC][256];
    const RowTile t = row_tile<16 * NS>(a.offsets, a.M, a.R, [](int) { return (int)blockIdx.y; });
    if (t.r1 == 0) return;
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
    const int n0 = blockIdx.x * (16 * NC);
    const int steps = a.K / kMxStep;
    const int s0 = steps * wv / 4, s1 = steps * (wv + 1) / 4;

    const uint8_t* wp[NC];
    const uint8_t* sp[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = min(n0 + 16 * c + m, a.N - 1);
        wp[c] = a.codes + ((int64_t)t.m * a.N + col) * (a.K / 2) + 16 * g;
        sp[c] = a.scales + ((int64_t)t.m * steps * a.N + col) * 4 + g;
    }
    uint4 w[WD][NC];
    int ws[WD][NC];
    auto load_w = [&](int d, int st) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            w[d][c] = ldg16(wp[c] + (int64_t)st * (kMxStep / 2));
            ws[d][c] = sp[c][(int64_t)st * a.N * 4];
        }
    };
    if (s0 < s1) {
#pragma unroll
        for (int d = 0; d < WD; ++d) load_w(d, min(s0 + d, s1 - 1));
    }
    int src[NS], qrow[NS];                                        // x row of y row r0 + 16 s + m; its row in the workspace
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const int r = t.r0 + 16 * s + m;
        src[s] = r < t.r1 ? x_row(a, r) : -1;
        qrow[s] = a.gathered ? min(r, t.r1 - 1) : max(src[s], 0);
    }
    uint4 xv[XD][NS][2];
    int xsv[XD][NS];
    auto load_x = [&](int d, int st) {                            // (!FUSED) operand registers from the workspace
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int64_t row = qrow[s];
            const uint8_t* p = a.xq + row * (a.K / 128 * XB) + (int64_t)st * XB + 16 * g;
            xv[d][s][0] = ldg16(p);
            xv[d][s][1] = FMT == kMxFp8 ? ldg16(p + 64) : make_uint4(0u, 0u, 0u, 0u);
            xsv[d][s] = a.xs[((int64_t)st * a.xrows + row) * 4 + g];
        }
    };
    floatx4 acc[NS][NC];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[s][c] = zero4();
    if constexpr (!FUSED) {
        if (s0 < s1) {
#pragma unroll
            for (int d = 0; d < XD; ++d) load_x(d, min(s0 + d, s1 - 1));
        }
    }
    // WD steps; but for the last ones (`more`) without a branch, which would make
    // each step wait for the loads it has just issued (one row through 8192 x 32768:
    // 34.2 us with branches, 27.1 without)
    auto run = [&](int st, auto more) {
        constexpr bool MORE = decltype(more)::value;
        if constexpr (FUSED) {
            // rows in turn, 16 elements a lane: steps st .. st + 7 of this wave
            const int left = min(8, s1 - st) * kMxStep;           // elements of K (the loads past them repeat the last)
            const int at = min(16 * lane, left - 16);
            const int rows = t.r1 - t.r0;
            auto fetch = [&](int row, uint4 (&v)[2]) {
                const uint16_t* p = a.x + (int64_t)max(__builtin_amdgcn_readlane(src[0], row), 0) * a.x_stride
                                    + (int64_t)st * kMxStep + at;
                v[0] = ldg16(p);
                v[1] = ldg16(p + 8);
            };
            uint4 cur[2], nxt[2];
            fetch(0, nxt);
            asm volatile("" ::: "memory");                        // the steps before have read the buffer
            for (int row = 0; row < rows; ++row) {
                cur[0] = nxt[0];
                cur[1] = nxt[1];
                if (row + 1 < rows) fetch(row + 1, nxt);
                uint32_t q[4];
                int X;
                round16<FMT>(cur, q, X);
                uint8_t* o = &xl[wv][row * RS + lane * (XB / 8)];
                if constexpr (FMT == kMxFp4) *reinterpret_cast<uint2*>(o) = make_uint2(q[0], q[1]);
                else *reinterpret_cast<uint4*>(o) = make_uint4(q[0], q[1], q[2], q[3]);
                if (!(lane & 1)) xl[wv][16 * RS + row * SS + (lane >> 1)] = (uint8_t)X;
            }
            __builtin_amdgcn_wave_barrier();                      // one wave's LDS accesses complete in order
            asm volatile("" ::: "memory");
        }
#pragma unroll
        for (int d = 0; d < WD; ++d) {
            if (MORE || st + d < s1) {
                i32x8 q[NS];
                int xs[NS];
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    uint4 lo, hi = make_uint4(0u, 0u, 0u, 0u);
                    if constexpr (FUSED) {
                        const uint8_t* p = &xl[wv][m * RS + d * XB + 16 * g];
                        lo = ldg16(p);
                        if constexpr (FMT == kMxFp8) hi = ldg16(p + 64);
                        xs[s] = xl[wv][16 * RS + m * SS + 4 * d + g];
                    } else {
                        lo = xv[d % XD][s][0];
                        hi = xv[d % XD][s][1];
                        xs[s] = xsv[d % XD][s];
                    }
                    q[s] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
                }
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int c = 0; c < NC; ++c) acc[s][c] = mfma_mx<FMT>(w[d][c], ws[d][c], q[s], xs[s], acc[s][c]);
                if constexpr (!FUSED)
                    load_x(d % XD, min(st + d + XD, s1 - 1));
                if constexpr (MORE) load_w(d, min(st + d + WD, s1 - 1));
            }
        }
    };
    int st = s0;
    for (; st + WD < s1; st += WD) run(st, std::true_type{});
    if (st < s1) run(st, std::false_type{});
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c) *reinterpret_cast<floatx4*>(&red[wv][s * NC + c][4 * lane]) = acc[s][c];
    __syncthreads();
    // tile i = (subtile s, column tile c) is summed by wave i % 4
#pragma unroll
    for (int i = 0; i < NS * NC; ++i) {
        if ((i & 3) != wv) continue;
        floatx4 v = *reinterpret_cast<const floatx4*>(&red[0][i][4 * lane]);
#pragma unroll
        for (int q = 1; q < 4; ++q) {
            const floatx4 u = *reinterpret_cast<const floatx4*>(&red[q][i][4 * lane]);
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        const int s = i / NC, c = i % NC, r = t.r0 + 16 * s + m;
        if (r < t.r1) store4(a, r, n0 + 16 * c + 4 * g, src[s] >= 0 ? v : zero4(), a.vec >= 2 && n0 + 16 * (c + 1) <= a.N);
    }
}

// ------------------------------------------------------------------ many rows ----
// A workgroup of 8 waves takes BT rows x BN columns in WN x WT waves.  Each K
// step's codes and scale words arrive by direct global -> LDS loads, STAGES - 1
// steps ahead; every wave issues the same number of loads a step, so one counted
// wait covers them.  A code row is 64 (E2M1) or 128 (E4M3) bytes; its 16-byte
// segments are stored XOR-swizzled by the row against bank conflicts.
// 16384 x 8192 x 4096 in FP8: 419 to 433 us in a long run of launches (440 to 500 in
// its first twenty), 2.6 PFLOP/s (a large library product in FP8: 2.65);
// 5001 rows in 8 groups through 4096 x 8192 in FP4: 118 to 128 us, two rounds of
// 192-row tiles, 2.7 PFLOP/s, half of what the instruction's 16 cycles would allow.
// (Four waves of 128 x 128, one a SIMD with 256 accumulators each, read a quarter
// less from the LDS and measured 479 against 450 us on 16384 x 8192 x 4096 in FP8:
// one wave's waits leave its matrix core idle.)
namespace {

template <int FMT, int BT_, int BN_>
struct GemmCfg {
    static constexpr int BT = BT_, BN = BN_;
    static constexpr int WN = BT >= 192 || BN == 128 ? 2 : 4, WT = 8 / WN, NW = WN * WT;
    static constexpr int NI = BN / WN / 16, NJ = BT / WT / 16;     // column and row subtiles of a wave
    static constexpr int XB = FMT == kMxFp4 ? 64 : 128;            // bytes of an x row per step
    static constexpr int X_B = BT * XB, W_B = BN * 64, XS_B = BT * 4, WS_B = BN * 4;
    static constexpr int STAGE = X_B + W_B + XS_B + WS_B;
    static constexpr int STAGES = 4 * STAGE <= 160 * 1024 ? 4 : 3;
    static constexpr int X_P = X_B / 1024, W_P = W_B / 1024, S_P = (BN + BT) / 64;   // wave loads a stage
    static constexpr int X_INSTR = (X_P + NW - 1) / NW, W_INSTR = W_P / NW, S_INSTR = (S_P + NW - 1) / NW;
    static constexpr int LOADS = X_INSTR + W_INSTR + S_INSTR;
};

EM_DEV void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

// At most N of this wave's loads in flight, its LDS reads done; then the barrier.
template <int N>
EM_DEV void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

template <int I> struct Set { static constexpr int value = I; };     // one of two register sets

// Segment slot of row r's 16-byte segment s.  A 16-byte read is served 16 lanes
// at a time, but not 16 neighbours: lanes 0-3, 12-15 and 20-27 go together.  So
// the 64-byte rows of one segment (four to a 256-byte line of banks) and the
// middle ones of the next segment have to fall on different slots, which the
// plain s ^ (r / 4) does not give (4 conflict cycles a read with it; here 0.1 to 0.2
// over all of the kernel's LDS instructions, y's way out among them).
template <int ROW_B>
EM_DEV int swz(int r, int s) { return ROW_B == 128 ? s ^ ((r >> 1) & 7) : s ^ (-(r >> 2) & 3); }

}  // namespace

template <int FMT, int BT, int BN>
__global__ void __launch_bounds__(512)
mxp_gemm(MxProduct a) {
    using C = GemmCfg<FMT, BT, BN>;
    constexpr int NI = C::NI, NJ = C::NJ, XB = C::XB;
    __shared__ __attribute__((aligned(16))) uint8_t lds[C::STAGES * C::STAGE];
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;

    // tile order: XCD x = blockIdx % 8 takes a contiguous part of the tiles,
    // which run down groups of 8 row tiles before moving a column tile on, so
    // that the tiles of one XCD in flight share their x and W rows in its L2
    const int nn = (a.N + C::BN - 1) / C::BN;
    int tn = 0;
    const RowTile t = row_tile<BT>(a.offsets, a.M, a.R, [&](int rows) {
        const int total = rows * nn, per = (total + 7) >> 3, i = blockIdx.x >> 3;
        const int b = (blockIdx.x & 7) * per + i;
        if (i >= per || b >= total) return -1;
        const int grp = b / (8 * nn), left = min(8, rows - 8 * grp), in = b - grp * 8 * nn;
        tn = in / left;
        return 8 * grp + in % left;
    });
    if (t.r1 == 0) return;
    const int n0 = tn * C::BN, nrow = t.r1 - t.r0;

    // ---- load sources (one per wave instruction of a stage; where the pieces run
    // out before the waves, the first ones are loaded again)
    const int steps = a.K / kMxStep;
    const uint8_t* xsrc[C::X_INSTR];                    // x rows may lie anywhere in a workspace of any size
    uint32_t woff[C::W_INSTR], soff[C::S_INSTR];
    constexpr int XR = 1024 / XB;                       // x rows per load
#pragma unroll
    for (int q = 0; q < C::X_INSTR; ++q) {
        const int tr = XR * ((C::X_INSTR * wv + q) % C::X_P) + lane / (XB / 16);
        xsrc[q] = a.xq + (int64_t)xq_row(a, t.r0 + min(tr, nrow - 1)) * (a.K * XB / 128)
                  + 16 * swz<XB>(tr, lane % (XB / 16));
    }
    const uint8_t* wbase = a.codes + ((int64_t)t.m * a.N + n0) * (a.K / 2);
    const uint8_t* wsbase = a.scales + ((int64_t)t.m * steps * a.N + n0) * 4;
#pragma unroll
    for (int q = 0; q < C::W_INSTR; ++q) {
        const int tr = 16 * (C::W_INSTR * wv + q) + lane / 4;
        woff[q] = min(tr, a.N - 1 - n0) * (a.K / 2) + 16 * swz<64>(tr, lane % 4);
    }
    // scale words of 64 rows a piece: W's, then x's
#pragma unroll
    for (int q = 0; q < C::S_INSTR; ++q) {
        const int piece = (C::S_INSTR * wv + q) % C::S_P, tr = 64 * piece + lane;
        soff[q] = piece < C::BN / 64 ? 4 * min(tr, a.N - 1 - n0)
                                     : 4 * xq_row(a, t.r0 + min(tr - C::BN, nrow - 1));
    }
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    auto fetch = [&](int st, int to, int u) {           // load u of step st's, into the stage of step `to`
        const uint32_t stage = __builtin_amdgcn_readfirstlane(base + (to % C::STAGES) * C::STAGE);
        if (u < C::X_INSTR) {
            lds_load16(xsrc[u] + (int64_t)st * XB, stage + 1024 * ((C::X_INSTR * wv + u) % C::X_P));
        } else if (u < C::X_INSTR + C::W_INSTR) {
            const int q = u - C::X_INSTR;
            lds_load16(wbase + st * 64, woff[q], stage + C::X_B + 1024 * (C::W_INSTR * wv + q));
        } else {
            const int q = u - C::X_INSTR - C::W_INSTR, piece = (C::S_INSTR * wv + q) % C::S_P;
            const uint8_t* src = piece < C::BN / 64 ? wsbase + (int64_t)st * a.N * 4 : a.xs + (int64_t)st * a.xrows * 4;
            lds_load4(src, soff[q], stage + C::X_B + C::W_B + 256 * piece);
        }
    };

    const int wn = wv / C::WT, wt = wv % C::WT;
    floatx4 acc[NI][NJ];
#pragma unroll
    for (int p = 0; p < NI; ++p)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[p][j] = zero4();

    // Fragments of x are read before their step begins, those of W one column
    // subtile ahead, so that the matrix cores have operands from a step's first
    // cycle and the LDS reads run under the products.
    typename XOp<FMT>::type xf[2][NJ];
    int xs[2][NJ];
    uint4 wf[2];
    int wsc[2];
    // this lane's places in a subtile's rows (16 rows on, the swizzle is the same)
    const int xlo = m * XB + 16 * swz<XB>(m, g), xhi = m * XB + 16 * swz<XB>(m, 4 + g), wlo = m * 64 + 16 * swz<64>(m, g);
    const int sc = 4 * m + g;
    auto stage_of = [&](int st) -> const uint8_t* { return lds + (st % C::STAGES) * C::STAGE; };
    auto read_x = [&](auto set, const uint8_t* X, int u) {            // unit u of the XU reads of a step
        constexpr int f = decltype(set)::value;
        const int j = FMT == kMxFp8 ? u >> 1 : u, h = FMT == kMxFp8 ? u & 1 : 0, r = 16 * (NJ * wt + j);
        const uint4 v = ldg16(X + r * XB + (h ? xhi : xlo));
        auto& o = xf[f][j];
        o[4 * h] = (int)v.x; o[4 * h + 1] = (int)v.y; o[4 * h + 2] = (int)v.z; o[4 * h + 3] = (int)v.w;
        if (h == 0) xs[f][j] = X[C::X_B + C::W_B + C::WS_B + 4 * r + sc];
    };
    auto read_w = [&](const uint8_t* X, int p) {
        const int r = 16 * (NI * wn + p);
        wf[p & 1] = ldg16(X + C::X_B + r * 64 + wlo);
        wsc[p & 1] = X[C::X_B + C::W_B + 4 * r + sc];
    };
    constexpr int XU = FMT == kMxFp8 ? 2 * NJ : NJ;
    // Of the next step, x and the first of W are read from column subtile MID on,
    // behind a barrier that knows its stage landed.  With three stages a second
    // barrier, at the step's start, frees the stage of the step before for the loads
    // right away and gives them almost two steps; with four, the one at the
    // start does both and they have two.  Past the last step the loads repeat it
    // into stages that nothing reads: no branch in the loop (with one, the
    // accumulators are copied at its join).
    constexpr int MID = C::STAGES == 3 ? NI * 3 / 4 : 0;
    auto step = [&](int st, auto set) {
        constexpr int f = decltype(set)::value;
        const uint8_t* X = stage_of(st);
        const uint8_t* Xn = stage_of(st + 1);                         // past the last step: read, never used
        const int ahead = min(st + C::STAGES - 1, steps - 1);
        if constexpr (MID > 0) {
            lds_barrier();
#pragma unroll
            for (int u = 0; u < C::LOADS; ++u) fetch(ahead, st + C::STAGES - 1, u);
        }
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            if (p == MID) wait_loads_barrier<MID ? C::LOADS : C::LOADS * (C::STAGES - 3)>();
            read_w(p + 1 < NI ? X : Xn, (p + 1) % NI);
            if (p >= MID) {
#pragma unroll
                for (int u = (p - MID) * XU / (NI - MID); u < (p - MID + 1) * XU / (NI - MID); ++u) read_x(Set<1 - f>{}, Xn, u);
            }
            if constexpr (MID == 0) {                                 // spread between the products, which they would hold up together
#pragma unroll
                for (int u = p * C::LOADS / NI; u < (p + 1) * C::LOADS / NI; ++u) fetch(ahead, st + C::STAGES - 1, u);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const auto& x = xf[f][j];
                i32x8 x8 = {x[0], x[1], x[2], x[3], 0, 0, 0, 0};
                if constexpr (FMT == kMxFp8) x8 = x;
                acc[p][j] = mfma_mx<FMT>(wf[p & 1], wsc[p & 1], x8, xs[f][j], acc[p][j]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int st = 0; st < C::STAGES - 1; ++st)
#pragma unroll
        for (int u = 0; u < C::LOADS; ++u) fetch(min(st, steps - 1), st, u);
    wait_loads_barrier<C::LOADS * (C::STAGES - 2)>();
#pragma unroll
    for (int u = 0; u < XU; ++u) read_x(Set<0>{}, stage_of(0), u);
    read_w(stage_of(0), 0);
    int st = 0;
    for (; st + 1 < steps; st += 2) {
        step(st, Set<0>{});
        step(st + 1, Set<1>{});
    }
    if (st < steps) step(st, Set<0>{});
    wait_loads_barrier<0>();                                          // nothing more lands in the stages

    // ---- y: lane (g, m) holds columns 4 g .. 4 g + 3 of each column subtile, x row m.
    // Through the LDS, so that a wave stores whole 256- or 128-byte row segments: 32-byte
    // pieces leave the L2 half-written lines to merge.  Aligned ones go past it, since the
    // lines that it keeps cost the next kernel their write-back; rows at odd places and
    // the last columns in words or halves (11845 rows of 4222 columns, K = 384: 117 us
    // with 2-byte stores from the accumulators, 60 here).
    constexpr int RB = NI * 32, RSTR = RB + 16;              // bytes of a wave's row, their LDS stride
    uint8_t* o = lds + wv * (16 * NJ * RSTR);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int r = t.r0 + 16 * (NJ * wt + j) + m;
        const bool live = r < t.r1 && x_row(a, r) >= 0;
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            const floatx4 v = live ? acc[p][j] : zero4();
            const f32x2 lo = {v.x, v.y}, hi = {v.z, v.w};
            *reinterpret_cast<uint2*>(o + (16 * j + m) * RSTR + 32 * p + 8 * g) =
                make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2)),
                           __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2)));
        }
    }
    __builtin_amdgcn_wave_barrier();                         // one wave's LDS accesses complete in order
    asm volatile("" ::: "memory");
    const int r0 = t.r0 + 16 * NJ * wt, c0 = n0 + 16 * NI * wn, left = a.N - c0;   // the wave's rows, columns and those that exist
    if (a.vec == 3 && left >= 16 * NI) {
        constexpr int LPR = RB / 16, RPI = 64 / LPR;         // lanes per row, rows per store
#pragma unroll
        for (int i = 0; i < 16 * NJ / RPI; ++i) {
            const int tr = RPI * i + lane / LPR;
            if (r0 + tr >= t.r1) continue;
            const u32x4 v = *reinterpret_cast<const u32x4*>(o + tr * RSTR + 16 * (lane % LPR));
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(a.y + (int64_t)(r0 + tr) * a.y_stride + c0 + 8 * (lane % LPR)));
        }
    } else if (a.vec) {
        constexpr int LPR = RB / 4, RPI = 64 / LPR;
        const int n = 2 * (lane % LPR);
#pragma unroll 8
        for (int i = 0; i < 16 * NJ / RPI; ++i) {
            const int tr = RPI * i + lane / LPR;
            if (r0 + tr >= t.r1 || n >= left) continue;
            const uint32_t v = *reinterpret_cast<const uint32_t*>(o + tr * RSTR + 2 * n);
            uint16_t* p = a.y + (int64_t)(r0 + tr) * a.y_stride + c0 + n;
            if (n + 1 < left) *reinterpret_cast<uint32_t*>(p) = v;
            else *p = (uint16_t)v;
        }
    } else {
#pragma unroll 8
        for (int i = 0; i < 16 * NJ * (RB / 128); ++i) {
            const int tr = i / (RB / 128), n = lane + 64 * (i % (RB / 128));
            if (r0 + tr < t.r1 && n < left) a.y[(int64_t)(r0 + tr) * a.y_stride + c0 + n] = *reinterpret_cast<const uint16_t*>(o + tr * RSTR + 2 * n);
        }
    }
}

// ------------------------------------------------------------------ host side ----
namespace {

// Row tiles of BT rows that R rows in M matrices can make at most.
int64_t max_row_tiles(const MxProduct& a, int BT) {
    return a.offsets ? a.R / BT + (a.M < a.R ? a.M : a.R) : (a.R + BT - 1) / BT;
}

template <int NS, int NC, bool FUSED>
hipError_t launch_stream_nc(const MxProduct& a, hipStream_t s) {
    const dim3 grid((a.N + 16 * NC - 1) / (16 * NC), (unsigned)max_row_tiles(a, 16 * NS));
    prof_begin(s);
    if (a.fmt == kMxFp4) mxp_stream<kMxFp4, NS, NC, FUSED><<<grid, 256, 0, s>>>(a);
    else mxp_stream<kMxFp8, NS, NC, FUSED><<<grid, 256, 0, s>>>(a);
    prof_end(s, "mxp_stream");
    return hipGetLastError();
}

// 32 columns a workgroup, 16 where that leaves half of the compute units idle.
template <int NS, bool FUSED>
hipError_t launch_stream(const MxProduct& a, hipStream_t s) {
    if constexpr (NS == 1)
        if (max_row_tiles(a, 16) * ((a.N + 31) / 32) <= 128) return launch_stream_nc<1, 1, FUSED>(a, s);
    return launch_stream_nc<NS, 2, FUSED>(a, s);
}

// How many times 16 rows of a matrix mxp_stream takes at once (0: not mxp_stream).
// Measured at K = 4096 and 8192, FP8 (us a call, streams of 16 / 32 / 64 rows
// against 64-row tiles): one matrix of 8192 columns 32 rows 14.2 / 12.3 / 12.1 /
// 16.6, 64 rows 23.6 / 18.4 / 16.6 / 16.9, 128 rows 41 / 31 / 27 / 18; 1024
// columns 128 rows 10.8 / 11.9 / 15.7 / 17.4, 1024 rows 46 / 35 / 31 / 20: the
// fewest rows that make one workgroup a CU, and tiles where 64 do not.  512
// matrices of 128 columns, 64 rows in all 11.9 against 23, 256 rows 24 / 24; 64 of
// 1024 columns, 64 rows 28 / 25, 512 rows 42 / 27: tiles once they number about
// half of the CUs, since a tile's loads keep more of a matrix in flight.
int stream_rows(const MxProduct& a) {
    const int live = !a.offsets ? 1 : a.M < a.R ? a.M : a.R;       // matrices that the rows spread over
    const int64_t avg = ((int64_t)a.R + live - 1) / live, cols = (a.N + 31) / 32;
    if (max_row_tiles(a, 64) * a.N / 256 >= 130) return 0;
    for (int ns = 1; ns <= 4; ns *= 2)
        if (max_row_tiles(a, 16 * ns) * cols <= 256 || (avg <= 16 * ns && (a.offsets || ns == 1))) return ns;
    return 0;
}

// Whether mxp_stream's workgroups round the x rows that they need, which spares a
// launch of 3 to 4 us, but costs each of them 0.25 us per row and 4096 of K (the
// conversions): taken while a matrix's average rows times K are at most 16 x 4096.
// Measured (us a call, rounded there / before it, FP8): one matrix of 8192 x 4096
// 1 row 7.6 / 10.4, 16 rows 10.4 / 10.8; 4096 x 8192 8 rows 10.7 / 11.0, 16 rows
// 15.1 / 12.1; 1024 x 32768 1 row 12.7 / 18.4, 4 rows 20 / 21, 16 rows 47 / 29;
// 512 of 128 x 4096 80 rows 9.4 / 14.1.
bool rounds_in_stream(const MxProduct& a) {
    const int live = !a.offsets ? 1 : a.M < a.R ? a.M : a.R;
    return ((int64_t)a.R + live - 1) / live * a.K <= 16 * 4096;
}

// Rows of mxp_gemm's tiles.  A product takes as many rounds of tiles as 256 CUs
// need, each as long as a tile: measured at K = 4096, tiles of 64 / 128 / 192 / 256
// rows x 256 columns 18 / 27 / 36 / 44 us in FP4 and 20 / 31 / 45 / 59 in FP8; of 64 /
// 128 / 256 rows x 128 columns, for matrices of no more, 12 / 17.5 / 26 and 13.5 / 20 /
// 34.  The rows with the least rounds times length are taken, at 256 columns, or 128
// for matrices of no more (narrow tiles of wider matrices are not weighed); each matrix
// with rows is counted half a tile more.  (8192 columns, K = 4096, FP4, us a call by
// rows: 1000 40 / 30 / 32 / 35, 1536 58 / 49 / 39 / 41, 2048 76 / 57 / 62 / 48;
// 8 matrices of 4096 x 8192 in FP8, 5001 rows: 235 / 180 / 183 / 207; 512 of 128 x
// 4096, 20480 rows: 53 with 256 columns, 43 with 128.)
int tile_rows(const MxProduct& a) {
    static constexpr int kRows[4] = {64, 128, 192, 256};
    static constexpr int kWide[2][4] = {{36, 54, 72, 88}, {40, 62, 90, 118}};       // half microseconds
    static constexpr int kNarrow[2][4] = {{24, 35, 0, 52}, {27, 40, 0, 68}};
    const int live = !a.offsets ? 0 : a.M < a.R ? a.M : a.R;
    const int64_t cols = (a.N + 255) / 256;
    const int* length = (a.N <= 128 ? kNarrow : kWide)[a.fmt == kMxFp8];
    int64_t best = 0;
    int rows = 0;
    for (int i = 0; i < 4; ++i) {
        const int bt = kRows[i];
        const int64_t halves = a.offsets ? 2ll * a.R / bt + live : 2ll * ((a.R + bt - 1) / bt);
        const int64_t cost = (halves * cols + 511) / 512 * length[i];
        if (cost && (!rows || cost < best)) {
            best = cost;
            rows = bt;
        }
    }
    return rows;
}

template <int BT, int BN>
hipError_t launch_gemm(const MxProduct& a, hipStream_t s) {
    const int64_t tiles = max_row_tiles(a, BT) * ((a.N + BN - 1) / BN);
    prof_begin(s);
    if (a.fmt == kMxFp4) mxp_gemm<kMxFp4, BT, BN><<<(unsigned)((tiles + 7) & ~7ll), 512, 0, s>>>(a);
    else mxp_gemm<kMxFp8, BT, BN><<<(unsigned)((tiles + 7) & ~7ll), 512, 0, s>>>(a);
    prof_end(s, "mxp_gemm");
    return hipGetLastError();
}

}  // namespace

// Rows of x that the workspace holds: of a longer x only those that y's rows read
// (rows that several y rows share are rounded once).
static int x_rows(const MxProduct& a) { return a.R < a.T ? a.R : a.T; }

size_t mx_product_ws_bytes(const MxProduct& a) {
    const size_t row = (size_t)a.K * (a.fmt == kMxFp4 ? 1 : 2) / 2 + (size_t)a.K / 32;
    return ((size_t)x_rows(a) * row + 511) & ~(size_t)255;
}

// The product from x in the workspace, or from codes that the caller has.
static hipError_t launch_coded(const MxProduct& a, int ns, hipStream_t s) {
    switch (ns) {
        case 1: return launch_stream<1, false>(a, s);
        case 2: return launch_stream<2, false>(a, s);
        case 4: return launch_stream<4, false>(a, s);
        default: break;
    }
    const int rows_a_tile = tile_rows(a);
    if (a.N <= 128) {
        switch (rows_a_tile) {
            case 64: return launch_gemm<64, 128>(a, s);
            case 128: return launch_gemm<128, 128>(a, s);
            default: return launch_gemm<256, 128>(a, s);
        }
    }
    switch (rows_a_tile) {
        case 64: return launch_gemm<64, 256>(a, s);
        case 128: return launch_gemm<128, 256>(a, s);
        case 192: return launch_gemm<192, 256>(a, s);
        default: return launch_gemm<256, 256>(a, s);
    }
}

hipError_t launch_mx_product(MxProduct a, void* ws, hipStream_t s) {
    const int ns = stream_rows(a);
    if (ns == 1 && rounds_in_stream(a)) return launch_stream<1, true>(a, s);
    a.xrows = x_rows(a);
    a.gathered = a.row_src && a.xrows < a.T;
    a.xq = static_cast<uint8_t*>(ws);
    a.xs = a.xq + (((size_t)a.xrows * a.K / (a.fmt == kMxFp4 ? 2 : 1) + 255) & ~(size_t)255);
    const MxRows rows{a.xrows, a.xrows, a.K, a.x_stride, a.fmt, 0, a.gathered ? a.row_src : nullptr, a.T};
    const hipError_t e = launch_mx_quantize(rows, a.x, const_cast<uint8_t*>(a.xq), const_cast<uint8_t*>(a.xs), s);
    if (e != hipSuccess) return e;
    return launch_coded(a, ns, s);
}

hipError_t launch_mx_product_coded(MxProduct a, hipStream_t s) {
    a.xrows = a.T;
    a.gathered = 0;
    return launch_coded(a, stream_rows(a), s);
}

}  // namespace em
