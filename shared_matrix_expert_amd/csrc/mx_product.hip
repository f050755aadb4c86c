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
//               LDS-tiled, bound by the matrix cores and the LDS reads.
#include "mx_format.h"
#include "operators.h"

namespace em {

namespace {

EM_DEV uint4 ldg16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

template <int FMT> constexpr int mx_code() { return FMT == kMxFp4 ? 4 : 0; }   // the instruction's format field

// acc += W (E2M1) . x (FMT) over 128 elements of K.
template <int FMT>
EM_DEV floatx4 mfma_mx(const uint4& w, int ws, const i32x8& x, int xs, const floatx4& acc) {
    const i32x8 a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, acc, 4, mx_code<FMT>(), 0, ws, 0, xs);
}

// ---- rows ------------------------------------------------------------------
// A row tile: rows [r0, r1) of y, all of matrix m.  Row tiles are numbered
// matrix by matrix; `total` is their count, r1 = 0 marks no tile.
struct RowTile { int m, r0, r1, total; };

// The row tile of this workgroup among tiles of BT rows: pick(total) names it,
// or is negative for none.  With offsets (device memory) every wave counts the
// tiles itself: each lane those of PER neighbouring matrices, then a scan over
// the lanes: one round of loads, against a chain of dependent ones in a binary
// search or a launch of its own.  Offsets outside 0..R or descending are
// clamped, so that no tile leaves y.
template <int BT, int PER, class Pick>
EM_DEV RowTile find_tile(const int32_t* __restrict__ offsets, int M, int R, Pick pick) {
    const int lane = lane_id();
    int b[PER + 1];
#pragma unroll
    for (int i = 0; i <= PER; ++i) b[i] = offsets[min(lane * PER + i, M)];
    int lo[PER], hi[PER], at[PER], mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {                   // past M both bounds are offsets[M]: no rows
        lo[i] = min(max(b[i], 0), R);
        hi[i] = min(max(b[i + 1], lo[i]), R);
        at[i] = mine;
        mine += (hi[i] - lo[i] + BT - 1) / BT;
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(sum, o, 64);
        if (lane >= o) sum += v;
    }
    RowTile t{0, 0, 0, __builtin_amdgcn_readlane(sum, 63)};
    const int rt = pick(t.total);
    if (rt < 0 || rt >= t.total) return t;
    const int own = __ffsll((long long)__ballot(sum > rt)) - 1;   // the lane whose tiles hold rt
    const int in = rt - __builtin_amdgcn_readlane(sum - mine, own);
    int mi = 0, first = 0, l = 0, h = 0;              // its last matrix with rows whose first tile is at or before it
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (at[i] <= in && hi[i] > lo[i]) { mi = lane * PER + i; first = at[i]; l = lo[i]; h = hi[i]; }
    t.m = __builtin_amdgcn_readlane(mi, own);
    t.r0 = __builtin_amdgcn_readlane(l, own) + (in - __builtin_amdgcn_readlane(first, own)) * BT;
    t.r1 = min(__builtin_amdgcn_readlane(h, own), t.r0 + BT);
    return t;
}

template <int BT, class Pick>
EM_DEV RowTile row_tile(const int32_t* __restrict__ offsets, int M, int R, Pick pick) {
    if (offsets) return M <= 64 ? find_tile<BT, 1>(offsets, M, R, pick) : find_tile<BT, 16>(offsets, M, R, pick);
    RowTile t{0, 0, 0, (R + BT - 1) / BT};
    const int rt = pick(t.total);
    if (rt < 0 || rt >= t.total) return t;
    t.r0 = rt * BT;
    t.r1 = min(R, t.r0 + BT);
    return t;
}

// x row of y row r, -1 where row_src names none.
EM_DEV int x_row(const MxProduct& a, int r) {
    if (!a.row_src) return r;
    const int s = a.row_src[r];
    return (unsigned)s < (unsigned)a.T ? s : -1;
}

// Four consecutive columns of a y row.
EM_DEV void store4(const MxProduct& a, int64_t r, int n, const floatx4& v) {
    uint16_t* p = a.y + r * a.y_stride + n;
    const f32x2 lo = {v.x, v.y}, hi = {v.z, v.w};
    const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2));
    const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2));
    if (a.vec && n + 4 <= a.N) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w0, w1);
        return;
    }
    if (n < a.N) p[0] = (uint16_t)w0;
    if (n + 1 < a.N) p[1] = (uint16_t)(w0 >> 16);
    if (n + 2 < a.N) p[2] = (uint16_t)w1;
    if (n + 3 < a.N) p[3] = (uint16_t)(w1 >> 16);
}

// ---- x rounded in registers -------------------------------------------------
// One K step of an x row as an operand: the lane's raw bf16 elements in v (FP4:
// its block's 32; FP8: K 16 g .. + 15 and 64 + 16 g .. + 15), the codes and this
// lane's scale byte out.
EM_DEV const uint16_t* x_piece(const uint16_t* row, int g, int h, int fmt) {
    return row + (fmt == kMxFp4 ? 32 * g + 16 * h : 64 * h + 16 * g);
}

template <int FMT>
EM_DEV void round_x(const uint4 (&v)[4], i32x8& q, int& xs) {
    if constexpr (FMT == kMxFp4) {
        const uint32_t a = max(max(amax8_bf16(v[0]), amax8_bf16(v[1])), max(amax8_bf16(v[2]), amax8_bf16(v[3])));
        xs = e8m0_of<FMT>(a);
        const bool bad = xs == 255;
        const float sc = e8m0_f32(bad ? 127 : xs);
        const i32x8 z = {0, 0, 0, 0, 0, 0, 0, 0};
        const i32x8 c = {(int)fp4x8_bf16(v[0], sc), (int)fp4x8_bf16(v[1], sc), (int)fp4x8_bf16(v[2], sc),
                         (int)fp4x8_bf16(v[3], sc), 0, 0, 0, 0};
        q = bad ? z : c;
    } else {
        // the lanes 2 c and 2 c + 1 of a row share block c (first half of the
        // codes) and block 2 + c (second half)
        uint32_t a0 = max(amax8_bf16(v[0]), amax8_bf16(v[1]));
        uint32_t a1 = max(amax8_bf16(v[2]), amax8_bf16(v[3]));
        uint32_t both = a0 | (a1 << 16);
        both = max_u16x2(both, (uint32_t)__shfl_xor((int)both, 16, 64));
        const int X0 = e8m0_of<FMT>(both & 0xFFFFu), X1 = e8m0_of<FMT>(both >> 16);
        const int l = lane_id();
        // block g's byte: held by lanes of group 2 (g & 1) as X0 (g < 2) or X1
        const int other = __shfl(X0 | (X1 << 8), (l & 15) + 32 * ((l >> 4) & 1), 64);
        xs = (l & 32) ? other >> 8 : other & 255;
        const bool b0 = X0 == 255, b1 = X1 == 255;
        const float s0 = e8m0_f32(b0 ? 127 : X0), s1 = e8m0_f32(b1 ? 127 : X1);
        const uint32_t l0 = e4m3_limit(b0 ? 127 : X0), l1 = e4m3_limit(b1 ? 127 : X1);
        const uint32_t c[8] = {fp8x4_bf16(v[0].x, v[0].y, s0, l0), fp8x4_bf16(v[0].z, v[0].w, s0, l0),
                               fp8x4_bf16(v[1].x, v[1].y, s0, l0), fp8x4_bf16(v[1].z, v[1].w, s0, l0),
                               fp8x4_bf16(v[2].x, v[2].y, s1, l1), fp8x4_bf16(v[2].z, v[2].w, s1, l1),
                               fp8x4_bf16(v[3].x, v[3].y, s1, l1), fp8x4_bf16(v[3].z, v[3].w, s1, l1)};
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = (i < 4 ? b0 : b1) ? 0 : (int)c[i];
    }
}

}  // namespace

// ------------------------------------------------------------------ few rows -----
// A workgroup takes one row tile (16 NS rows of one matrix) and 16 NC columns;
// its four waves split K into contiguous quarters and their partial sums are
// added through LDS in wave order.  Weights and x run DEPTH steps ahead in
// registers.
template <int FMT, int NS, int NC>
__global__ void __launch_bounds__(256)
mxp_stream(MxProduct a) {
    constexpr int DEPTH = NS == 1 ? 4 : 2;
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
    const uint16_t* xp[NS];
    bool live[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const int r = t.r0 + 16 * s + m;
        const int src = r < t.r1 ? x_row(a, r) : -1;
        live[s] = src >= 0;
        xp[s] = a.x + (int64_t)max(src, 0) * a.x_stride;
    }
    floatx4 acc[NS][NC];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[s][c] = zero4();

    uint4 w[DEPTH][NC];
    int ws[DEPTH][NC];
    uint4 xv[DEPTH][NS][4];
    auto load = [&](int d, int st) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            w[d][c] = ldg16(wp[c] + (int64_t)st * (kMxStep / 2));
            ws[d][c] = sp[c][(int64_t)st * a.N * 4];
        }
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint16_t* p = x_piece(xp[s] + (int64_t)st * kMxStep, g, h, FMT);
                xv[d][s][2 * h] = ldg16(p);
                xv[d][s][2 * h + 1] = ldg16(p + 8);
            }
    };
    if (s0 < s1) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(d, min(s0 + d, s1 - 1));
        for (int st = s0; st < s1; st += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (st + d < s1) {
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        i32x8 q;
                        int xs;
                        round_x<FMT>(xv[d][s], q, xs);
#pragma unroll
                        for (int c = 0; c < NC; ++c) acc[s][c] = mfma_mx<FMT>(w[d][c], ws[d][c], q, xs, acc[s][c]);
                    }
                    if (st + d + DEPTH < s1) load(d, st + d + DEPTH);
                }
            }
        }
    }
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
        if (r < t.r1) store4(a, r, n0 + 16 * c + 4 * g, live[s] ? v : zero4());
    }
}

// ------------------------------------------------------------------ many rows ----
// A workgroup of 8 waves takes BT rows x 256 columns, WN x (8 / WN) waves of
// (256 / WN) columns x (BT WN / 8) rows.  Each K step's codes and scale words
// arrive by direct global -> LDS loads, two steps ahead in three stages; every
// wave issues the same number of loads a step, so one counted wait covers them.
// A code row is 64 (E2M1) or 128 (E4M3) bytes; its 16-byte segments are stored
// XOR-swizzled by the row, so that the 16 rows of a fragment read fall on
// distinct bank groups.
namespace {

template <int FMT, int BT_>
struct GemmCfg {
    static constexpr int BT = BT_, BN = 256, TH = 512;
    static constexpr int WN = BT == 256 ? 2 : 4, WT = 8 / WN;
    static constexpr int NI = BN / WN / 16, NJ = BT / WT / 16;     // column and row subtiles of a wave
    static constexpr int XB = FMT == kMxFp4 ? 64 : 128;            // bytes of an x row per step
    static constexpr int X_B = BT * XB, W_B = BN * 64, XS_B = BT * 4, WS_B = BN * 4;
    static constexpr int STAGE = X_B + W_B + XS_B + WS_B, STAGES = 3;
    static constexpr int X_INSTR = (X_B / 1024 + 7) / 8;           // 1 KB loads of x per wave per stage
    static constexpr int W_INSTR = W_B / 1024 / 8;
    static constexpr int LOADS = X_INSTR + W_INSTR + 1;
};

// Direct global -> LDS load of 16 (or 4) bytes a lane to `dst` + 16 (4) * lane.
// Written out because the compiler, which cannot tell the stages of the ring
// apart, waits for every such load of its own before the next LDS read; these
// are counted by wait_loads instead.  They have no register output.
EM_DEV void dma16(const uint8_t* src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "s"(dst) : "memory", "m0");
}
EM_DEV void dma4(const uint8_t* src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(src), "s"(dst) : "memory", "m0");
}

// At most N of this wave's loads in flight, its LDS reads done; then the barrier.
template <int N>
EM_DEV void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// Segment slot of row r's 16-byte segment s.
template <int ROW_B>
EM_DEV int swz(int r, int s) { return ROW_B == 128 ? s ^ ((r >> 1) & 7) : s ^ ((r >> 2) & 3); }

}  // namespace

template <int FMT, int BT>
__global__ void __launch_bounds__(512)
mxp_gemm(MxProduct a) {
    using C = GemmCfg<FMT, BT>;
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

    // ---- load sources (one per wave instruction of a stage)
    const int steps = a.K / kMxStep;
    const uint8_t* xsrc[C::X_INSTR];
    const uint8_t* wsrc[C::W_INSTR];
    int xdst[C::X_INSTR];
    constexpr int XR = 1024 / XB;                       // x rows per load
#pragma unroll
    for (int q = 0; q < C::X_INSTR; ++q) {
        const int piece = (C::X_INSTR * wv + q) % (C::X_B / 1024);   // a tile of fewer pieces than waves: loaded twice
        const int tr = XR * piece + lane / (XB / 16), slot = lane % (XB / 16);
        const int r = t.r0 + min(tr, nrow - 1);
        xsrc[q] = a.xq + (int64_t)max(x_row(a, r), 0) * (a.K * XB / 128) + 16 * swz<XB>(tr, slot);
        xdst[q] = piece * 1024;
    }
    const uint8_t* wm = a.codes + (int64_t)t.m * a.N * (a.K / 2);
#pragma unroll
    for (int q = 0; q < C::W_INSTR; ++q) {
        const int tr = 16 * (C::W_INSTR * wv + q) + lane / 4;
        wsrc[q] = wm + (int64_t)min(n0 + tr, a.N - 1) * (a.K / 2) + 16 * swz<64>(tr, lane % 4);
    }
    // scale words: waves 0-3 the W rows', waves 4-7 the x rows' (BT = 64: the same 64)
    const uint8_t* ssrc;
    int64_t sstep;
    int sdst;
    if (wv < 4) {
        ssrc = a.scales + ((int64_t)t.m * steps * a.N + min(n0 + 64 * wv + lane, a.N - 1)) * 4;
        sstep = (int64_t)a.N * 4;
        sdst = C::X_B + C::W_B + 256 * wv;
    } else {
        const int p = (wv - 4) % (BT / 64);
        ssrc = a.xs + (int64_t)max(x_row(a, t.r0 + min(64 * p + lane, nrow - 1)), 0) * 4;
        sstep = (int64_t)a.T * 4;
        sdst = C::X_B + C::W_B + C::WS_B + 256 * p;
    }
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    auto fetch = [&](int st) {
        const uint32_t stage = __builtin_amdgcn_readfirstlane(base + (st % C::STAGES) * C::STAGE);
#pragma unroll
        for (int q = 0; q < C::X_INSTR; ++q) dma16(xsrc[q] + (int64_t)st * XB, stage + xdst[q]);
#pragma unroll
        for (int q = 0; q < C::W_INSTR; ++q) dma16(wsrc[q] + (int64_t)st * 64, stage + C::X_B + 1024 * (C::W_INSTR * wv + q));
        dma4(ssrc + st * sstep, stage + sdst);
    };

    const int wn = wv / C::WT, wt = wv % C::WT;
    floatx4 acc[NI][NJ];
#pragma unroll
    for (int p = 0; p < NI; ++p)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[p][j] = zero4();

    fetch(0);
    if (steps > 1) fetch(1);
    for (int st = 0; st < steps; ++st) {
        // step st has landed (the next one may be in flight), and every wave is
        // done with the stage that step st + 2 overwrites
        if (st + 1 < steps) wait_loads_barrier<C::LOADS>(); else wait_loads_barrier<0>();
        if (st + 2 < steps) fetch(st + 2);
        const uint8_t* X = lds + (st % C::STAGES) * C::STAGE;
        const uint8_t* W = X + C::X_B;
        const uint8_t* WS = W + C::W_B;
        const uint8_t* XS = WS + C::WS_B;
        i32x8 xf[NJ];
        int xs[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int r = 16 * (NJ * wt + j) + m;
            const uint4 lo = ldg16(X + r * XB + 16 * swz<XB>(r, g));
            uint4 hi = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (FMT == kMxFp8) hi = ldg16(X + r * XB + 16 * swz<XB>(r, 4 + g));
            xf[j] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
            xs[j] = XS[4 * r + g];
        }
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            const int r = 16 * (NI * wn + p) + m;
            const uint4 wf = ldg16(W + r * 64 + 16 * swz<64>(r, g));
            const int wsc = WS[4 * r + g];
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[p][j] = mfma_mx<FMT>(wf, wsc, xf[j], xs[j], acc[p][j]);
        }
    }

    // ---- y: lane (g, m) holds columns 4 g .. 4 g + 3 of each column subtile, x row m
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int r = t.r0 + 16 * (NJ * wt + j) + m;
        if (r >= t.r1) continue;
        const bool live = x_row(a, r) >= 0;
#pragma unroll
        for (int p = 0; p < NI; ++p) store4(a, r, n0 + 16 * (NI * wn + p) + 4 * g, live ? acc[p][j] : zero4());
    }
}

// ------------------------------------------------------------------ host side ----
namespace {

// Row tiles of BT rows that R rows in M matrices can make at most.
int64_t max_row_tiles(const MxProduct& a, int BT) {
    return a.offsets ? a.R / BT + (a.M < a.R ? a.M : a.R) : (a.R + BT - 1) / BT;
}

template <int NS>
hipError_t launch_stream(const MxProduct& a, hipStream_t s) {
    constexpr int NC = 2;
    const dim3 grid((a.N + 16 * NC - 1) / (16 * NC), (unsigned)max_row_tiles(a, 16 * NS));
    prof_begin(s);
    if (a.fmt == kMxFp4) mxp_stream<kMxFp4, NS, NC><<<grid, 256, 0, s>>>(a);
    else mxp_stream<kMxFp8, NS, NC><<<grid, 256, 0, s>>>(a);
    prof_end(s, "mxp_stream");
    return hipGetLastError();
}

template <int BT>
hipError_t launch_gemm(const MxProduct& a, hipStream_t s) {
    const int64_t tiles = max_row_tiles(a, BT) * ((a.N + 255) / 256);
    prof_begin(s);
    if (a.fmt == kMxFp4) mxp_gemm<kMxFp4, BT><<<(unsigned)((tiles + 7) & ~7ll), 512, 0, s>>>(a);
    else mxp_gemm<kMxFp8, BT><<<(unsigned)((tiles + 7) & ~7ll), 512, 0, s>>>(a);
    prof_end(s, "mxp_gemm");
    return hipGetLastError();
}

}  // namespace

size_t mx_product_ws_bytes(const MxProduct& a) {
    const size_t row = (size_t)a.K * (a.fmt == kMxFp4 ? 1 : 2) / 2 + (size_t)a.K / 32;
    return (a.T * row + 511) & ~(size_t)255;
}

hipError_t launch_mx_product(MxProduct a, void* ws, hipStream_t s) {
    const int live = a.offsets && a.M < a.R ? a.M : 1;      // matrices that the rows spread over
    const int64_t avg = ((int64_t)a.R + live - 1) / live;
    if (avg <= 64) return avg <= 16 ? launch_stream<1>(a, s) : avg <= 32 ? launch_stream<2>(a, s) : launch_stream<4>(a, s);
    a.xq = static_cast<uint8_t*>(ws);
    a.xs = a.xq + (((size_t)a.T * a.K / (a.fmt == kMxFp4 ? 2 : 1) + 255) & ~(size_t)255);
    const MxRows rows{a.T, a.T, a.K, a.x_stride, a.fmt, 0};
    const hipError_t e = launch_mx_quantize(rows, a.x, const_cast<uint8_t*>(a.xq), const_cast<uint8_t*>(a.xs), s);
    if (e != hipSuccess) return e;
    return avg >= 192 ? launch_gemm<256>(a, s) : launch_gemm<64>(a, s);
}

}  // namespace em
