// Products of token rows with bf16 matrices, grouped by matrix with ragged rows, and
// their gradients:
//   DP_Y    y[r][n]     = sum_k x[src(r)][k] W_m[n][k]       (m the matrix of row r)
//   DP_DX   dx[r][k]    = sum_n dy[r][n] W_m[n][k]           (or summed over a token's rows)
//   DP_DXT  dx[t][k]    = sum over token t's rows r of the same, in one sum over all matrices
//   DP_DW   dW_m[n][k]  = sum over m's rows r of dy[r][n] x[src(r)][k]
// All three are out[i][j] = sum_c P[i][c] Q[j][c].  An operand whose c lies along its
// rows comes from the LDS as it is; one whose c runs down the rows (W in dx, both in dW)
// is transposed on the way out of the LDS (ds_read_b64_tr_b16).  The matrix cores take
// Q as their row operand, so that a lane holds four neighbouring j of one i.
//
//   dp_stream  y of few rows a matrix: bound by the weight bytes.  Four waves split K and
//              stream W straight into operand registers.
//   dp_tile    everything else: LDS tiles by direct global -> LDS loads, counted by hand.
//   dp_join    slices of c, and the rows of a token, added in a fixed order (float32).
#include <type_traits>

#include "common.h"
#include "lds_load.h"
#include "operators.h"
#include "row_tile.h"

namespace em {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

EM_DEV uint4 ldg16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

EM_DEV uint32_t pack2(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

enum DpMode { DP_Y = 0, DP_DX = 1, DP_DW = 2, DP_DWG = 3, DP_DXT = 4 };   // DWG: dW with gathered x rows

// What lanes without an element read: rows and columns past an operand's end.
__device__ const uint4 dp_zero = {0u, 0u, 0u, 0u};

// x row of y row r, -1 where row_src names none.
EM_DEV int x_row(const DenseProduct& a, int r) {
    if (!a.row_src) return r;
    const int s = a.row_src[r];
    return (unsigned)s < (unsigned)a.T ? s : -1;
}

// Four neighbouring columns of an out row.
EM_DEV void store4(void* out, int f32, int64_t at, const floatx4& v) {
    if (f32) *reinterpret_cast<floatx4*>(static_cast<float*>(out) + at) = v;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
}

}  // namespace

// ------------------------------------------------------------------ few rows -----
// A workgroup takes one row tile (16 rows of one matrix) and 16 NC columns; its four
// waves split K into contiguous quarters, D steps of 32 ahead, and their partial sums
// are added through LDS in wave order.  Bound by W's bytes and by the latencies in front of
// them (offsets, the row list, x): 80 rows over 512 of 128 x 4096, 80 MB, 19.0 us; 8 rows
// through 8192 x 4096, 67 MB from the memory-side cache, 13.6 us, 4.9 TB/s.
template <int NC>
__global__ void __launch_bounds__(256)
dp_stream(DenseProduct a) {
    constexpr int D = 8;
    __shared__ __attribute__((aligned(16))) float red[4][NC][256];
    const RowTile t = row_tile<16>(a.offsets, a.M, a.R, [](int) { return (int)blockIdx.y; });
    if (t.r1 == 0) return;
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
    const int n0 = blockIdx.x * (16 * NC);
    const int steps = a.K / 32, rest = a.K % 32;
    const int s0 = steps * wv / 4, s1 = steps * (wv + 1) / 4;

    const uint16_t* wp[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) wp[c] = a.w + ((int64_t)t.m * a.N + min(n0 + 16 * c + m, a.N - 1)) * a.K + 8 * g;
    uint4 w[D][NC], x[D];
    auto load_w = [&](int d, int st) {
#pragma unroll
        for (int c = 0; c < NC; ++c) w[d][c] = ldg16(wp[c] + 32 * st);
    };
    if (s0 < s1) {
#pragma unroll
        for (int d = 0; d < D; ++d) load_w(d, min(s0 + d, s1 - 1));
    }
    const int src = x_row(a, min(t.r0 + m, t.r1 - 1));
    const uint16_t* xp = a.x + (int64_t)max(src, 0) * a.x_stride + 8 * g;
    floatx4 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = zero4();
    if (s0 < s1) {
#pragma unroll
        for (int d = 0; d < D; ++d) x[d] = ldg16(xp + 32 * min(s0 + d, s1 - 1));
    }
    auto run = [&](int st, auto more) {                       // D steps, without a branch but for the last ones
        constexpr bool MORE = decltype(more)::value;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (MORE || st + d < s1) {
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[c] = mfma_bf16(w[d][c], x[d], acc[c]);
                if constexpr (MORE) x[d] = ldg16(xp + 32 * min(st + d + D, s1 - 1));
                if constexpr (MORE) load_w(d, min(st + d + D, s1 - 1));
                __builtin_amdgcn_sched_barrier(0);            // loads complete in order: x asked for later would wait for W's
            }
        }
    };
    int st = s0;
    for (; st + D < s1; st += D) run(st, std::true_type{});
    if (st < s1) run(st, std::false_type{});
    if (rest && wv == 3) {                                    // the last 8, 16 or 24 of K: zeros past them on both sides
        const bool in = 8 * g < rest;
        const int off = in ? 32 * steps : -8 * g;             // else the row's first elements, not used
        const uint4 v = ldg16(xp + off), xr = in ? v : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint4 u = ldg16(wp[c] + off), wr = in ? u : make_uint4(0u, 0u, 0u, 0u);
            acc[c] = mfma_bf16(wr, xr, acc[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) *reinterpret_cast<floatx4*>(&red[wv][c][4 * lane]) = acc[c];
    __syncthreads();
    if (wv >= NC) return;                                     // column tile c is summed by wave c
    floatx4 v = *reinterpret_cast<const floatx4*>(&red[0][wv][4 * lane]);
#pragma unroll
    for (int q = 1; q < 4; ++q) v += *reinterpret_cast<const floatx4*>(&red[q][wv][4 * lane]);
    const int r = t.r0 + m, n = n0 + 16 * wv + 4 * g;
    if (r < t.r1 && n < a.N) store4(a.out, a.out_f32, (int64_t)r * a.out_stride + n, src >= 0 ? v : zero4());
}

// ------------------------------------------------------------------ LDS tiles ----
// A workgroup takes BT i x BN j of out in WT x WN waves, 64 of c a step.  P's and Q's
// tiles arrive by direct global -> LDS loads two steps ahead, every wave as many loads a
// step, counted by hand.  P's fragments of a step are read into registers during the
// step before, so P needs two stages and Q three.  Bound by the matrix cores: y of 8192^3
// 737 us, 1.49 PFLOP/s, dx 754, dW 816 (large library products of the three layouts 749, 854,
// 965); 5001 rows in 8 groups, 4096 x 8192, y 324, dx 310, dW 397.
//
// An operand with c along its rows: 128-byte rows (whole cache lines), 16-byte segments
// XOR-swizzled by the row (mx_product.hip's rule).  One with c down the rows: 64 rows of BX
// elements, segments swizzled in pairs by the row, so that the four rows that sixteen
// lanes read together fall on different banks.
//
// Rows and columns past an operand's end repeat its last ones, and what they give is not
// stored.  Past the end of c, and for an x row of dW that row_src does not name, lanes
// load zeros from dp_zero, so that nothing outside an operand meets a product; dy of such a
// row becomes zeros in the registers.
//
// A load takes a uniform base and a 32-bit lane offset (4 to 7% faster than a 64-bit
// address a lane at 8192^3); WIDE, for rows so far apart that the offsets do not fit,
// and the last steps of c take whole addresses.
namespace {

template <int MODE, int BT_, int BN_>
struct DpCfg {
    static constexpr bool DW = MODE == DP_DW || MODE == DP_DWG;
    static constexpr bool JT = MODE != DP_Y, IT = DW;                 // c runs down the rows of Q, of P
    static constexpr bool GATHER = MODE == DP_DWG;
    static constexpr int BT = BT_, BN = BN_;
    static constexpr int NW = BN == 256 || (BN == 128 && BT == 256) ? 8 : 4;
    static constexpr int WN = BN == 256 ? (BT == 256 ? 2 : 4) : BN == 128 ? 2 : (BT == 256 ? 1 : 2), WT = NW / WN;
    static constexpr int NI = BN / WN / 16, NJ = BT / WT / 16;        // j and i subtiles of a wave
    static constexpr int J_B = BN * 128, I_B = BT * 128;              // bytes of a stage of Q, of P
    static constexpr int JL = J_B / 1024 / NW, LOADS = JL + I_B / 1024 / NW;   // a wave's loads a step: Q's, then P's
    static constexpr int OUT_B = 16 * (NI * 64 + 16);                 // a wave's sixteen out rows on their way out
    static constexpr int TILES_B = 3 * J_B + 2 * I_B > NW * OUT_B ? 3 * J_B + 2 * I_B : NW * OUT_B;
    static constexpr int LDS_B = TILES_B + (GATHER ? 4 * 256 : 0);    // (GATHER) the x rows of four steps behind the tiles
    static_assert(LDS_B <= 160 * 1024, "");
};

template <int N>
EM_DEV void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" : : "n"(N) : "memory");
}
template <int N>
EM_DEV void wait_lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(%0)\n\ts_barrier" : : "n"(N) : "memory");
}

template <int I> struct Set { static constexpr int value = I; };

// Slot of 16-byte segment s: of row r of 128 bytes; of c row r of BX elements.
EM_DEV int swz_row(int r, int s) { return s ^ ((r >> 1) & 7); }
template <int BX>
EM_DEV int swz_col(int r, int s) { return s ^ 2 * ((r & 3) | (BX >= 128 ? (r >> 1) & 4 : 0)); }

// A tile of out: matrix mat, rows i0 .. i1 of P, from row j0 of Q; part z of the slices of c,
// which is clen long and starts at row c0 of dy and x (dW).
struct DpTile { int mat, i0, i1, j0, z, c0, clen; };

// Tile b of `total` tiles that XCD x = block % 8 takes neighbouring ones of; -1 past them.
EM_DEV int xcd_tile(int block, int total) {
    const int per = (total + 7) >> 3, at = block >> 3, b = (block & 7) * per + at;
    return at < per && b < total ? b : -1;
}

}  // namespace

template <int MODE, int BT, int BN, bool WIDE>
EM_DEV void dp_body(const DenseProduct& a, const DpTile& t, uint8_t* lds) {
    using C = DpCfg<MODE, BT, BN>;
    constexpr int NI = C::NI, NJ = C::NJ;
    const int lane = lane_id(), wv = wave_id(), g = lane >> 4, m = lane & 15;
    const int mat = t.mat, i0 = t.i0, i1 = t.i1, j0 = t.j0, z = t.z, c0 = t.c0, clen = t.clen;
    const int steps = (clen + 63) >> 6, whole_steps = clen >> 6;
    const int s0 = MODE == DP_DXT ? 0 : (int)((int64_t)steps * z / a.slices);
    const int s1 = MODE == DP_DXT ? z * a.pass_steps : (int)((int64_t)steps * (z + 1) / a.slices);   // (z: the tile's passes)

    // ---- loads.  Load u of a wave brings piece u NW + wv: Q's first, then P's.
    const uint16_t* wm = a.w + (int64_t)mat * a.N * a.K;          // (not with dW)
    // Uniform base at step 0, and bytes a step.
    const char* jbase = reinterpret_cast<const char*>(MODE == DP_Y ? wm + (int64_t)j0 * a.K : !C::DW ? wm : a.x + (int64_t)c0 * a.x_stride);
    const char* ibase = reinterpret_cast<const char*>(MODE == DP_Y ? (a.row_src ? a.x : a.x + (int64_t)i0 * a.x_stride) : a.dy + (int64_t)(MODE == DP_DX ? i0 : c0) * a.dy_stride);
    const int64_t jstride = !C::DW ? a.K : a.x_stride;            // of Q's rows, where c runs down them
    const int64_t jadv = C::JT ? 128 * jstride : 128, iadv = C::IT ? 128 * a.dy_stride : 128;
    // A lane's place in load u: its row of c and column, or its row and first c.
    auto place = [&](int u, int& row, int& col) {
        const bool isj = u < C::JL;
        const int piece = (isj ? u : u - C::JL) * C::NW + wv, bx = isj ? BN : BT;
        if (isj ? C::JT : C::IT) {
            row = piece * (512 / bx) + lane / (bx / 8);
            const int slot = lane % (bx / 8), at = 8 * (isj ? swz_col<BN>(row, slot) : swz_col<BT>(row, slot));
            col = min((isj ? j0 : i0) + at, (isj ? a.K : a.N) - 8);
        } else {
            row = piece * 8 + lane / 8;
            col = 8 * swz_row(row, lane % 8);
            row = isj ? min(row, a.N - 1 - j0) : min(row, i1 - 1 - i0);
            if (MODE == DP_Y && !isj && a.row_src) row = max(x_row(a, i0 + row), 0);   // the row of x
        }
    };
    // The first c of a lane's 16 bytes of load u within a step.
    auto c_of = [&](int u) {
        const bool isj = u < C::JL;
        const int piece = (isj ? u : u - C::JL) * C::NW + wv, bx = isj ? BN : BT;
        if (isj ? C::JT : C::IT) return piece * (512 / bx) + lane / (bx / 8);
        return 8 * swz_row(piece * 8 + lane / 8, lane % 8);
    };
    // Bytes of a lane from load u's base at its step.
    auto offset = [&](int u, int row, int col) -> int64_t {
        const bool isj = u < C::JL;
        const int64_t stride = isj ? (MODE == DP_Y ? (int64_t)a.K : jstride) : MODE == DP_Y ? a.x_stride : a.dy_stride;
        return 2 * (row * stride + col);
    };
    uint32_t off[C::LOADS];
    int64_t woff[WIDE ? C::LOADS : 1];
#pragma unroll
    for (int u = 0; u < C::LOADS; ++u) {
        if constexpr (MODE == DP_DXT) continue;                   // (made at each load)
        int row, col;
        place(u, row, col);
        if constexpr (WIDE) woff[u] = offset(u, C::GATHER && u < C::JL ? 0 : row, col);
        else off[u] = (uint32_t)offset(u, C::GATHER && u < C::JL ? 0 : row, col);
    }
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const char* zero = reinterpret_cast<const char*>(&dp_zero);
    // (GATHER) x rows of step st to their place in the LDS (every wave brings all of them),
    // and from there those of this wave's loads
    int from_row[C::GATHER ? C::JL : 1];
    // (GATHER) c of the step whose P comes next that have no x row; the rows of the one behind it
    uint64_t unnamed = 0;
    int seen = 0;
    auto rows_of = [&](int st) { return reinterpret_cast<const int*>(lds + C::TILES_B) + (st & 3) * 64; };
    auto without_x = [&](int row) { return __ballot((unsigned)row >= (unsigned)a.T); };
    auto fetch_rows = [&](int st) {
        const int r = c0 + min(64 * st + lane, clen - 1);
        lds_load4(a.row_src, 4u * (uint32_t)r, __builtin_amdgcn_readfirstlane(base + C::TILES_B + (st & 3) * 256));
    };
    auto read_rows = [&](int st) {
#pragma unroll
        for (int u = 0; u < C::JL; ++u) from_row[u] = rows_of(st)[c_of(u)];
    };
    auto jstage = [&](int st) { return (uint32_t)(st % 3) * C::J_B; };
    auto istage = [&](int st) { return 3 * C::J_B + (uint32_t)(st & 1) * C::I_B; };
    auto fetch = [&](int st, int u, auto fast) {                  // FAST: every c of the step exists
        constexpr bool FAST = decltype(fast)::value;
        const bool isj = u < C::JL;
        const uint32_t dst = __builtin_amdgcn_readfirstlane(base + (isj ? jstage(st) + 1024 * (u * C::NW + wv)
                                                                        : istage(st) + 1024 * ((u - C::JL) * C::NW + wv)));
        if constexpr (MODE == DP_DXT) {                           // st: step of a pass over all matrices' rows
            const int pass = st / a.pass_steps, c = 64 * (st - pass * a.pass_steps) + c_of(u), all = a.M * a.N;
            const char* p = zero;
            if (isj) {
                int row, col;
                place(u, row, col);
                if (c < all) p = jbase + 2 * ((int64_t)c * a.K + col);
            } else if (c < all && pass < t.z) {
                const int tok = min(i0 + ((u - C::JL) * C::NW + wv) * 8 + lane / 8, i1 - 1), mt = c / a.N;
                const int r = pass == 0 || pass < a.passes[tok] ? a.map[((int64_t)pass * a.T + tok) * a.M + mt] : -1;
                if (r >= 0) p = reinterpret_cast<const char*>(a.dy + r * a.dy_stride + (c - mt * a.N));
            }
            lds_load16(p, dst);
            return;
        }
        const char* from = isj ? jbase + (C::GATHER ? -(int64_t)c0 * 2 * a.x_stride : st * jadv) : ibase + st * iadv;
        if (C::GATHER && isj) {
            const int s = from_row[u];
            const bool in = (unsigned)s < (unsigned)a.T && (FAST || 64 * st + c_of(u) < clen);
            lds_load16(in ? from + 2 * (s * a.x_stride) + (WIDE ? woff[u] : (int64_t)off[u]) : zero, dst);
        } else if constexpr (FAST && !WIDE) {
            lds_load16(from, off[u], dst);
        } else {
            const char* p = from + (WIDE ? woff[u] : (int64_t)off[u]);
            lds_load16(64 * st + c_of(u) < clen ? p : zero, dst);
        }
    };

    const int wn = wv / C::WT, wt = wv % C::WT;
    floatx4 acc[NI][NJ];
#pragma unroll
    for (int p = 0; p < NI; ++p)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[p][j] = zero4();

    // ---- operand reads: half h of a step's c.  Transposed: lanes 4 q .. 4 q + 3 of sixteen
    // read 16 columns of c row q, and lane m gets column m's four c; two reads make the
    // eight c of its slot.
    const int row_at[2] = {m * 128 + 16 * swz_row(m, g), m * 128 + 16 * swz_row(m, 4 + g)};   // (16 rows on, the swizzle is the same)
    int turn = swz_col<128>(8 * g + (m >> 2), 0);                 // what swz_col turns by, the same for all c rows of a lane
    auto read_t = [&](uint32_t tile, int sub, int h, auto bx) {
        constexpr int BX = decltype(bx)::value;
        const int at = (8 * g + (m >> 2)) * (2 * BX) + 16 * ((m >> 1) & 1) + 8 * (m & 1);
        const uint8_t* p = lds + tile + (16 * ((BX >= 128 ? turn : turn & 6) ^ 2 * sub) + at);
        uint4 o;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + (32 * h + 4 * q) * (2 * BX)));
            const uint2 w = __builtin_bit_cast(uint2, v);
            if (q == 0) { o.x = w.x; o.y = w.y; }
            else { o.z = w.x; o.w = w.y; }
        }
        return o;
    };
    auto read_j = [&](int st, int p, int h) {
        if constexpr (C::JT) return read_t(jstage(st), NI * wn + p, h, std::integral_constant<int, BN>{});
        else return ldg16(lds + jstage(st) + 16 * (NI * wn + p) * 128 + row_at[h]);
    };
    auto read_i = [&](int st, int j, int h) {
        if constexpr (C::IT) return read_t(istage(st), NJ * wt + j, h, std::integral_constant<int, BT>{});
        else return ldg16(lds + istage(st) + 16 * (NJ * wt + j) * 128 + row_at[h]);
    };
    uint4 fi[2][2][NJ], fj[2][2];                                 // [set][half][subtile]; [subtile & 1][half]
    // (GATHER: x rows are asked for four steps ahead, at a step's end: landed at the next
    // step's MID, read at its end, used in the step after.)
    // A row without x adds nothing, whatever its dy is: its x is loaded as zeros, and its dy, which
    // need not be finite, becomes zeros in the registers (a branch a step; looked at in every
    // load of dy it cost up to 15%).
    auto drop_rows = [&](uint4 (&p)[2][NJ], uint64_t rows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t b = (uint32_t)(rows >> (32 * h)) >> (8 * g);           // a lane's eight c, two a word
            auto keep = [&](int i) { return (b >> (2 * i) & 1 ? 0u : 0xFFFFu) | (b >> (2 * i + 1) & 1 ? 0u : 0xFFFF0000u); };
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                p[h][j].x &= keep(0);
                p[h][j].y &= keep(1);
                p[h][j].z &= keep(2);
                p[h][j].w &= keep(3);
            }
        }
    };
    // A step: its first barrier says that the step before is read (its stage of Q is free, and
    // this step's of P, which is in registers), the one at MID that the next step has landed.
    // The loads of the step after it are spread between the products; the next step's P is
    // read from MID on, Q one subtile ahead.
    constexpr int MID = NI / 2, SPAN = NI - MID > 1 ? NI - MID - 1 : 1;   // subtiles with reads of P
    auto step = [&](int st, auto set, auto fast) {
        constexpr int f = decltype(set)::value;
        uint64_t behind = 0;                                      // (GATHER) unnamed of step st + 2
        asm volatile("" : "+v"(turn));                            // the lane addresses are made anew: kept, they take registers
        // all of this wave's reads of P are done: those of Q behind the last of them (NI > 2: in
        // the last subtile) may be in flight
        wait_lds_barrier<NI == 2 ? 0 : C::JT ? 4 : 2>();
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            if (p == MID) {
                wait_loads_barrier<MID * C::LOADS / NI>();
                if constexpr (C::GATHER) {
                    behind = without_x(seen);
                    seen = rows_of(st + 3)[lane];
                }
            }
            if (p >= MID) {
#pragma unroll
                for (int u = (p - MID) * 2 * NJ / SPAN; u < (p - MID + 1) * 2 * NJ / SPAN && u < 2 * NJ; ++u)
                    fi[1 - f][u / NJ][u % NJ] = read_i(st + 1, u % NJ, u / NJ);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) fj[(p + 1) & 1][h] = p + 1 < NI ? read_j(st, p + 1, h) : read_j(st + 1, 0, h);
#pragma unroll
            for (int u = p * C::LOADS / NI; u < (p + 1) * C::LOADS / NI; ++u) fetch(st + 2, u, fast);
            if (C::GATHER && p == NI - 1) {
                read_rows(st + 3);
                fetch_rows(st + 4);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[p][j] = mfma_bf16(fj[p & 1][h], fi[f][h][j], acc[p][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (C::GATHER) {
            if (unnamed) drop_rows(fi[1 - f], unnamed);           // (step st + 1's)
            unnamed = behind;
        }
    };
    if (s0 < s1) {
        if constexpr (C::GATHER) {
#pragma unroll
            for (int st = 0; st < 4; ++st) fetch_rows(s0 + st);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if constexpr (C::GATHER) read_rows(s0 + st);
#pragma unroll
            for (int u = 0; u < C::LOADS; ++u) fetch(s0 + st, u, std::false_type{});
        }
        uint64_t first = 0;                                       // (GATHER) unnamed of step s0
        if constexpr (C::GATHER) {
            read_rows(s0 + 2);
            first = without_x(rows_of(s0)[lane]);
            unnamed = without_x(rows_of(s0 + 1)[lane]);
            seen = rows_of(s0 + 2)[lane];
        }
        wait_loads_barrier<C::LOADS>();
#pragma unroll
        for (int u = 0; u < 2 * NJ; ++u) fi[0][u / NJ][u % NJ] = read_i(s0, u % NJ, u / NJ);
        if (C::GATHER && first) drop_rows(fi[0], first);
#pragma unroll
        for (int h = 0; h < 2; ++h) fj[0][h] = read_j(s0, 0, h);
        int st = s0;
        for (; MODE != DP_DXT && st + 1 < s1 && st + 3 < whole_steps; st += 2) {
            step(st, Set<0>{}, std::true_type{});
            step(st + 1, Set<1>{}, std::true_type{});
        }
        for (; st + 1 < s1; st += 2) {
            step(st, Set<0>{}, std::false_type{});
            step(st + 1, Set<1>{}, std::false_type{});
        }
        if (st < s1) step(st, Set<0>{}, std::false_type{});
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");    // nothing more lands in the stages
    }

    // ---- out, sixteen rows of a wave at a time through the LDS, so that whole row segments
    // are stored: lane (g, m) holds columns 4 g .. 4 g + 3 of each j subtile, row m.  out itself
    // is stored past the caches (8192^3 814 -> 797 us, dW of 5001 rows 8 x 4096 x 8192 433 ->
    // 395), partial sums are read again and are not.
    const int rows = C::DW ? a.M * a.N : a.R;
    const bool whole = a.slices == 1 && !a.to_part;
    const int64_t stride = whole ? a.out_stride : a.cols;
    void* out = whole ? a.out : a.part + (int64_t)z * rows * a.cols - a.col0;            // (DP_DXT: whole)
    const int f32 = whole ? a.out_f32 : 1, J = a.col0 + a.cols;
    const int64_t r0 = (C::DW ? (int64_t)mat * a.N : 0) + i0 + 16 * NJ * wt;
    const int left = i1 - i0 - 16 * NJ * wt, col0 = j0 + 16 * NI * wn;
    constexpr int RS = NI * 64 + 16;
    uint8_t* o = lds + wv * C::OUT_B;
    bool named[NJ];                                               // rows of y whose x row row_src names
#pragma unroll
    for (int j = 0; j < NJ; ++j) named[j] = MODE != DP_Y || x_row(a, min(i0 + 16 * (NJ * wt + j) + m, i1 - 1)) >= 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int p = 0; p < NI; ++p) *reinterpret_cast<floatx4*>(o + m * RS + 64 * p + 16 * g) = named[j] ? acc[p][j] : zero4();
        __builtin_amdgcn_wave_barrier();                          // one wave's LDS accesses complete in order
        asm volatile("" ::: "memory");
        if constexpr (MODE == DP_DXT) {
            // the one sum multiplies every matrix's rows, by zeros where the token has no row of
            // it: what is not finite is summed anew from the token's own rows alone (all of it:
            // 1501 tokens' three of 8 x 16 x 4096 0.4 ms, 16384 tokens' eight of 64 x 16 x 4096 22)
            bool bad = false;
#pragma unroll
            for (int p = 0; p < NI; ++p)
#pragma unroll
                for (int v = 0; v < 4; ++v) bad |= !(fabsf(acc[p][j][v]) < __builtin_inff());
            if (__ballot(bad)) {
                for (int e = lane; e < 16 * 16 * NI; e += 64) {
                    float* at = reinterpret_cast<float*>(o + e / (16 * NI) * RS) + e % (16 * NI);
                    const int tok = i0 + 16 * (NJ * wt + j) + e / (16 * NI), col = col0 + e % (16 * NI);
                    if (fabsf(*at) < __builtin_inff() || tok >= i1 || col >= a.K) continue;
                    float sum = 0.f;
                    for (int pass = 0; pass < a.passes[tok]; ++pass)
                        for (int mt = 0; mt < a.M; ++mt) {
                            const int r = a.map[((int64_t)pass * a.T + tok) * a.M + mt];
                            for (int n = 0; r >= 0 && n < a.N; ++n)
                                sum = fmaf(bf16_to_f32(a.dy[r * a.dy_stride + n]), bf16_to_f32(a.w[((int64_t)mt * a.N + n) * a.K + col]), sum);
                        }
                    *at = sum;
                }
                __builtin_amdgcn_wave_barrier();
                asm volatile("" ::: "memory");
            }
        }
        if (f32) {
            constexpr int LPR = NI * 4, RPI = 64 / LPR;
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
                const int tr = RPI * i + lane / LPR, col = col0 + 4 * (lane % LPR);
                const floatx4 v = *reinterpret_cast<const floatx4*>(o + tr * RS + 16 * (lane % LPR));
                floatx4* to = reinterpret_cast<floatx4*>(static_cast<float*>(out) + (r0 + 16 * j + tr) * stride + col);
                if (16 * j + tr < left && col < J) {
                    if (whole) __builtin_nontemporal_store(v, to);
                    else *to = v;
                }
            }
        } else {
            constexpr int LPR = NI * 2, RPI = 64 / LPR;
#pragma unroll
            for (int i = 0; i < (16 + RPI - 1) / RPI; ++i) {
                const int tr = RPI * i + lane / LPR, col = col0 + 8 * (lane % LPR);
                if (tr >= 16) continue;
                const floatx4 u = *reinterpret_cast<const floatx4*>(o + tr * RS + 32 * (lane % LPR));
                const floatx4 v = *reinterpret_cast<const floatx4*>(o + tr * RS + 32 * (lane % LPR) + 16);
                const u32x4 w = {pack2(u.x, u.y), pack2(u.z, u.w), pack2(v.x, v.y), pack2(v.z, v.w)};
                if (16 * j + tr < left && col < J)
                    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + (r0 + 16 * j + tr) * stride + col));
            }
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
    }
}

// Tiles of the largest size come in rounds of 256, one a compute unit; what is left of the
// last round, if it is half of one or less, is made as tiles of half the rows (5001 rows
// in 8 groups, 4096 columns, K = 8192: 364 us whole, 338 with halves).
template <int MODE, int BT, int BN, bool WIDE>
__global__ void __launch_bounds__((DpCfg<MODE, BT, BN>::NW * 64))
dp_tile(DenseProduct a) {
    using C = DpCfg<MODE, BT, BN>;
    constexpr bool HALVES = BT == 256 && BN == 256;
    __shared__ __attribute__((aligned(16))) uint8_t lds[C::LDS_B];
    const int nn = (a.cols + BN - 1) / BN;
    int half = -1;                                                // 0, 1: a tile's first or second half
    auto pick = [&](int total) {
        const int block = blockIdx.x;
        const int rest = HALVES && a.slices == 1 ? total & 255 : 0, whole = rest > 128 ? total : total - rest;
        if (whole == total || block < whole) return xcd_tile(block, whole);
        const int h = xcd_tile(block - whole, 2 * rest);
        if (h < 0) return -1;
        half = h & 1;
        return whole + (h >> 1);
    };
    DpTile d{};
    if constexpr (C::DW) {
        const int ni = (a.N + BT - 1) / BT, tiles = ni * nn, each = a.M * tiles;
        int tile;
        if (a.M == 1 || tiles < 8) {
            const int b = pick(each * a.slices);
            if (b < 0) return;
            d.z = b / each;
            const int in = b - d.z * each;
            d.mat = in / tiles;
            tile = in - d.mat * tiles;
        } else {                                                  // rows differ by matrix: every XCD takes a part of each
            const int per = (tiles + 7) >> 3, at = blockIdx.x >> 3, q = at / per;
            tile = (blockIdx.x & 7) * per + at - q * per;
            d.z = q / a.M;
            d.mat = q - d.z * a.M;
            if (tile >= tiles || d.z >= a.slices) return;
        }
        d.i0 = tile / nn * BT;
        d.i1 = min(a.N, d.i0 + BT);
        d.j0 = tile % nn * BN;
        d.c0 = a.offsets ? min(max(a.offsets[d.mat], 0), a.R) : 0;
        d.clen = (a.offsets ? min(max(a.offsets[d.mat + 1], d.c0), a.R) : a.R) - d.c0;
    } else if constexpr (MODE == DP_DXT) {                        // tokens; z: the most passes that one of them needs
        const int b = pick(a.row_tiles * nn);
        if (b < 0) return;
        d.i0 = b / nn * BT;
        d.i1 = min(a.T, d.i0 + BT);
        d.j0 = b % nn * BN;
        for (int t0 = d.i0; t0 < d.i1; t0 += 64) {
            const int n = a.passes[min(t0 + lane_id(), d.i1 - 1)];
            for (int p = d.z + 1; __ballot(n >= p); ++p) d.z = p;
        }
    } else {
        const RowTile t = row_tile<BT>(a.offsets, a.M, a.R, [&](int rows) {
            rows = min(rows, a.row_tiles);                       // more only where offsets descend
            const int each = rows * nn;
            int b = pick(each * a.slices);
            if (b < 0) return -1;
            d.z = b / each;
            b -= d.z * each;
            // down groups of 8 row tiles before a column tile on
            const int grp = b / (8 * nn), left = min(8, rows - 8 * grp), in = b - grp * 8 * nn;
            d.j0 = a.col0 + in / left * BN;
            return 8 * grp + in % left;
        });
        if (t.r1 == 0) return;
        d.mat = t.m;
        d.i0 = t.r0;
        d.i1 = t.r1;
        d.clen = MODE == DP_Y ? a.K : a.N;
    }
    if constexpr (HALVES) {
        if (half >= 0) {
            d.i0 += half * (BT / 2);
            d.i1 = min(d.i1, d.i0 + BT / 2);
            if (d.i0 < d.i1) dp_body<MODE, BT / 2, BN, WIDE>(a, d, lds);
            return;
        }
    }
    dp_body<MODE, BT, BN, WIDE>(a, d, lds);
}

// map[p][t][m]: the p-th row of token t that belongs to matrix m, -1 for none (passes past
// the first: only where some matrix has that many); passes[t]: the most rows that token t
// has of one matrix.  A thread a token, offsets and counts in the LDS.
constexpr int kMapMatrices = 128, kMapRows = 32;                  // most matrices, and rows of a token
__global__ void __launch_bounds__(64)
dp_token_map(const int32_t* __restrict__ offsets, const int32_t* __restrict__ token_rows, int per_token, int T, int M, int R,
             int32_t* __restrict__ map, int32_t* __restrict__ passes) {
    __shared__ int32_t off[kMapMatrices + 1];
    __shared__ uint8_t count[64][kMapMatrices];
    for (int i = threadIdx.x; i <= M; i += 64) off[i] = offsets ? min(max(offsets[i], 0), R) : i ? R : 0;
    __syncthreads();
    const int t = blockIdx.x * 64 + threadIdx.x;
    if (t >= T) return;
    uint8_t* n = count[threadIdx.x];
    for (int m = 0; m < M; ++m) {
        n[m] = 0;
        map[(int64_t)t * M + m] = -1;
    }
    int most = 0;
    for (int j = 0; j < per_token; ++j) {
        const int r = token_rows[(int64_t)t * per_token + j];
        if (r < off[0] || r >= off[M]) continue;
        int lo = 0, hi = M;                                       // off[lo] <= r < off[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (off[mid] <= r) lo = mid;
            else hi = mid;
        }
        const int p = n[lo]++;
        int32_t* to = map + ((int64_t)p * T + t) * M;
        if (p == most) {
            most = p + 1;
            for (int m = 0; p > 0 && m < M; ++m) to[m] = -1;
        }
        to[lo] = r;
    }
    passes[t] = most;
}

// ------------------------------------------------------------------ sums ---------
// out[i] = the slices of row i, or of the rows of token i in slot order, added in
// order.  Rows past the matrices' (which no tile has written) are left as they were, or
// add nothing to a token.  Bound by the partial sums' bytes.
__global__ void __launch_bounds__(256)
dp_join(RowJoin a) {
    const int quads = (a.cols + 3) / 4;
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    const int64_t row = i / quads;
    const int col = (int)(i - row * quads) * 4;
    if (row >= a.out_rows) return;
    int64_t lo = 0, hi = a.rows;
    if (a.offsets) {
        lo = min(max((int64_t)a.offsets[0], (int64_t)0), a.rows);
        hi = min(max((int64_t)a.offsets[a.M], lo), a.rows);
    }
    floatx4 s = zero4();
    if (a.token_rows) {
        for (int j = 0; j < a.per_token; ++j) {
            const int64_t r = a.token_rows[row * a.per_token + j];
            if (r < lo || r >= hi) continue;
            for (int z = 0; z < a.slices; ++z) s += *reinterpret_cast<const floatx4*>(a.part + (z * a.rows + r) * (4 * quads) + col);
        }
    } else {
        if (row < lo || row >= hi) return;
        for (int z = 0; z < a.slices; ++z) s += *reinterpret_cast<const floatx4*>(a.part + (z * a.rows + row) * (4 * quads) + col);
    }
    const int64_t at = row * a.out_stride + col;
    if (a.whole) {
        store4(a.out, a.out_f32, at, s);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (col + i >= a.cols) break;
        if (a.out_f32) static_cast<float*>(a.out)[at + i] = s[i];
        else static_cast<uint16_t*>(a.out)[at + i] = (uint16_t)pack2(s[i], s[i]);
    }
}

// ------------------------------------------------------------------ host side ----
hipError_t launch_join(const RowJoin& j, hipStream_t s) {
    const int64_t n = j.out_rows * ((j.cols + 3) / 4);
    if (!n) return hipSuccess;
    prof_begin(s);
    dp_join<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(j);
    prof_end(s, "dp_join");
    return hipGetLastError();
}

namespace {

// Row tiles of BT rows that R rows in M matrices can make at most.
int64_t max_row_tiles(const DenseProduct& a, int BT) {
    const int live = a.M < a.R ? a.M : a.R;
    return a.M > 1 ? a.R / BT + live : (a.R + BT - 1) / BT;
}

struct DpPlan { int bt, bn, slices; };

// Whether lane offsets within a tile pass 32 bits: 256 rows of dy or x, or a gathered row
// anywhere in x.
bool wide_rows(const DenseProduct& a, int mode) {
    const int64_t rows = mode == DP_Y && a.row_src ? a.T : 256, x = mode == DP_DX || mode == DP_DWG ? 0 : a.x_stride;
    return rows * x >= (1ll << 31) || 256 * (mode == DP_Y ? 0 : a.dy_stride) >= (1ll << 31);
}

// Tile sizes and slices of c: the least of an estimate in us from measured times.  A
// launch takes 4; a tile takes `fixed` (its first loads, its way out) and a step of 64 of
// c `alone` where it has a compute unit to itself, `full` where `fit` tiles share it (as
// many as the LDS holds); slices are joined by a launch more and pass through memory
// twice.  Measured with 2000 rows of 4096 x 4096 (a round of 64 steps on all of the chip)
// and 64 rows (tiles alone).  What it chooses between (us, T x M x N x K, tiles i x j /
// slices, inputs in the memory-side cache): y of 2000 x 1 x 4096 x 4096 128x256 58, 256x256 58,
// 64x64 97; 500 x 1 x 2048 x 2048 64x64 11, 256x256 25; 64 x 1 x 4096 x 4096 64x64/8 14, 64x64
// 28; dx of 4096 tokens' four of 64 x 512 x 1024 128x128 32, 256x256 31, 64x64 42; dW of 16384 x
// 1 x 128 x 4096 128x64/8 38, 64x256/8 35, 64x256 155.
DpPlan plan(const DenseProduct& a, int mode, int most_slices = 16, float* us_out = nullptr) {
    struct Cost { int bt, bn, fit; float fixed, alone, full, dw_full; };
    static constexpr Cost kTiles[9] = {
        {64, 64, 4, 2.6f, 0.37f, 0.73f, 1.05f},  {64, 128, 2, 2.8f, 0.44f, 0.69f, 0.92f},  {64, 256, 1, 3.2f, 0.54f, 0.66f, 0.69f},
        {128, 64, 2, 2.8f, 0.42f, 0.63f, 0.69f}, {128, 128, 2, 3.6f, 0.55f, 1.20f, 1.13f}, {128, 256, 1, 4.2f, 0.65f, 0.97f, 0.99f},
        {256, 64, 1, 3.4f, 0.55f, 0.73f, 0.74f}, {256, 128, 1, 4.2f, 0.63f, 0.97f, 0.99f}, {256, 256, 1, 6.5f, 1.05f, 1.40f, 1.52f}};
    const int J = mode == DP_Y ? a.N : a.K, live = a.M < a.R ? a.M : (a.R ? a.R : 1);
    const float each = (float)a.R / live;                         // rows of a matrix, on average
    const float c = mode == DP_Y ? a.K : mode == DP_DX ? a.N : each;
    const int steps = (int)((c + 63) / 64) > 0 ? (int)((c + 63) / 64) : 1;
    const double out = mode == DP_DW ? (double)a.M * a.N * a.K : (double)a.R * J;
    DpPlan best{};
    float least = 0;
    for (const Cost& t : kTiles) {
        const float nn = (J + t.bn - 1) / t.bn, q = each / t.bt, up = (float)(int)(q + 0.9f);
        // row tiles of a matrix: among few matrices the last one is half empty on average; many
        // (routed experts) have about as many rows each
        const float rows = a.M == 1 ? (float)((a.R + t.bt - 1) / t.bt) : (float)live * (a.M < 64 ? q + 0.5f : up > q + 0.25f ? up : q + 0.25f);
        const float tiles = nn * (mode == DP_DW ? (float)a.M * ((a.N + t.bt - 1) / t.bt) : rows);
        const float full = mode == DP_DW ? t.dw_full : t.full;
        const int fit = mode == DP_DW && t.bt + t.bn == 256 && t.bt == 128 ? 1 : t.fit;   // (gathered x rows do not fit beside two)
        for (int z = 1; z <= most_slices && (z == 1 || (steps >= 2 * z && tiles * z < 4096)); z *= 2) {
            const float n = tiles * z / 256, chain = t.fixed + (float)((steps + z - 1) / z) * full;     // a full round
            const int rounds = (int)(n / fit);
            const float rest = n - rounds * fit;                // tiles a compute unit in the last round
            float us = 4 + rounds * chain;
            if (rest > 0 && rest <= 0.5f && t.bt + t.bn == 512 && z == 1) {   // tiles of half the rows
                us += 4.2f + steps * 0.97f;
            } else if (rest > 0) {
                const float share = fit == 1 ? (rounds ? 1.f : rest) : (rest < 1 ? 0.f : (rest - 1) / (fit - 1));
                us += t.fixed + (float)((steps + z - 1) / z) * (t.alone + (full - t.alone) * (share < 1 ? share : 1.f));
            }
            if (z > 1) us += 4 + 0.15f * z + (float)(out * (8 * z + 2) / 5e6);
            if (!best.bt || us < least) {
                least = us;
                best = DpPlan{t.bt, t.bn, z};
            }
        }
    }
    if (us_out) *us_out = least;
    return best;
}

template <int MODE, int BT, int BN, bool WIDE = false>
hipError_t launch_tile(const DenseProduct& a, int64_t blocks, hipStream_t s) {
    prof_begin(s);
    dp_tile<MODE, BT, BN, WIDE><<<(unsigned)((blocks + (BT + BN == 512 ? 128 : 0) + 7) & ~7ll), DpCfg<MODE, BT, BN>::NW * 64, 0, s>>>(a);
    prof_end(s, MODE == DP_Y ? "dp_tile_y" : MODE == DP_DX || MODE == DP_DXT ? "dp_tile_dx" : "dp_tile_dw");
    return hipGetLastError();
}

template <int MODE, int BT>
hipError_t launch_tile(const DenseProduct& a, int bn, int64_t blocks, hipStream_t s) {
    if (bn == 64) return launch_tile<MODE, BT, 64>(a, blocks, s);
    if constexpr (MODE != DP_DWG || BT < 256) {
        if (bn == 256) return launch_tile<MODE, BT, 256>(a, blocks, s);
    }
    return launch_tile<MODE, BT, 128>(a, blocks, s);
}

template <int MODE>
hipError_t launch_tile(DenseProduct a, DpPlan p, hipStream_t s) {
    const bool wide = wide_rows(a, MODE);
    if (wide) p.bt = p.bn = 128;
    else if (MODE == DP_DWG && p.bt + p.bn == 512) p.bt = 128;     // the x rows have no place beside the largest tiles
    if (!a.cols) a.cols = MODE == DP_Y ? a.N : a.K;
    const int nn = (a.cols + p.bn - 1) / p.bn;
    a.slices = p.slices;
    a.row_tiles = (int)max_row_tiles(a, p.bt);
    constexpr bool DW = MODE == DP_DW || MODE == DP_DWG;
    const int64_t tiles = (DW ? (int64_t)((a.N + p.bt - 1) / p.bt) : a.row_tiles) * nn;              // (dW: of a matrix)
    const int64_t blocks = (DW ? a.M * (a.M > 1 && tiles >= 8 ? (tiles + 7) & ~7ll : tiles) : tiles) * p.slices;
    if (wide) return launch_tile<MODE, 128, 128, true>(a, blocks, s);
    switch (p.bt) {
        case 64: return launch_tile<MODE, 64>(a, p.bn, blocks, s);
        case 128: return launch_tile<MODE, 128>(a, p.bn, blocks, s);
        default: return launch_tile<MODE, 256>(a, p.bn, blocks, s);
    }
}

// Whether dp_stream makes y: sixteen rows a matrix on average, twelve of many (routed
// experts, some of which have more than sixteen), and not very many workgroups of a short K.
// us, streamed and by dp_tile (the better of its tiles): 16 rows through 4096 x 4096 9.3 and 12.6,
// 16 through 8192 x 8192 24.2 and 26.3, 24 through 4096 x 4096 12.7 and 12.7; 80 rows over 512 of
// 128 x 4096 18.3 and 22.4; over 64 of 128 x 4096 with as many rows each 512 rows 15.0 and 17.8,
// 768 15.8 and 18.4, routed at random 21.9 and 18.3, 24.1 and 18.5, 1024 rows 25.6 and 18.7; 4096
// over 512 of 128 x 512 32.7 and 16.0, 512 over 64 of 1024 x 1024 26.1 and 22.5.
bool streams(const DenseProduct& a) {
    const int live = a.M < a.R ? a.M : a.R;
    if (a.R > (int64_t)live * (a.M < 64 ? 16 : 12)) return false;
    return a.K >= 1024 || (int64_t)live * ((a.N + 31) / 32) <= 1024;
}

hipError_t launch_stream(const DenseProduct& a, hipStream_t s) {
    const int64_t tiles = max_row_tiles(a, 16), live = a.M == 1 ? tiles : a.M < a.R ? a.M : a.R;
    const int64_t wgs = live * ((a.N + 31) / 32), last = (wgs - 1) % 256 + 1;
    prof_begin(s);
    // 32 columns a workgroup; 16 where 32 leave half of the compute units idle, throughout or in the
    // last of two or three rounds (us with 16 and 32: 16 rows through 4096 x 4096 10.2 and 10.8, through
    // 8192 x 8192, 256 workgroups, 31.8 and 25.1; 80 rows over 512 of 128 x 4096 19.6 and 22.2, 120 25.1
    // and 22.1, 160 31.0 and 33.4; 512 over 64 of 512 x 1024, 1024 workgroups, 17.9 and 16.1)
    if (wgs <= 128 || (wgs > 256 && wgs < 768 && last <= 128)) dp_stream<1><<<dim3((a.N + 15) / 16, (unsigned)tiles), 256, 0, s>>>(a);
    else dp_stream<2><<<dim3((a.N + 31) / 32, (unsigned)tiles), 256, 0, s>>>(a);
    prof_end(s, "dp_stream");
    return hipGetLastError();
}

size_t up(size_t v) { return (v + 255) & ~(size_t)255; }

size_t part_bytes(const DenseProduct& a, int mode, int slices) {
    return up((size_t)slices * (mode == DP_DW ? (size_t)a.M * a.N * a.K : (size_t)a.R * (mode == DP_Y ? a.N : a.K)) * 4);
}

}  // namespace

size_t dense_product_ws_bytes(const DenseProduct& a) {
    if (!a.R || streams(a)) return 256;
    const DpPlan p = plan(a, DP_Y);
    return p.slices > 1 ? part_bytes(a, DP_Y, p.slices) : 256;
}

hipError_t launch_dense_product(DenseProduct a, void* ws, hipStream_t s) {
    if (streams(a)) return launch_stream(a, s);
    const DpPlan p = plan(a, DP_Y);
    a.part = static_cast<float*>(ws);
    const hipError_t e = launch_tile<DP_Y>(a, p, s);
    if (e != hipSuccess || p.slices == 1) return e;
    return launch_join(RowJoin{a.part, p.slices, a.R, a.N, a.out, a.out_stride, a.out_f32, 1, a.R, a.offsets, a.M, nullptr, 0}, s);
}

// Columns of dx that are made for tokens at once: their rows' partial sums then stay in the
// 256 MB memory-side cache between the two launches (16384 tokens' ten of 512 x 128 x 4096: 1565 us at once, 1419 so;
// 48 and 96 MB at once measured more on the smaller ones).
int token_cols(const DenseProduct& a, int slices) {
    const int64_t fit = (192ll << 20) / ((int64_t)a.R * slices * 4 + 1);
    const int64_t cols = fit / 256 * 256;
    return cols < 256 ? 256 : cols < a.K ? (int)cols : a.K;
}

// dx of tokens in one sum over all matrices (DP_DXT), where that is estimated to take less
// than the rows' products and their way through memory: few matrices of few rows, LoRA's
// inputs among them.  A step waits for its rows' places in the map, so it counts for two of
// plan()'s; the rows' half counts what the caches leave of 8 bytes written and read again.
// us, rows and then added -> one sum, fp32 out, T tokens' k of M matrices: T 512 k 3 of
// 8 x 16 x 4096 18.6 -> 16.0, T 1501 36.1 -> 18.3, T 16384 352 -> 87; T 1501 k 8 of
// 64 x 16 x 4096 78 -> 55; and left as rows: T 16 of 8 x 16 x 4096 15.8 -> 16.0, T 1501 k 3 of
// 8 x 128 x 4096 39 -> 48, k 2 of 4 x 256 x 1024 17.4 -> 24.4, T 4096 k 2 of 128 x 8 x 1024 30 -> 44.
struct TokenPlan { bool one_sum; DpPlan p; size_t bytes; };
TokenPlan token_plan(const DenseProduct& a) {
    TokenPlan t{};
    const int64_t c = (int64_t)a.M * a.N, bytes = ((int64_t)kMapRows * a.M + 1) * a.T * 4;
    if (c > 1024 || a.M > kMapMatrices || bytes > (256ll << 20)) return t;
    DenseProduct one{};
    one.T = one.R = a.T; one.M = 1; one.N = (int)c; one.K = a.K;
    float sum = 0, rows = 0;
    t.p = plan(one, DP_DX, 1, &sum);
    if (t.p.bt > 128) t.p.bt = 128;
    if (t.p.bn < 128 || t.p.bt < 128) t.p.bn = 128;
    plan(a, DP_DX, 16, &rows);
    t.one_sum = 2 * sum + a.M / 16.f < rows + 5 + (float)((double)a.R * a.K * 4 / 4.5e6);
    t.bytes = (size_t)bytes;
    return t;
}

// dx's partial sums (or rows, for tokens) and dW's share the workspace: dW runs first.
size_t dense_backward_ws_bytes(const DenseProduct& a) {
    const DpPlan pw = plan(a, DP_DW), px = plan(a, DP_DX);
    size_t w = pw.slices > 1 ? part_bytes(a, DP_DW, pw.slices) : 256;
    const size_t x = px.slices > 1 ? part_bytes(a, DP_DX, px.slices) : 0;
    const int cols = token_cols(a, px.slices);
    const size_t t = up((size_t)px.slices * a.R * (cols < a.K ? cols : a.K) * 4);
    const TokenPlan tp = token_plan(a);
    if (x > w) w = x;
    if (t > w) w = t;
    return tp.one_sum && tp.bytes > w ? tp.bytes : w;
}

hipError_t launch_dense_backward(const DenseGrad& gr, void* ws, hipStream_t s) {
    DenseProduct a = gr.p;
    a.part = static_cast<float*>(ws);
    if (gr.dw) {
        const DpPlan p = plan(a, DP_DW);
        a.out = gr.dw; a.out_stride = a.K; a.out_f32 = gr.dw_f32;
        hipError_t e = a.row_src ? launch_tile<DP_DWG>(a, p, s) : launch_tile<DP_DW>(a, p, s);
        if (e == hipSuccess && p.slices > 1) {
            const int64_t rows = (int64_t)a.M * a.N;
            e = launch_join(RowJoin{a.part, p.slices, rows, a.K, gr.dw, a.K, gr.dw_f32, 1, rows, nullptr, 0, nullptr, 0}, s);
        }
        if (e != hipSuccess) return e;
    }
    if (!gr.dx) return hipSuccess;
    const DpPlan p = plan(a, DP_DX);
    a.out = gr.dx; a.out_stride = gr.dx_stride; a.out_f32 = gr.dx_f32;
    if (!gr.token_rows) {
        const hipError_t e = a.R ? launch_tile<DP_DX>(a, p, s) : hipSuccess;
        if (e != hipSuccess || p.slices == 1) return e;
        return launch_join(RowJoin{a.part, p.slices, a.R, a.K, gr.dx, gr.dx_stride, gr.dx_f32, 1, a.R, a.offsets, a.M, nullptr, 0}, s);
    }
    const TokenPlan tp = token_plan(a);
    if (tp.one_sum && gr.per_token <= kMapRows) {
        int32_t* passes = static_cast<int32_t*>(ws);
        int32_t* map = passes + a.T;
        prof_begin(s);
        dp_token_map<<<(a.T + 63) / 64, 64, 0, s>>>(a.offsets, gr.token_rows, gr.per_token, a.T, a.M, a.R, map, passes);
        prof_end(s, "dp_token_map");
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.map = map;
        a.passes = passes;
        a.pass_steps = (a.M * a.N + 63) / 64;
        a.slices = 1;
        a.cols = a.K;
        a.row_tiles = (a.T + tp.p.bt - 1) / tp.p.bt;
        const int64_t blocks = (int64_t)a.row_tiles * ((a.K + tp.p.bn - 1) / tp.p.bn);
        if (tp.p.bt == 64) return launch_tile<DP_DXT, 64, 128>(a, blocks, s);
        return tp.p.bn == 128 ? launch_tile<DP_DXT, 128, 128>(a, blocks, s) : launch_tile<DP_DXT, 128, 256>(a, blocks, s);
    }
    a.to_part = 1;
    // few rows of very many tokens: no more than 2^31 threads add them (2^20 tokens by 8192 columns)
    const int64_t threads = (1ll << 33) / a.T / 256 * 256;
    const int fit = token_cols(a, p.slices), most = fit < threads ? fit : (int)threads;
    for (a.col0 = 0; a.col0 < a.K; a.col0 += a.cols) {
        a.cols = a.K - a.col0 < most ? a.K - a.col0 : most;
        hipError_t e = a.R ? launch_tile<DP_DX>(a, p, s) : hipSuccess;
        void* dx = static_cast<char*>(gr.dx) + (int64_t)a.col0 * (gr.dx_f32 ? 4 : 2);
        if (e == hipSuccess)
            e = launch_join(RowJoin{a.part, p.slices, a.R, a.cols, dx, gr.dx_stride, gr.dx_f32, 1, a.T, a.offsets, a.M, gr.token_rows,
                                   gr.per_token}, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace em
