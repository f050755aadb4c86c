// Row tiles of a product whose rows are grouped by matrix.
#pragma once

#include "common.h"

namespace em {

// A row tile: rows [r0, r1) of y, all of matrix m.  Row tiles are numbered
// matrix by matrix; `total` is their count, r1 = 0 marks no tile.
struct RowTile { int m, r0, r1, total; };

// Inclusive sum over the lanes up to each one, with DPP row shifts and
// broadcasts (no LDS).
template <int CTRL, int ROWS>
EM_DEV int dpp_add(int v) { return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false); }
EM_DEV int scan_add(int v) {
    v = dpp_add<0x111, 0xF>(v);       // row_shr:1, 2, 4, 8: sums within a row of 16 lanes
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);       // row_bcast:15 into rows 1 and 3, then :31 into rows 2 and 3
    return dpp_add<0x143, 0xC>(v);
}

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
    const int sum = scan_add(mine);
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
    if (offsets) {
        if (M <= 64) return find_tile<BT, 1>(offsets, M, R, pick);
        return M <= 512 ? find_tile<BT, 8>(offsets, M, R, pick) : find_tile<BT, 16>(offsets, M, R, pick);
    }
    RowTile t{0, 0, 0, (R + BT - 1) / BT};
    const int rt = pick(t.total);
    if (rt < 0 || rt >= t.total) return t;
    t.r0 = rt * BT;
    t.r1 = min(R, t.r0 + BT);
    return t;
}

}  // namespace em
