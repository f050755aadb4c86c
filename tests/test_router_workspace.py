"""Workspace of the router's backward pass (no GPU needed): its planes hold what
the products' tiles read past them, and no more than that."""
import pytest

import shared_matrix_expert_amd as em
from test_router_train import dims

TILE = 128                                                # the largest tile's rows


def up(n, a):
    return -(-n // a) * a


@pytest.mark.parametrize("rows", [64, 128])
def test_tiles_read_inside_the_planes(rows):
    """The furthest element that a tile of `rows` reads, for every T and E by 32."""
    for Tp in range(32, 1024 + 32, 32):
        for Ep in range(32, 1024 + 32, 32):
            held = (3 * Tp + TILE - 32) * Ep
            dx = (2 * Tp + up(Tp, rows) - 1) * Ep + Ep                      # last row of the last tile, all of its columns
            dw = (3 * Tp - 1) * Ep + up(Ep, rows)                           # last token, last column of the last tile
            assert max(dx, dw) <= held


def test_size_of_one_slice():
    """A batch of one slice: the planes and the chunks' sums of dbias."""
    for T, E, d in ((1, 8, 128), (11, 88, 640)):
        Tp, Ep = up(T, 32), up(E, 32)
        want = up((3 * Tp + TILE - 32) * Ep * 2, 256) + up(Tp // 4 * E * 4, 256)
        assert em.edge_moe_route_backward_ws_bytes(dims(T, E, 2, d)) == want
