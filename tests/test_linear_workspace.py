"""Host-side check that every plan of the linear layer's products that the library accepts finds room in the
workspace for the partial sums of its split tiles."""
import random

import pytest

import output_head_kl_b200 as K

WIDTHS = (128, 192, 256)
WAVE = 74                 # tiles from which on split tiles join by way of the workspace (dW: always)
SHARES = 80               # shares of split tiles that run at once
SMS = (132, 148, 160)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from output_head_kl_b200 import build
    build.build()


def _up(n, to):
    return -(-n // to) * to


def _tiles(rows, cols, width):
    return -(-rows // 256) * -(-cols // width)


def _fixed_bytes(M, d_out, backward):
    """The workspace without the partial sums: flag word, tickets and, for the gradient, dz and the column sums."""
    n = _up(256 + SHARES // 2 * 16 * 4 + (4 * -(-d_out // 256) if backward else 0), 256)
    if backward:
        cols = -(-d_out // 256)
        chunks = max(1, min(-(-8 * 512 // cols), -(-M // 32), 256))
        n += _up(M * d_out * 2, 256) + _up(chunks * d_out * 4, 256)
    return n


def _share_bytes(product, rows, cols, length):
    """The most bytes of partial sums that a plan of out[rows, cols] can need: tiles of the last wave x splits."""
    most = 0
    blocks = -(-length // 64)
    for width in WIDTHS:
        tiles = _tiles(rows, cols, width)
        if product != K.LINEAR_DW and tiles < WAVE:
            continue      # a cluster joins its shares over shared memory
        for sms in SMS:
            tail = tiles % (sms // 2)
            for splits in range(2, 9):
                if blocks // splits >= 4 and tail * splits <= min(sms // 2, SHARES):
                    most = max(most, tail * splits * 256 * width * 4)
    return most


def _check(M, d_in, d_out):
    forward = K.kdkl_linear_workspace_bytes(M, d_in, d_out)
    assert forward - _fixed_bytes(M, d_out, False) >= _share_bytes(K.LINEAR_FORWARD, M, d_out, d_in)
    room = K.kdkl_linear_workspace_bytes(M, d_in, d_out, True) - _fixed_bytes(M, d_out, True)
    assert room >= _share_bytes(K.LINEAR_DX, M, d_in, d_out), (M, d_in, d_out)
    assert room >= _share_bytes(K.LINEAR_DW, d_out, d_in, M), (M, d_in, d_out)


@pytest.mark.parametrize("M,d_in,d_out", [(2048, 256, 8), (3503, 248, 64), (2048, 256, 256), (2048, 512, 768),
                                          (1536, 256, 512), (2048, 1024, 200)])
def test_many_shares_of_192_wide_tiles(M, d_in, d_out):
    """Widths at which tiles of 192 columns are more, and their shares larger in all, than tiles of 256."""
    _check(M, d_in, d_out)


def test_every_plan_has_room():
    for M in (1, 255, 2048, 4097, 20000, 1 << 20):
        for d_in in range(64, 1345, 64):
            for d_out in (8, 136, 256, 264, 512, 768, 1032, 4096):
                _check(M, d_in, d_out)
    rng = random.Random(3)
    for _ in range(4000):
        _check(rng.randint(1, 9000), 8 * rng.randint(1, 700), 8 * rng.randint(1, 700))


def test_sizes_do_not_grow_without_bound():
    """The partial sums are those of one wave at most, however many rows or columns there are."""
    for M, d_in, d_out in ((1 << 20, 4096, 4096), (20000, 8192, 8192)):
        room = K.kdkl_linear_workspace_bytes(M, d_in, d_out, True) - _fixed_bytes(M, d_out, True)
        assert room <= SHARES * 256 * 256 * 4
