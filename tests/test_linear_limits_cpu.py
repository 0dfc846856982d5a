"""Sizes that the linear-layer operators' launches do not take, refused on the host."""

import ctypes

import pytest

from matrix_roots_amd import binding as B

# fake, never-dereferenced "device" addresses, far apart
P = [k << 44 for k in range(1, 6)]
SHAPE = 2


@pytest.mark.parametrize("m, n", [((1 << 30) - 127, 1), (1 << 30, 128), ((1 << 29) - 127, 129), (1 << 22, 32641)])
def test_more_blocks_than_a_launch_has(m, n):
    """2^23 blocks of 512 threads are 2^32 threads."""
    p = B.QuantizeProblem(m=m, n=n, X=P[0], ldx=n, Q=P[1], ldq=n, S=P[2], lds=(n + 127) // 128, x_dtype=B.MR_BF16,
                          q_dtype=B.MR_E4M3, block=B.MR_BLOCK_VECTOR)
    lib = B.library()
    assert lib.quantize_blocks(ctypes.addressof(p), None) == SHAPE
    assert b"blocks" in lib.mr_last_error_message()
