"""What the copies of the 8-bit floating point product may read (csrc/window.hpp, compiled for the
host): rows of the operand and nothing behind them, whichever way a buffer's range check counts a
wave's offset."""
import ctypes
import itertools
import subprocess

import numpy as np
import pytest

from weight_only_bit_moe_amd import build as B

SOURCE = """
#include "window.hpp"
extern "C" void window(int first, int n, int rows, uint32_t ld, uint32_t K, long long *start, long long *bytes)
{
    const wna16::Window w = wna16::window_of(first, n, rows, ld, K);
    *start = w.start;
    *bytes = w.bytes;
}
"""


@pytest.fixture(scope="module")
def window(tmp_path_factory):
    at = tmp_path_factory.mktemp("window")
    (at / "w.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", B.CSRC, str(at / "w.cpp"), "-o", str(at / "w.so")],
                   check=True)
    f = ctypes.CDLL(str(at / "w.so")).window
    f.argtypes = [ctypes.c_int] * 3 + [ctypes.c_uint32] * 2 + [ctypes.POINTER(ctypes.c_longlong)] * 2

    def call(first, n, rows, ld, K):
        s, b = ctypes.c_longlong(), ctypes.c_longlong()
        f(first, n, rows, ld, K, ctypes.byref(s), ctypes.byref(b))
        return s.value, b.value
    return call


def let_through(voff, soff, size):
    """The words at lanes' offsets that a range check may pass, by each way of counting soff: not at
    all, added, or taken from the size in 32 bits."""
    return voff < size, voff + soff < size, voff < (size - soff) % 2 ** 32


def reads(ld, K):
    """(lane offset in a row, wave offset) of every copy of a row: whole blocks of 128, then the last
    one, whose pieces past K read the row's first."""
    piece = np.arange(0, 128, 4)                         # words: 8 pieces of 16 bytes
    for k in range(0, K - K % 128, 128):
        yield piece, k
    if K % 128:
        k = K - K % 128
        yield np.where(k + piece // 16 * 16 < K, k + piece, piece % 16), 0


SIZES = [(16, 16), (32, 16), (128, 128), (144, 144), (160, 144), (400, 272), (2048, 2048), (4112, 4096), ((1 << 23) - 16, 4080)]


@pytest.mark.parametrize("ld,K", SIZES)
def test_copies_read_rows_of_the_operand_only(window, ld, K):
    for rows in (1, 2, 7, 8, 9, 63, 64, 65, 100, 128, 191, 200, 255, 256):
        for first in range(0, 256, 8):
            start, size = window(first, 8, rows, ld, K)
            assert size < 2 ** 32
            r = np.arange(8)[:, None]
            for column, k in reads(ld, K):
                voff = r * ld + column[None]
                at = start + voff + k
                inside = (at // ld < rows) & (at % ld < K)
                wanted = first + r < rows
                for passed in let_through(voff, k, size):
                    assert not (passed & ~inside).any(), (rows, first, k)
                    # and rows that there are arrive, as themselves
                    assert passed[np.broadcast_to(wanted, passed.shape)].all()
                    assert (at // ld == first + r)[np.broadcast_to(wanted, passed.shape)].all()


def test_a_window_of_all_rows_would_not_do():
    """Rows reached by the wave's offset: past the end they are outside one way of counting only."""
    ld, K, rows = 4096, 4096, 3
    size = (rows - 1) * ld + K
    passes = [set(), set(), set()]
    for first, r in itertools.product(range(0, 256, 8), range(8)):
        for way, passed in enumerate(let_through(np.array([r * ld]), first * ld, size)):
            if passed[0] and first + r >= rows:
                passes[way].add(first + r)
    assert passes[0] and not passes[1] and passes[2]
