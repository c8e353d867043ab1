"""Arithmetic of the operators' rows (csrc/ops_rows.h), compiled for the host:
what a row's bulk copy takes, which operands share bytes, and when a team
gives up."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_allreduce_reduction_gb300", "csrc")

SOURCE = r"""
#include "ops_rows.h"
using namespace vrccl;
extern "C" void rowWindowOf(uintptr_t base, size_t ld, size_t row, size_t rows, size_t cols, size_t elem, uintptr_t* out) {
  const unsigned cut = cutRows(ld, elem);
  const Window w = rowWindow(base, ld, row, rows, cols, elem, cut);
  out[0] = w.row; out[1] = w.end; out[2] = w.lo; out[3] = w.hi;
  out[4] = w.headEnd(); out[5] = w.tailBegin(); out[6] = maybeCut(row, rows, cut);
}
extern "C" int meet(uintptr_t p, size_t ld, size_t rows, size_t cols, uintptr_t q, size_t le, size_t rowsq, size_t colsq) {
  return overlap(matrixSpan((void*)p, ld, rows, cols, 2), matrixSpan((void*)q, le, rowsq, colsq, 2));
}
extern "C" int wordOf(int turn) { return givenUpWord(turn); }
extern "C" int leaves(int word, int turn) { return givenUp(word, turn); }
"""


@pytest.fixture(scope="module")
def rows_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cc").write_text(SOURCE)
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "the library's build needs a host compiler too"
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "rows.cc"), "-o", str(d / "rows.so")],
                   check=True)
    return ctypes.CDLL(str(d / "rows.so"))


@pytest.mark.parametrize("elem", [2, 4])
def test_copies_of_short_rows_stay_inside_the_matrix(rows_lib, elem):
    """Every copied 16-byte block lies between the matrix's first and last
    byte, and copy and single elements together make up the row."""
    fn = rows_lib.rowWindowOf
    fn.argtypes = [ctypes.c_size_t] * 6 + [ctypes.POINTER(ctypes.c_size_t)]
    out = (ctypes.c_size_t * 7)()
    for skew in range(0, 16, elem):
        base = 4096 + skew
        for cols in range(1, 20):
            for ld in (cols, cols + 1, cols + 3, cols + 8):
                for rows in (1, 2, 3, 9, 17):
                    last = base + ((rows - 1) * ld + cols) * elem
                    for row in range(rows):
                        fn(base, ld, row, rows, cols, elem, out)
                        at, end, lo, hi, head, tail, cut = out
                        where = (skew, cols, ld, rows, row)
                        assert (at, end) == (base + row * ld * elem, base + (row * ld + cols) * elem), where
                        assert lo % 16 == 0 and hi % 16 == 0 and lo <= hi, where
                        assert lo == hi or (base <= lo and hi <= last), where
                        copied = set(range(max(lo, at), min(hi, end)))
                        single = list(range(at, head)) + list(range(tail, end))
                        assert len(single) == len(set(single)) and not copied & set(single), where
                        assert copied | set(single) == set(range(at, end)), where
                        assert cut or not single, where


def test_a_team_gives_up_at_one_barrier(rows_lib):
    """Whatever a faster thread has written in the next turn, a thread that
    reads the word late stays with it; at that turn's barrier all leave."""
    for turn in (0, 1):  # a turn's parity
        word = 0
        assert not rows_lib.leaves(word, turn)  # the fast thread goes on
        word = rows_lib.wordOf(turn ^ 1)  # and gives up the next turn's wait
        assert not rows_lib.leaves(word, turn)  # the slow one reads only now
        assert rows_lib.leaves(word, turn ^ 1)  # both, past the next barrier


def test_operands_side_by_side_do_not_overlap(rows_lib):
    """overlap() against the sets of elements: exact for one stride and for
    runs, never false where two strides share an element."""
    rows_lib.meet.argtypes = [ctypes.c_size_t] * 8
    elements = lambda at, ld, rows, cols: {at + 2 * (r * ld + c) for r in range(rows) for c in range(cols)}  # noqa: E731
    accepted = 0
    shapes = [(ld, rows, cols) for ld in (6, 7) for rows in (1, 2, 4) for cols in (1, 3, 6)]
    for a in shapes:
        for b in shapes:
            for at in range(2048 - 60, 2048 + 60, 2):
                share = bool(elements(2048, *a) & elements(at, *b))
                got = bool(rows_lib.meet(2048, *a, at, *b))
                if a[0] == b[0] or (a[1] == 1 or b[1] == 1):
                    one = a[1] == 1 or b[1] == 1  # a run that reaches past a row's gap counts as touching it
                    assert got == share or (one and got), (a, b, at)
                    accepted += not got
                else:
                    assert got or not share, (a, b, at)
    assert accepted > 1000
    # column slices of one buffer, and a run between the rows
    assert not rows_lib.meet(4096, 512, 100, 256, 4096 + 512, 512, 100, 256)
    assert rows_lib.meet(4096, 512, 100, 256, 4096 + 510, 512, 100, 256)
    assert not rows_lib.meet(4096, 512, 100, 256, 4096 + 7 * 1024 + 512, 1, 1, 100)
