"""Arithmetic of rows in chunks of eight (csrc/ops_chunks.h), compiled for the
host: which bytes a warp's lanes load and store on every skew, the dropout's
generator and its threshold, and division by multiplication."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import replica as o

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_allreduce_reduction_gb300", "csrc")

SOURCE = r"""
#include <initializer_list>
#include "ops_chunks.h"
using namespace vrccl;
// The bytes that the store of a row by lanes writes, and which lane writes each: as storeChunk, lane by lane.
extern "C" void storeOf(unsigned skew, int E, int cols, int firstChunk, int lanes, int step, int* writer, int* times) {
  const int NB = kChunk * E / 16;
  for (int lane = 0; lane < lanes; ++lane) {
    const Place place = {lane, lanes, firstChunk + lane, step};
    if (lane >= step) continue;
    const int at = (firstChunk + lane) * kChunk * E, left = cols - (firstChunk + lane) * kChunk;
    if (left <= 0) continue;
    auto mark = [&](int byte, int n) {
      if ((byte + (int)skew) % n) writer[byte] = 1000;  // not aligned
      for (int i = 0; i < n; ++i) writer[byte + i] += lane, ++times[byte + i];
    };
    auto rest = [&](int from, int n) {
      for (int size : {8, 4, 2})
        if (n & size) mark(from + restPiece(n, size), size);
    };
    if (skew == 0) {
      for (int b = 0; b < NB; ++b) {
        const int n = left * E - 16 * b;
        if (n >= 16)
          mark(at + 16 * b, 16);
        else if (n > 0)
          rest(at + 16 * b, n);
      }
      continue;
    }
    const int head = headOf(skew);
    if (!headStored(skew, E, left, place)) {
      if (left * E < head) {
        for (int e = 0; e < left; ++e) mark(at + e * E, E);
        continue;
      }
      for (int size : {2, 4, 8})
        if (head & size) mark(at + headPiece(head, size), size);
    }
    for (int b = 0; b < NB; ++b) {
      const int from = at + head + 16 * b, n = restOf(b, skew, E, left);
      if (wholeBlock(b, skew, E, left, place))
        mark(from, 16);
      else if (n > 0)
        rest(from, n);
    }
  }
}
extern "C" int loaded(uintptr_t block, uintptr_t rowEnd, uintptr_t begin, uintptr_t end) { return blockLoaded(block, rowEnd, begin, end); }
extern "C" int together(uintptr_t p, int E, int left, uintptr_t begin, uintptr_t end) { return fromBlocks(p, E, left, begin, end); }
extern "C" void philoxOf(uint64_t key, uint64_t counter, uint64_t stream, uint32_t* out) {
  const Random128 r = philox(key, counter, stream);
  for (int i = 0; i < 4; ++i) out[i] = r.w[i];
}
extern "C" int threshold(float p) { return dropThreshold(p); }
extern "C" int keepsOf(uint32_t word, int odd, int drop) {
  Random128 r = {{word, word, word, word}};
  return keeps(r, 4 + odd, (uint32_t)drop * 65536u - 1, drop == 0);
}
extern "C" uint32_t divided(uint32_t n, uint32_t d) { return quotient(n, divisionOf(d)); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("chunks")
    (d / "chunks.cc").write_text(SOURCE)
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "the library's build needs a host compiler too"
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "chunks.cc"), "-o", str(d / "chunks.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "chunks.so"))
    lib.threshold.argtypes = [ctypes.c_float]
    lib.philoxOf.argtypes = [ctypes.c_uint64] * 3 + [ctypes.POINTER(ctypes.c_uint32)]
    lib.keepsOf.argtypes = [ctypes.c_uint32, ctypes.c_int, ctypes.c_int]
    lib.loaded.argtypes = [ctypes.c_size_t] * 4
    lib.together.argtypes = [ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_size_t, ctypes.c_size_t]
    return lib


@pytest.mark.parametrize("E", [2, 4])
def test_every_byte_of_a_row_is_stored_once(lib, E):
    """And none beside them, every piece on a boundary of its size."""
    for skew in range(0, 16, E):
        for cols in list(range(1, 40)) + [255, 256, 257, 300, 511, 512, 513]:
            for lanes, step in ((8, 8), (16, 16), (32, 32), (32, 31)):
                if lanes < 32 and cols > 8 * lanes:
                    continue
                writer, times = (ctypes.c_int * 8192)(), (ctypes.c_int * 8192)()
                for first in range(0, (cols + 7) // 8, step):
                    lib.storeOf(skew, E, cols, first, lanes, step, writer, times)
                t, end = np.array(times), cols * E
                assert (t[:end] == 1).all() and t[end:].sum() == 0, (skew, cols, step)
                # a lane writes its own chunk and what it took from the next one
                lane = np.arange(end) // (8 * E) % step
                assert all(w in (at, at - 1, step - 1 if at == 0 and step < lanes else at) for w, at in zip(writer[:end], lane))


@pytest.mark.parametrize("E", [2, 4])
def test_loads_stay_inside_the_matrix(lib, E):
    """Every block that is loaded lies between the matrix's first and last
    byte, and a chunk put together from blocks has all of its bytes in loaded ones."""
    for skew in range(0, 16, E):
        for cols in (1, 3, 7, 8, 9, 16, 17, 300):
            for ld in (cols, cols + 1, cols + 3, cols + 8):
                for rows in (1, 2, 5):
                    begin = 4096 + skew
                    end = begin + ((rows - 1) * ld + cols) * E
                    for row in range(rows):
                        start = begin + row * ld * E
                        row_end = start + cols * E
                        for chunk in range((cols + 7) // 8):
                            p, left = start + chunk * 8 * E, cols - chunk * 8
                            got = set()
                            for b in range(8 * E // 16 + 1):
                                block = (p & ~15) + 16 * b
                                if lib.loaded(block, row_end, begin, end):
                                    assert begin <= block and block + 16 <= end
                                    got |= set(range(block, block + 16))
                            if lib.together(p, E, left, begin, end):
                                assert set(range(p, p + min(left, 8) * E)) <= got
                            elif begin + 32 <= p and p + 48 <= end:
                                raise AssertionError("only the matrix's ends are taken one by one")


def test_philox_known_answers(lib):
    """The published test vectors (all bits 0, all 1, digits of pi), and the oracle's form."""
    ones = (1 << 64) - 1
    out = (ctypes.c_uint32 * 4)()
    for key, counter, stream, want in (
            (0, 0, 0, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            (ones, ones, ones, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            (0x299F31D0A4093822, 0x85A308D3243F6A88, 0x0370734413198A2E, (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        lib.philoxOf(key, counter, stream, out)
        assert tuple(out) == want == tuple(o.philox(key, counter, stream))
    g = np.random.default_rng(0)
    for _ in range(50):
        args = [int(x) for x in g.integers(0, 1 << 63, 3)]
        lib.philoxOf(*args, out)
        assert list(out) == o.philox(*args)


def test_threshold_and_keeping(lib):
    assert [lib.threshold(p) for p in (0.0, 2.0 ** -18, 2.0 ** -17, 0.1, 0.5, 1 - 2.0 ** -17, 1.0)] == [0, 0, 1, 6554, 32768, 65536, 65536]
    for drop in (0, 1, 2, 6554, 32768, 65535, 65536):
        for half in (0, 1, 2, 6553, 6554, 6555, 32767, 32768, 65534, 65535):
            for other in (0, 65535):
                assert lib.keepsOf(other << 16 | half, 0, drop) == (half >= drop), (drop, half)
                assert lib.keepsOf(half << 16 | other, 1, drop) == (half >= drop), (drop, half)


def test_division_by_a_product(lib):
    g = np.random.default_rng(2)
    for d in [2, 3, 5, 7, 17, 31, 32, 33, 126, 512, 513, 1000, 12345, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, (1 << 26) - 1]:
        top = (1 << 31) - 1
        for n in [0, 1, d - 1, d, d + 1, top - 1, top, top // d * d, top // d * d - 1] + [int(x) for x in g.integers(0, top, 200)] + \
                [q * d - 1 for q in map(int, g.integers(1, top // d + 1, 200))]:
            assert lib.divided(n, d) == n // d, (d, n)
