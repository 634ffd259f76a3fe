"""Where the parts of embed_backward's workspace lie, on the CPU: each on the boundary
that its accesses need, none in another, all within the bytes that the query gives, for
every workspace that a caller may give (on 16 bytes) and for fewer positions too.
The layout is the library's own header."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q5_lm_head_gb300", "csrc")
SHIM = """
#include "embed_space.h"
extern "C" void space(int64_t at, int64_t n, int64_t v, int k, int sms, int64_t *o) {
  const muse::BackwardSpace s = muse::backward_space(n, v, k, sms);
  const int64_t base = reinterpret_cast<int64_t>(muse::space_base(reinterpret_cast<void *>(at)));
  const int64_t all[] = {base, base + (int64_t)s.order, base + (int64_t)s.sorted, base + (int64_t)s.span, base + (int64_t)s.used,
                         base + (int64_t)s.done, base + (int64_t)s.part, (int64_t)s.bytes, s.chunk, s.chunks};
  for (int i = 0; i < 10; ++i) o[i] = all[i];
}
"""


@pytest.fixture(scope="module")
def space(tmp_path_factory):
    at = tmp_path_factory.mktemp("space")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(at / "shim.cpp"), "-o", str(at / "shim.so")], check=True)
    lib = ctypes.CDLL(str(at / "shim.so"))
    i64, i32 = ctypes.c_int64, ctypes.c_int
    lib.space.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(i64)]

    def ask(work, n, v, k, sms=152):
        out = (i64 * 10)()
        lib.space(work, n, v, k, sms, out)
        return list(out)
    return ask


@pytest.mark.parametrize("k", [256, 1024, 6656, 332800, 1 << 20])
@pytest.mark.parametrize("off", [0, 16, 32, 48, 240])
def test_parts_lie_on_their_boundaries(space, off, k):
    work, v, tiles = (1 << 40) + off, 202048, k // 256
    for n in (0, 1, 2, 3, 4, 5, 31, 301, 4099, 10944, 10945, 16384, 100001, 10 ** 6):
        *at, size, chunk, chunks = space(work, n, v, k)
        words = [1, n, n, 2 * n, (v + 31) // 32, chunks * tiles, chunks * 2 * k]
        for begin, many, each in zip(at, words, (4, 4, 4, 8, 4, 4, 32)):
            assert begin % each == 0, (n, begin, each)
        for (begin, many), after in zip(zip(at, words), at[1:] + [work + size]):
            assert work <= begin and begin + 4 * many <= after
        for fewer in (n // 2, n - 1, n * 2 // 3):
            if fewer >= 0:
                *b, _, _, c = space(work, fewer, v, k)
                assert b[-1] + 4 * c * 2 * k <= work + size
