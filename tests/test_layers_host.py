"""Host-side plans of the expert-layer operators, from a small program that includes them (compiled here, no GPU needed),
and the generator that the dropout tests take their masks from."""
import random
import subprocess
import textwrap

import numpy as np
import pytest
from test_layers_gpu import philox

from newton_schulz_quintic_gb300 import build

# lines of numbers in: rows, cols, backward, wide, bytes of x's and y's values, which of x y dz dr pre are there (a mask)
PROGRAM = textwrap.dedent("""
    #include <cstdio>
    #include "ns_block_norm.cuh"
    using namespace ns::block_norm;
    int main() {
      long rows, cols;
      int backward, wide, xe, ye, mask;
      while (std::scanf("%ld %ld %d %d %d %d %d", &rows, &cols, &backward, &wide, &xe, &ye, &mask) == 7) {
        NormParams p{};
        const void *here = reinterpret_cast<const void *>(0x1000);
        p.rows = rows;
        p.cols = static_cast<int>(cols);
        p.x = mask & 1 ? here : nullptr;
        p.y = mask & 2 ? here : nullptr;
        p.dz = mask & 4 ? here : nullptr;
        p.dr = mask & 8 ? here : nullptr;
        p.pre = mask & 16 ? here : nullptr;
        p.ld_x = p.ld_y = p.ld_dz = p.ld_dr = cols;
        const Shape s(p, backward, wide, xe == 2 ? ns::kBF16 : ns::kF32, ye == 2 ? ns::kBF16 : ns::kF32, 152);
        std::printf("%d %d %d %d %d %d %d", s.threads, s.packs, s.rows, s.per_sm, s.smem, s.ring.slots, s.ring.slot_bytes);
        for (int q = 0; q < kStreams; ++q) std::printf(" %d", s.ring.row_bytes[q]);
        std::printf("\\n");
      }
      return 0;
    }
""")


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    at = tmp_path_factory.mktemp("shape")
    src, exe = at / "shape.cu", at / "shape"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, str(src), "-o", str(exe)], check=True, capture_output=True)

    def go(cases):
        r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True)
        assert r.returncode == 0, r.returncode
        rows = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
        assert len(rows) == len(cases)
        names = ("threads", "packs", "rows", "per_sm", "smem", "slots", "slot_bytes")
        return [dict(zip(names, v), row_bytes=v[len(names):]) for v in rows]
    return go


X, Y, DZ, DR, PRE = 1, 2, 4, 8, 16
COLS = (1, 8, 127, 256, 2303, 4096, 6144, 8192, 8200, 12288, 16383, 16384)


def test_norm_plans_of_calls_without_rows(shapes):
    # the matrices of such a call may be null pointers
    cases = [(0, cols, b, int(cols % 8 == 0), 2, 2, mask) for cols in COLS for b in (0, 1) for mask in (0, PRE, X, X | Y | PRE)]
    for s in shapes(cases):
        assert s["slots"] >= 1 and 0 <= s["smem"] <= 227 * 1024


def test_norm_plans_fit_the_shared_memory(shapes):
    cases = [(rows, cols, b, wide, xe, ye, mask) for cols in COLS for rows in (1, 7, 5000) for b in (0, 1)
             for wide in ([0, 1] if cols % 8 == 0 else [0]) for xe, ye in ((2, 2), (4, 2), (4, 4))
             for mask in ([X | Y, X | PRE, X | Y | PRE] if not b else [X | Y | DR, X | DZ | DR | PRE, X | Y | DZ | PRE, X | Y | DZ | DR | PRE])]
    for c, s in zip(cases, shapes(cases)):
        # with the kernel's own 2 KB; one slot at least holds what goes through the ring
        assert s["smem"] + 2048 <= 227 * 1024 and 1 <= s["slots"] <= 8, (c, s)
        assert s["smem"] >= s["slots"] * s["slot_bytes"] and s["slot_bytes"] == s["rows"] * sum(s["row_bytes"]), (c, s)
        assert s["threads"] * s["packs"] * 8 >= c[1] and s["threads"] * s["rows"] <= 512, (c, s)


def test_norm_plans_copy_what_is_read(shapes):
    # through the ring: X for the norm of r alone, dZ with pre alone; Y wherever there is room
    cases = [(5000, cols, 1, int(cols % 8 == 0), 2, 2, mask) for cols in COLS for mask in (X | Y | DR, X | Y | DZ | PRE, X | Y | DZ | DR | PRE)]
    for c, s in zip(cases, shapes(cases)):
        x, y, dz, dr = s["row_bytes"]
        assert (x > 0) == bool(c[6] & PRE), (c, s)
        assert y > 0 and (dr == 0 or c[6] & DR) and (dz == 0 or c[6] & PRE), (c, s)


def philox4x32(counter, key):
    """Philox4x32-10 of four counter words and two key words."""
    a, b, c, d = counter
    k0, k1 = key
    m = 0xFFFFFFFF
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32) ^ b ^ k0, q & m, (p >> 32) ^ d ^ k1, p & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return a, b, c, d


def test_the_reference_generator_has_the_published_answers():
    # zeros, ones, and the digits of pi; and the form that the dropout tests compare with is this one
    m = 0xFFFFFFFF
    assert philox4x32((0, 0, 0, 0), (0, 0)) == (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    assert philox4x32((m, m, m, m), (m, m)) == (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)
    assert philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == (
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)
    r = random.Random(1)
    for third in (0, 1):
        for n, seed in [(0, 0), ((1 << 64) - 1, (1 << 64) - 1)] + [(r.getrandbits(64), r.getrandbits(64)) for _ in range(20)]:
            got = philox(np.array([n], np.uint64), seed, third)[0]
            assert tuple(int(v) for v in got) == philox4x32((n & m, n >> 32, third, 0), (seed & m, seed >> 32))
