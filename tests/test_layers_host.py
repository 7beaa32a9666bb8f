"""Host-side plans of the expert-layer operators, from a small program that includes them (compiled here, no GPU needed)."""
import os
import subprocess
import textwrap

import pytest

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
