"""The product's own index functions (csrc/mxfp4_product.cuh, csrc/mxfp4.cuh), compiled for the host: the cut of
an expert's rows into tiles up to the largest row count, and the packed weights' layout."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_routed_sqrt_b200", "csrc")

PROGRAM = """
#include <cstdio>
#include "mxfp4_product.cuh"
int main() {
    for (int r = 0; r < ds4::MX_TM; ++r)
        for (int b = 0; b < ds4::MX_TK / ds4::MX_BLOCK; ++b)
            printf("at %d %d %u %u\\n", r, b, ds4::mx_code_off(r, b), ds4::mx_scale_off(r, b));
    int rows, NT;
    while (scanf("%d %d", &rows, &NT) == 2) {
        const int tiles = ds4::mx_row_tiles(rows, NT);
        printf("cut %d %d %d %d\\n", rows, NT, tiles, tiles > 0 ? ds4::mx_tile_rows(rows, tiles, NT) : 0);
    }
}
"""
ROWS = [0, 1, 15, 16, 17, 31, 32, 33, 191, 192, 193, 1920, 1921, 1936, 4097, 65535, 8 << 20, (1 << 31) - 193, (1 << 31) - 192,
        (1 << 31) - 191, (1 << 31) - 32, (1 << 31) - 31, (1 << 31) - 1]


@pytest.fixture(scope="module")
def printed(tmp_path_factory):
    where = tmp_path_factory.mktemp("layout")
    source, program = str(where / "layout.cu"), str(where / "layout")
    with open(source, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "--expt-relaxed-constexpr", "-I", CSRC,
                    "-o", program, source], check=True, capture_output=True)
    asked = "\n".join("%d %d" % (r, nt) for nt in (32, 192) for r in ROWS)
    lines = subprocess.run([program], input=asked, check=True, capture_output=True, text=True).stdout.split("\n")
    return [line.split() for line in lines if line]


def test_rows_are_cut_into_equal_tiles(printed):
    cuts = [[int(v) for v in line[1:]] for line in printed if line[0] == "cut"]
    assert len(cuts) == 2 * len(ROWS)
    for rows, NT, tiles, per in cuts:
        assert tiles == -(-rows // NT)
        if rows:
            assert per % 16 == 0 and 16 <= per <= NT
            assert (tiles - 1) * per < rows <= tiles * per       # no tile empty, no row left


def test_packed_tile_holds_every_code_and_scale_once(printed):
    at = [[int(v) for v in line[1:]] for line in printed if line[0] == "at"]
    assert sorted(a[2] for a in at) == list(range(0, 16384, 16))
    assert sorted(a[3] for a in at) == list(range(16384, 17408))
    for r, b, code, scale in at:
        assert code == r * 128 + 16 * (b ^ (r % 8))
        assert scale == 16384 + b // 4 * 512 + r % 32 * 16 + r // 32 * 4 + b % 4
