"""The GEMM's reads of block scales stay inside their arrays, for every tile of
every output width: the row index that the source forms is evaluated here.  (Tiles
are 256 wide, the 128x128 scales have a row per 128 columns: of an odd number of
them the last warps' columns lie outside.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_gb300", "csrc")


def _index():
    """The row of b_sinv that a warp whose columns start at colbase reads."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "gemm.cu")).read())
    m = re.findall(r"const uint32_t btile = \(uint32_t\)(.*?) / 128u;\s*"
                   r"const float \*bt = g\.b_sinv \+ \(int64_t\)btile \* g\.lds_b;", src)
    assert len(m) == 1, m
    return eval(f"lambda colbase, N: {m[0].replace('g.N', 'N')} // 128")


def test_rows_of_the_column_blocks_scales():
    index = _index()
    for N in range(16, 2600, 16):
        bn = 256 if N >= 256 else 128
        rows = -(-N // 128)
        for tn in range(-(-N // bn)):
            for half in (32, 64, 128):  # columns per warp
                for colbase in range(tn * bn, (tn + 1) * bn, half):
                    i = index(colbase, N)
                    assert 0 <= i < rows, f"N {N}: columns from {colbase} read row {i} of {rows}"
                    if colbase < N:
                        assert i == colbase // 128
