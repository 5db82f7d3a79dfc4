"""What norm.hip promises the compiler about addresses, read from the device code's intermediate form as it is compiled
here: a row of 8-bit values ends in a piece that may start at any byte where its columns are no multiple of a piece, so its
stores must not be declared aligned to words. Runs without a GPU."""
import os
import re
import subprocess

import pytest

from collective_window_put_amd import build

ANY, WHOLE, STREAM = 0, 1, 2  # a kernel's way to take rows: of any length; of whole pieces; those past the caches


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{(type, threads to a row, pieces, norm, mode): body} of k_rows."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    to = tmp_path_factory.mktemp("ir") / "norm.ll"
    flags = ["-O1" if f == "-O3" else f for f in build.FLAGS]
    subprocess.run([build.HIPCC, *flags, "--cuda-device-only", "-S", "-emit-llvm", os.path.join(build.CSRC, "norm.hip"),
                    "-o", str(to)], check=True, capture_output=True)
    got = {}
    for m in re.finditer(r"^define [^\n]*@\S*k_rowsILi(\d+)ELi(\d+)ELi(\d+)ELb(\d)ELi(\d)E[^\n]*\n(.*?)^}", to.read_text(), flags=re.S | re.M):
        got[tuple(map(int, m.groups()[:5]))] = m.group(6)
    return got


def _stores(body, kind):
    return [int(a) for a in re.findall(r"store " + re.escape(kind) + r" [^\n]*, align (\d+)", body)]


def test_ends_of_rows_in_8_bits_may_lie_anywhere(kernels):
    # from bf16 alone a store of two words is one of eight values; the norm's own outputs and the row's zeros are others
    seen = 0
    for (dtype, _, _, norm, mode), body in kernels.items():
        if dtype != 1 or norm:
            continue
        at = _stores(body, "<2 x i32>") + _stores(body, "i64")
        if mode == ANY:
            assert at and set(at) == {1}, at
        else:
            assert at and set(at) <= {4, 8, 16}, at  # from 16 bytes' multiples: words
        seen += mode == ANY
    assert seen >= 6
