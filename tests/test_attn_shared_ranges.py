"""The join of gdn_attn_decode_shared reads no slot outside the workspace,
whatever the words hold in which the first kernel notes a job's ranges (after a
wait that gave up they are the caller's memory).  The library's own function,
compiled for the host."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_linear_06_gb300", "csrc")
MIN, MAX = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def ranges_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("ranges")
    src, so = d / "r.cpp", d / "r.so"
    src.write_text('#include "gdn_attn_ranges.h"\n'
                   'extern "C" void ranges_of(int a, int b, int n, int* out) {\n'
                   '  const gdn::Ranges r = gdn::ranges_of(a, b, n);\n'
                   '  out[0] = r.first;\n  out[1] = r.count;\n}\n')
    subprocess.run([shutil.which("g++") or "g++", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)], check=True)
    fn = ctypes.CDLL(str(so)).ranges_of

    def call(a, b, n):
        out = (ctypes.c_int * 2)()
        fn(a, b, n, out)
        return out[0], out[1]
    return call


@pytest.mark.parametrize("shares", [1, 2, 76, 80])
def test_any_words_give_shares_that_exist(ranges_of, shares):
    words = [MIN, MIN + 1, -1000, -1, 0, 1, shares // 2, shares - 1, shares, shares + 1, 10 ** 6, MAX - 1, MAX]
    for a in words:
        for b in words:
            first, count = ranges_of(a, b, shares)
            assert 0 <= first < shares and 0 <= count and first + count <= shares
            # the slots of job j are j + share, of which the workspace has jobs + shares
            for job, jobs in ((0, 1), (6, 7)):
                assert count == 0 or job + first + count <= jobs + shares


@pytest.mark.parametrize("shares", [1, 2, 76, 80])
def test_noted_ranges_are_taken_as_they_are(ranges_of, shares):
    for a in range(shares):
        for b in range(a, shares):
            assert ranges_of(a, b, shares) == (a, b - a + 1)
    assert ranges_of(0, -1, shares) == (0, 0)      # a job without a range


def test_the_join_reads_the_noted_words_through_it():
    src = open(os.path.join(CSRC, "gdn_attn_shared.cu")).read()
    join = src[src.index("attn_shared_join(const"):]
    join = join[:join.index("cuTensorMapEncodeTiled")]
    assert join.count("p.span[") == 2 and join.count("ranges_of(") == 2
