"""The largest sizes that the window attention takes (no GPU): the bound itself with plain numbers, and the calls that reach it."""
import ctypes
import os
import subprocess

import pytest

from test_attention_abi import WINDOW, _window_good
from test_ops_abi import F, kda  # noqa: F401  (kda: the fixture)

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_kda_gb300", "csrc")


def test_the_edges_of_the_bound(tmp_path):
    """More tokens than 2^31 - 513 come with plans too long to be built here."""
    cases = [(2 ** 31 - 513, 1, 1, 1), (2 ** 31 - 512, 1, 1, 0), (2 ** 31 - 1, 1, 1, 0), (128, 7, 2 ** 27 - 1, 1), (128, 7, 2 ** 27, 0),
             (127, 8, 2 ** 27 - 1, 1), (1, 2 ** 30 - 1, 1, 1), (1, 2 ** 30, 1, 0), (2 ** 31 - 513, 1, 64, 1), (2 ** 31 - 513, 1, 65, 0), (2 ** 30, 1, 128, 0),
             (2 ** 30, 2 ** 30, 2 ** 31 - 1, 0)]
    source, binary = tmp_path / "limits.cpp", tmp_path / "limits"
    source.write_text('#include <cstdio>\n#include "window_limits.h"\nint main() {\n'
                      + "".join(f'std::printf("%d ", kda::window_sizes_ok({t}LL, {n}LL, {h}LL));\n' for t, n, h, _ in cases) + "}\n")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(source), "-o", str(binary)], check=True)
    got = subprocess.run([str(binary)], check=True, capture_output=True, text=True).stdout.split()
    assert got == [str(want) for *_, want in cases]


@pytest.mark.parametrize("sequences,refused", [(32, False), (33, True)])
def test_calls_with_more_blocks_than_a_grid_has(sequences, refused, kda):  # noqa: F811
    """Sequences of one token and 33,554,400 heads of 64: 32 are below 2^30 blocks and go on to the next check (an output that is not there)."""
    plan = kda.kda_plan_segments(list(range(sequences + 1)), 1)
    _, good = _window_good(kda)
    H = 33554400
    good.update(plan=plan.ctypes.data_as(ctypes.c_void_p), H=H, Hk=1, ldq=H * 64, o=None, ldo=H * 64, lse=F)
    want = kda.KDA_ERR_UNSUPPORTED if refused else kda.KDA_ERR_INVALID_ARG
    assert kda._lib.kda_window_attention_forward(*(good[n] for n in WINDOW + "o ldo lse stream".split())) == want
    good.update(do=F, lddo=H * 64, dq=F, lddq=H * 64, dk=F, lddk=64, dv=F, lddv=64, ws=F, ws_bytes=2 ** 62)
    names = WINDOW + "o ldo lse do lddo dq lddq dk lddk dv lddv ws ws_bytes stream".split()
    assert kda._lib.kda_window_attention_backward(*(good[n] for n in names)) == want
