"""CPU test of how attention over caches with scales cuts its work: the cases of
the GPU tests take the ways that they are there for."""
import os
import subprocess

import pytest

import test_gpu_kv_scaled as first
import test_gpu_kv_scaled_more as more
from lossless_bf16_tensor_amd import build

PROGRAM = r"""
#include "kv_attend.h"
#include <stdlib.h>
int main(int n, char **v)
{
    for (int i = 1; i + 6 < n; i += 7) {
        unsigned x[7];
        for (int k = 0; k < 7; k++) x[k] = (unsigned)strtoul(v[i + k], nullptr, 10);
        const uzip_kv::Plan a = uzip_kv::make_plan(x[0], x[1], x[2], x[3], x[4], x[5], x[6], true);
        printf("%s\n", a.shared ? "shared" : a.walks ? "walks" : a.flat ? "runs" : "whole");
    }
}
"""


@pytest.fixture(scope="module")
def ways(tmp_path_factory):
    """ways(cases) of [(sequences, tokens, heads, kv heads, head dim, cache tokens, layout)]."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("no compiler")
    at = tmp_path_factory.mktemp("plans")
    (at / "plans.hip").write_text(PROGRAM)
    subprocess.run([build.HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-std=c++17", "-w", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"),
                    str(at / "plans.hip"), "-o", str(at / "plans")], check=True, capture_output=True)

    def call(cases):
        args = []
        for B, T, hq, H, D, S, layout in cases:
            page = int(layout[5:]) if layout.startswith("paged") else 1
            args += [str(x) for x in (B, H, D, -(-S // page) * page, T, hq, int(D % 16 == 0))]
        return subprocess.run([str(at / "plans"), *args], check=True, capture_output=True, text=True).stdout.split()
    return call


def test_many_rows_share_keys(ways):
    assert set(ways([(B, T, hq, H, D, S, layout) for B, T, hq, H, D, S, _, _, _, layout in first.SHARED])) == {"shared"}


def test_long_ragged_batches_take_shares(ways):
    assert set(ways([(B, T, hq, H, D, S, layout) for B, T, hq, H, D, S, _, _, _, layout, _ in more.WALKS])) == {"walks"}


def test_every_way_is_taken(ways):
    mark, = (m for m in first.test_many_sequences.pytestmark if m.name == "parametrize")
    assert set(ways([(B, T, hq, H, D, S, layout) for B, T, hq, H, D, S, _, _, layout in mark.args[1]])) == {"walks", "runs", "whole"}
