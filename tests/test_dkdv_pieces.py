"""How key tiles are cut into pieces for the dK/dV kernel (fa_kernels.h, a host function): by the number
of the device's SMs, within the workspace's room, and only where the longest CTA gets less to do."""
import os
import shutil
import subprocess

import pytest

import io_aware_exact_07_gb300 as fa

CSRC = os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "csrc")
PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "fa_kernels.h"
int main(int, char** v) {
  const int sms = atoi(v[1]);
  printf("%d %d\\n", fa::kMaxPieces, fa::kMinCutTiles);
  for (long long k = 1; k <= 320; k += k < 8 ? 1 : 13)
    for (long long q = 1; q <= 3000; q = q < 12 ? q + 1 : q * 3 / 2)
      printf("%lld %lld %d\\n", k, q, fa::dkdv_pieces(k, q, sms));
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    d = tmp_path_factory.mktemp("pieces")
    (d / "p.cu").write_text(PROGRAM)
    out = str(d / "p")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17",
                        "--expt-relaxed-constexpr", "-I", CSRC, "-o", out, str(d / "p.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


@pytest.mark.parametrize("sms", [1, 20, 76, 152, 160, 400])
def test_pieces(program, sms):
    lines = subprocess.run([program, str(sms)], capture_output=True, text=True, check=True).stdout
    (most, least), *rows = [[int(x) for x in r.split()] for r in lines.splitlines()]

    def steps(k, q, s):  # of the longest CTA: query tiles, 3 per unit, 6 for the merge
        return -(-k * s // sms) * (-(-q // s) + 3) + (6 if s > 1 else 0)
    cut = 0
    for k, q, s in rows:
        could = [1] + [x for x in range(2, most // k + 1) if 2 * x <= q and q >= least]
        assert s in could
        assert steps(k, q, s) == min(steps(k, q, x) for x in could), (k, q, s)
        if k >= sms:  # cut at most where the last round of units is short
            assert s == 1 or steps(k, q, s) < steps(k, q, 1)
        cut += s > 1
    assert cut > 0 or sms == 1
