"""Host side of gq_embed for the largest counts of tokens (no GPU: the calls run in a process that is shown none, and
end with the error of a launch without a device)."""

import os
import subprocess
import sys

import pytest

import block_quantized_matvec_gq_gb300 as gq
from block_quantized_matvec_gq_gb300 import build as gqbuild

CALL = """
import ctypes, sys
import block_quantized_matvec_gq_gb300 as gq
M, K = int(sys.argv[1]), int(sys.argv[2])
print(gq.lib().gq_embed(1, 1 << 20, 1 << 20, ctypes.c_float(1.0), 1 << 20, K, 2, 1, K, M, None))
"""


@pytest.mark.parametrize("M,K", [(1, 32), ((1 << 31) - 30000, 32), ((1 << 31) - 100, 32), ((1 << 31) - 1, 32), ((1 << 31) - 1, 1 << 24)])
def test_any_count_of_tokens_divides_into_warps(M, K):
    gqbuild.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    root = os.path.dirname(os.path.dirname(os.path.abspath(gq.__file__)))
    r = subprocess.run([sys.executable, "-c", CALL, str(M), str(K)], capture_output=True, text=True, env=env, cwd=root, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert int(r.stdout) == gq.GQ_ERR_CUDA
