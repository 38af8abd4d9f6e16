"""GPU checks of the 8-bit floating point calls at their rarer plans, values and arguments, against the fp64 oracle and with the
bounds of test_gpu_fp8.py (derived there)."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import fp8 as F

from gpu_common import require_gpu, torch_mod
import test_gpu_fp8 as T

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# ------------------------------------------------------------------ pinned tiles

def check_pinned():
    """Products of few rows, where the kernel that quantizes x by itself ends, on whatever tile is pinned."""
    import weight_only_int4_w4a16_amd as w4
    for M, K, N in [(1, 272, 260), (2, 1040, 100), (3, 400, 64), (40, 272, 260)]:
        for halves in (1, 2):
            T._announce(f"pinned {os.environ.get('W4A16_FP8_ROWS')} {M}x{K}x{N} {halves}")
            x, xv = T._rows((M, K), "bf16", M + K)
            xv = F.rows_value(*F.quantize_rows(xv))
            codes, scales, wv = T._weight((), N, K, N, halves=halves)
            f = w4.gemm_fp8 if halves == 1 else w4.gemm_fp8_swiglu
            for kind in ("bf16", "f32"):
                if halves == 1:
                    ref, bound = F.gemm_fp8_ref(xv, wv), T._sum_bound(xv, wv, kind)
                else:
                    ref, bound = T._glu_bound(xv, wv, kind)
                y = f(x, codes, scales, out_dtype=T._dtype(kind))
                T._within(y.cpu().double().numpy(), ref, T._stored(ref, bound, kind), kind)


@pytest.mark.parametrize("rows", [16, 32, 64, 128, 256])
def test_pinned_tiles(rows):
    """The pin is read once a process: a child runs its products."""
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "W4A16_FP8_ROWS": str(rows), "PYTHONPATH": os.pathsep.join([ROOT, here])}
    run = subprocess.run([sys.executable, "-c", "import test_gpu_fp8_calls as t; t.check_pinned()"], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=100)
    print(run.stdout, flush=True)
    assert run.returncode == 0, run.stderr[-3000:]
