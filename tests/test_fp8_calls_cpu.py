"""CPU checks of the 8-bit floating point calls as a whole: what sizes a call, makes its operands and launches it has to ask
the same plan, sizes and types are refused where the launches end, and sizes of scratch are public (nothing is launched)."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, BF16, F32, E4M3 = 0, 1, 2, 3

SIZES = [(1, 4096, 4096), (2, 256, 64), (1, 33024, 48), (2, 16400, 40)]

PINNED = """
import json, sys
from weight_only_int4_w4a16_amd import binding
L = binding.lib()
out = []
for M, K, N in json.loads(sys.argv[1]):
    for glu in (0, 1):
        out.append([M, K, N, glu, L.w4a16_fp8_kernel_name(M, K, N, glu).decode()] +
                   [L.w4a16_fp8_workspace_bytes(M, K, N, 1, glu, o) for o in (1, 2)])
print(json.dumps(out))
"""


@pytest.mark.parametrize("rows", [16, 32, 64, 128, 256])
def test_pinned_tiles_have_codes_to_read(rows):
    """W4A16_FP8_ROWS pins the row tile (read once a process, so each pin has one of its own). A tile reads codes, which a 16-bit
    x has in the workspace; only the sixteen-row kernel quantizes one or two rows by itself."""
    env = {**os.environ, "W4A16_FP8_ROWS": str(rows)}
    run = subprocess.run([sys.executable, "-c", PINNED, json.dumps(SIZES)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr
    for M, K, N, glu, name, bf16, f32 in json.loads(run.stdout.splitlines()[-1]):
        tile = {16: "16", 32: "32x128", 64: "64x128", 128: "128x256", 256: "256x256"}[rows]
        assert name == f"w4a16_fp8_{tile}"
        codes = M * K + 4 * M * -(-K // 128)
        if rows > 16:
            assert bf16 >= codes, (M, K, N, glu)
        if 16 < rows < 256:  # 32-bit results have no tile of 256 rows: the pin does not hold for them
            assert f32 >= codes, (M, K, N, glu)


# ------------------------------------------------------------------ where the launches end

@pytest.fixture(scope="module")
def L():
    from weight_only_int4_w4a16_amd import binding
    return binding.lib()


OK, ARG, UNSUPPORTED = 0, 1, 2
P, Q = 1 << 20, (1 << 20) + 4096  # aligned placeholder addresses, never dereferenced


@pytest.mark.parametrize("M,K,status", [
    # a wave takes 512 values of two rows: 2^24 workgroups of 256 threads are one too many
    ((1 << 27) - 1, 16, UNSUPPORTED), ((1 << 27) - 7, 128, UNSUPPORTED), ((1 << 27) - 7, 512, UNSUPPORTED), ((1 << 27) - 8, 512, ARG),
    (1 << 26, 528, UNSUPPORTED), ((1 << 26) - 8, 1024, ARG), (1, (1 << 31) - 16, ARG), (2 ** 31 - 1, 16, UNSUPPORTED),
])
def test_rows_end_where_their_launch_does(L, M, K, status):
    # (no address: sizes are looked at first)
    assert L.w4a16_quantize_fp8(None, M, K, BF16, 2 * P, Q, None) == status


@pytest.mark.parametrize("M,K,status", [
    ((1 << 31) - 128, 128, ARG), ((1 << 30) + 1, 256, UNSUPPORTED), (1 << 27, 1024, ARG), (1 << 27, 2048, UNSUPPORTED),
])
def test_tiles_end_where_their_launch_does(L, M, K, status):
    assert L.w4a16_quantize_fp8_columns(None, M, K, BF16, 2 * P, Q, None) == status
    assert L.w4a16_quantize_fp8_weight(None, M, K, BF16, 2 * P, Q, None, None, None) == status


@pytest.mark.parametrize("M,K,N,xdt,glu,odt,status", [
    # one kernel: its own grid alone counts
    (1 << 17, 16, 1 << 17, BF16, 0, BF16, ARG), (1 << 17, 16, 1 << 17, BF16, 0, F32, ARG), (1 << 18, 128, 1 << 17, E4M3, 1, BF16, ARG),
    ((1 << 27) - 8, 128, 64, E4M3, 0, BF16, ARG), ((1 << 29) - 1, 128, 64, E4M3, 0, BF16, ARG),
    # a second one, of 512 columns a wave, quantizes h from tiles of 64 columns
    (1 << 26, 16, 64, E4M3, 1, E4M3, UNSUPPORTED),
    # rows quantized in the call
    ((1 << 27) - 1, 128, 64, BF16, 0, BF16, UNSUPPORTED), (1 << 29, 128, 64, E4M3, 0, BF16, UNSUPPORTED),
])
def test_products_end_where_their_launches_do(L, M, K, N, xdt, glu, odt, status):
    assert L.w4a16_gemm_fp8(None, xdt, None, M, K, N, 2 * P, Q, glu, 3 * P, odt, None, None, 0, None) == status


def test_grouped_products_end_where_their_launches_do(L):
    def call(tokens, K, N, glu, odt):
        return L.w4a16_gemm_fp8_grouped(None, E4M3, None, Q, tokens, 1, 3, 0, K, N, 2 * P, Q, glu, 3 * P, odt, None, None, 0, None)
    # (the plan's placeholder passes, x's missing address does not)
    assert call(1 << 25, 128, 1024, 0, BF16) == ARG
    assert call(1 << 26, 128, 1024, 1, E4M3) == ARG  # tiles of 128 columns quantize h themselves
    assert call(1 << 26, 128, 8192, 0, BF16) == UNSUPPORTED


# ------------------------------------------------------------------ sizes of scratch

def test_scratch_of_types_that_are_refused():
    import torch
    import weight_only_int4_w4a16_amd as w4
    for dtype in (torch.float32, torch.float64, torch.uint8, torch.float8_e5m2, None):
        for quantized in (False, True):
            with pytest.raises(w4.W4A16Error, match="dtype") as e:
                w4.fp8_workspace_bytes(40, 256, 64, dtype, quantized=quantized)
            assert e.value.status == ARG
            with pytest.raises(w4.W4A16Error, match="dtype"):
                w4.fp8_grouped_workspace_bytes(20, 2, 3, 256, 64, dtype, quantized=quantized)
    assert w4.fp8_workspace_bytes(40, 256, 64, torch.float16) >= 40 * 256


def test_scratch_of_every_call_that_takes_a_workspace(L):
    import torch
    import weight_only_int4_w4a16_amd as w4
    for tokens, topk, groups, K, N in [(1, 1, 1, 256, 64), (20, 2, 3, 512, 256), (600, 4, 8, 2048, 1408)]:
        for x, dt in ((torch.bfloat16, BF16), (torch.float16, F16), (torch.float8_e4m3fn, E4M3)):
            for gather in (0, 1):
                for glu, quantized in ((0, 0), (1, 0), (1, 1)):
                    outs = (E4M3,) if quantized else (F32, BF16 if dt == E4M3 else dt)
                    want = max(L.w4a16_fp8_grouped_workspace_bytes(tokens, topk, groups, gather, K, N, dt, glu, o) for o in outs)
                    have = w4.fp8_grouped_workspace_bytes(tokens, topk, groups, K, N, x, bool(glu), bool(quantized), bool(gather))
                    assert have == want and (dt == E4M3 or have >= tokens * (1 if gather else topk) * K)
        M = tokens * topk
        assert w4.fp8_backward_workspace_bytes(M, K, N) == L.w4a16_fp8_backward_workspace_bytes(M, K, N) > M * (2 * N + K)
        have = w4.fp8_grouped_backward_workspace_bytes(tokens, topk, groups, K, N)
        assert have == L.w4a16_fp8_grouped_backward_workspace_bytes(tokens, topk, groups, K, N) > M * (2 * N + K)
    assert w4.fp8_backward_workspace_bytes(2 ** 32 + 4, 256, 64) == 0  # not the size of 4 rows
    assert w4.fp8_grouped_backward_workspace_bytes(2 ** 32 + 4, 1, 1, 256, 64) == 0
    assert w4.fp8_grouped_workspace_bytes(2 ** 32 + 4, 1, 1, 256, 64, torch.bfloat16) == 0


@pytest.mark.parametrize("M,K,N,glu", [(40, 1 << 23, 64, 0), (40, 1 << 15, 1 << 17, 1), (1, 1 << 23, 64, 0), ((1 << 29) - 1, 256, 64, 0)])
def test_refused_sizes_have_no_scratch_and_no_kernel(L, M, K, N, glu):
    for xdt, odt in ((E4M3, BF16), (BF16, BF16), (BF16, F32)):
        assert L.w4a16_gemm_fp8(P, xdt, Q, M, K, N, 2 * P, Q, glu, 3 * P, odt, None, None, 0, None) == UNSUPPORTED
        assert L.w4a16_fp8_workspace_bytes(M, K, N, xdt, glu, odt) == 0
        if M < 1 << 20:
            assert L.w4a16_gemm_fp8_grouped(P, xdt, Q, Q, M, 1, 2, 0, K, N, 2 * P, Q, glu, 3 * P, odt, None, None, 0, None) == UNSUPPORTED
            assert L.w4a16_fp8_grouped_workspace_bytes(M, 1, 2, 0, K, N, xdt, glu, odt) == 0
    assert L.w4a16_fp8_kernel_name(M, K, N, glu) == b"none"
    if not glu:
        assert L.w4a16_fp8_backward_workspace_bytes(M, N, K) == 0
        if M < 1 << 20:
            assert L.w4a16_fp8_grouped_backward_workspace_bytes(M, 1, 2, N, K) == 0
