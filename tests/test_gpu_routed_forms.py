"""GPU checks of the routed kernels' forms that few shapes reach, against the fp64 oracle with the bounds of
test_gpu_routed.py: the 128 x 512 tile of the grouped products, the eight waves that share a deep K, fp32 rows
combined to 16 bits past the caches."""
import numpy as np
import pytest

from gpu_common import require_gpu, torch_mod
from test_gpu_routed import _announce, _check_grouped, _dtype, _ids, _routed, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _kernel(rows, K, N, groups, g):
    import weight_only_int4_w4a16_amd as w4
    name = w4.grouped_kernel_name(rows, K, N, groups, g)
    _announce(f"grouped rows={rows} K={K} N={N} groups={groups} g={g} {name}")
    return name


@pytest.mark.parametrize("act,fmt,g,K,glu", [
    ("f16", "asym", 32, 1440, False), ("bf16", "asym", 64, 1472, False), ("bf16", "sym", 32, 1440, True),
    ("f16", "nf4", 64, 1472, True), ("bf16", "nf4", 32, 1440, True), ("f16", "sym", 128, 1536, False),
])
def test_grouped_on_the_128_row_tile(act, fmt, g, K, glu):
    """Part-filled tiles, a ragged last block of K and column tile, rows of no group; both ways to read x."""
    assert _kernel(2100, K, 7584, 2, g) == "w4a16_grouped_128x512"
    _check_grouped(2100, 1, 2, K, 7584, g, act, fmt, glu, gather=fmt != "asym")


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,g,K", [("asym", 32, 8224), ("asym", 64, 8256), ("sym", 128, 8320), ("sym", 32, 8224),
                                     ("nf4", 64, 8256), ("nf4", 32, 8224)])
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_deep_k_over_eight_waves(act, fmt, g, K, glu):
    """65 blocks of K, the last ragged, in eight shares that are not all as long."""
    assert _kernel(9, K, 96, 3, g) == "w4a16_grouped_16x64"
    _check_grouped(9, 1, 3, K, 96, g, act, fmt, glu, gather=not glu)


@pytest.mark.parametrize("width", [4096, 4001])  # whole cache lines and not
@pytest.mark.parametrize("to", ["f16", "bf16"])
def test_combine_of_fp32_rows_past_the_caches_to_16_bits(to, width):
    import weight_only_int4_w4a16_amd as w4
    torch = torch_mod()
    _announce(f"combine 2100x2 width={width} f32 -> {to}")
    ids = _ids(2100, 2, 5, 3)
    r, (offsets, _, _) = _routed(ids, 5)
    ys, _ = _rows((4200, width), "f32", 4)
    ys[int(offsets[-1]):] = float("nan")
    w = torch.rand(2100, 2, device="cuda")
    y32 = w4.combine(ys, r, w)
    assert np.isfinite(y32.cpu().numpy()).all()
    assert torch.equal(w4.combine(ys, r, w, out_dtype=_dtype(to)), y32.to(_dtype(to)))
