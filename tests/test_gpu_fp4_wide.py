"""Blocks of 32 along rows so long that their column segments are more than one grid
axis holds (65,535): the packed rows read back bit for bit."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SEGMENTS = 65535
# columns a segment: 4 warps' steps of 4 (bf16) or 2 (float32), a step 256 columns of up to 32 rows, else 64
CASES = [("f32", 1, SEGMENTS * 2048 + 5000), ("bf16", 2, SEGMENTS * 4096 + 8 * 613), ("f32", 33, SEGMENTS * 512 + 1060),
         ("bf16", 2, SEGMENTS * 4096 + 4096)]


@pytest.mark.parametrize("dt,R,C", CASES)
def test_more_segments_than_a_grid_axis(dt, R, C):
    x = torch.empty(R, C, dtype=TYPES[dt], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(C)
    for r in range(R):
        for c in range(0, C, 1 << 26):
            n = min(1 << 26, C - c)
            x[r, c:c + n] = torch.randn(n, generator=g, device="cuda").to(TYPES[dt])
    m = q.qmm_fp4_quantize(x, block=32)
    assert q.last_kernel() == "fp4_quantize_rows"
    y = q.qmm_fp4_dequantize(m, out_dtype=torch.float32)
    last = SEGMENTS * (4 * (4 if dt == "bf16" else 2) * (256 if R <= 32 else 64))
    for r in {0, R // 2, R - 1}:
        # whole blocks: the start, the middle, around the segments' limit, the end
        for c, n in ((0, 4096), (C // 64 * 32, 8192), (last - 8192, 16384), ((C - 5000) // 32 * 32, 6000)):
            want = O.fp4_values(x[r:r + 1, c:c + n].float().cpu().numpy(), 32, False)
            assert np.array_equal(y[r:r + 1, c:c + n].cpu().numpy(), want)
    # everywhere: the nearest code of a block whose largest magnitude is b is within b / 2
    for r in range(R):
        for c in range(0, C, 1 << 25):
            a, b = x[r, c:c + (1 << 25)].float(), y[r, c:c + (1 << 25)]
            assert ((a - b).abs() <= 1.1).all() and (b.abs() <= 8).all()
    del x, y, m
    torch.cuda.empty_cache()
