"""The rotation's angles in float32, read off from vectors (1, 0): the result is (cos, sin) itself.

Bound: the reduced angle lies in [-1/4, 1/4] half turns and is rounded to float32 once (2^-27 half turns, pi 2^-27
radians, passed on by the derivative), sincospif is good to one unit (2^-23 relative), the double angle to 2^-50 of itself."""
import math

import numpy as np
import pytest
import torch

from test_gpu_chunk import F32, _ctx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("theta", [10000.0, 1000000.0, 0.25])
@pytest.mark.parametrize("start", [0, 100000, 1 << 20, (1 << 31) - 4000])
def test_angles_are_good_to_float32(d, theta, start):
    T = 3000
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + start
    q = torch.zeros(T, 4, d, device="cuda")
    q[..., : d // 2] = 1.0
    kv = torch.zeros(T, 2, d, device="cuda")
    pool = torch.zeros(1, 2, 2, 2, 16, d, device="cuda")
    with _ctx(4, 2, d, F32, n=1, pages=1, theta=theta) as ctx:
        out = ctx.qk_norm_rope(q, kv, kv, pool, 0, pos, torch.full_like(pos, -1)).cpu().double().numpy()
        assert ctx.device_error() == (0, 0)
    assert (out == out[:, :1]).all()
    ang = np.arange(start, start + T, dtype=np.longdouble)[:, None] * np.longdouble(theta) ** (
        -2 * np.arange(d // 2, dtype=np.longdouble) / d)
    cos, sin = np.cos(ang), np.sin(ang)
    lo, hi = out[:, 0, : d // 2], out[:, 0, d // 2:]
    far = np.abs(ang) * 2.0 ** -50
    for got, want, slope in ((lo, cos, sin), (hi, sin, cos)):
        bound = (math.pi * 2.0 ** -27) * np.abs(slope) + 2.0 ** -23 * np.abs(want) + far + 1e-12
        over = float((np.abs(got - want) / bound).max())
        assert over <= 1, over
