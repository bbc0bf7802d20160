"""The products at the ends of their ranges, on the GPU: what is far from 0, limits of
sizes, small differences of precision.  Bounds are derived beside each test; a
rounding to type t is off by at most U[t] relative.
"""

import math

import pytest

from test_gpu_products import ACTS, ABC, DEV, M, SUM, T, U, act64, gen, orth64, real, slope64, types, whole, wide  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = [8.0, 11.9, 12.1, 19.9, 20.1, 40.0, 89.0, 104.0, 199.0, 201.0, 1e3, 6e4, 1e6, 1e10, 1.2e13, 3e13, 1e16, 1.8e19, 3e19, 1e25, 1e30, 3e38, math.inf]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("copies", [1, 40])
def test_slopes_far_from_zero(T, M, types, dt, act, copies):  # noqa: F811
    """A product with the identity shows the slopes.  From 104 on they are 0 and 1 (a sigmoid is below 2^-149 there, the others
    from 20 on), infinities included; before that a slope is off by 2^-20 (2 + |z|) as near 0.  A NaN stays one, and no other
    row or sum has it."""
    t = types[dt]
    z = T.tensor([s * v for v in FAR for s in (1, -1)] * copies, device=DEV).to(t)
    rows, n = z.numel(), 16
    pre, w = z[:, None].expand(rows, n).contiguous(), T.eye(n, device=DEV).to(t)
    x = T.ones(rows, 8, device=DEV).to(t)
    for grad_type in {t, T.float32}:
        one = T.ones(rows, n, device=DEV, dtype=grad_type)
        dx, _, db = M.linear_backward(w[:1].expand(rows, n).contiguous(), w, one, act=act, pre=pre, need_weight=False)
        finite = z.double().clamp(-1e30, 1e30)
        want = slope64(T, finite, act)
        far = z.abs() >= 104
        want = T.where(far, (z > 0).double(), want)
        tol = T.where(far, 0.0, 2.0 ** -20 * (2 + finite.abs()) + U[dt] * want.abs() + (2.0 ** -24 if dt == "f16" else 0))
        assert bool(((dx.double() - want[:, None]).abs() <= tol[:, None]).all()), (dt, act, (dx[:, 0].double() - want).tolist())
        assert bool(((db.double() - want.sum()).abs() <= 2.0 ** -20 * (2 + finite.abs()[~far]).sum() + rows * 2.0 ** -24 * want.abs().sum()).all())
        dw = M.linear_backward(x, w[:, :8].contiguous(), one, act=act, pre=pre, need_x=False).weight
        assert bool(dw.isfinite().all())
        torn = pre.clone()
        torn[5, 3] = math.nan
        got = M.linear_backward(x, w[:, :8].contiguous(), one, act=act, pre=torn)
        assert bool(got.x[5].isnan().all()) and bool(got.weight[3].isnan().all()) and bool(got.bias[3].isnan())
        got.x[5], got.weight[3], got.bias[3] = 0, 0, 0
        assert all(bool(v.isfinite().all()) for v in got)
