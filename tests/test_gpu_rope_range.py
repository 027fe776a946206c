"""Rotations by angles of any size: exact to 2^-53 of the angle, and a rotation beyond that too."""
import numpy as np
import pytest

from oracle import serve as ref
from test_gpu_rope import _f64, check

pytestmark = pytest.mark.gpu


def _heads():
    import torch
    return torch.from_numpy(np.random.default_rng(9).standard_normal((6, 3, 16))).cuda().float()


PLACES = np.array([2 ** 31 - 1, 1, 12345, 2 ** 20 + 1, 3, 0], np.int32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_large_angles(layout):
    """Frequencies beyond those of positions, angles of up to 2^50: beside the bound of other rotations,
    2^-52 of the angle (2^-53 from the reduction, as much for the oracle's product)."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    x = _heads()
    f = np.array([1.0, -3.7, 1e2, 12345.678, 2.0 ** 18 + 0.1, 1e-3, 0.0, 77.7])
    y, _ = ops.rope(x, None, torch.from_numpy(PLACES).cuda(), torch.from_numpy(f).cuda(), layout=layout)
    want, size = ref.rope(_f64(x), PLACES, f, layout, 1.0)
    angle = np.abs(PLACES.astype(np.float64)[:, None] * f[None]) * 2.0 ** -52
    angle = np.concatenate([angle, angle], 1) if layout == "half" else np.repeat(angle, 2, 1)
    err = np.abs(_f64(y) - want)
    tol = 2.0 ** -21 * size + angle[:, None] * size + 2.0 ** -24 * np.abs(want)
    print(f"err / bound {float((err / tol).max()):.3f}")
    assert (err <= tol).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("exponent", [22, 26, 35, 60, 200, 950])
def test_angles_beyond_all_places_still_turn(layout, exponent):
    """Angles so large that nothing of them is known modulo a turn: pairs keep their length (2^-10 of it is
    allowed: the series are not cut for angles beyond pi / 4)."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    x = _heads()
    f = torch.from_numpy(2.0 ** exponent * np.array([1.0, -1.7, 1.1, 1.9, 0.3, 1.33, 0.77, 1.21])).cuda()
    y, _ = ops.rope(x, None, torch.from_numpy(PLACES).cuda(), f, layout=layout)
    pair = (lambda t: t.unflatten(-1, (2, 8))) if layout == "half" else (lambda t: t.unflatten(-1, (8, 2)).transpose(-1, -2))
    before, after = pair(x.double()).square().sum(-2).sqrt(), pair(y.double()).square().sum(-2).sqrt()
    assert float(((after - before).abs() / before).max()) <= 2.0 ** -10
    assert torch.equal(y[5], x[5])                  # place 0


def test_frequencies_that_are_not_finite():
    """Their pairs are no numbers, the others are turned."""
    import torch
    from gated_deltanet_prefill_chunkwise_amd import ops
    x, f = _heads(), np.array([1.0, np.inf, 0.1, np.nan, 0.01, 0.3, 0.2, 1e-4])
    y, _ = ops.rope(x, None, torch.from_numpy(PLACES).cuda(), torch.from_numpy(f).cuda())
    bad = torch.tensor([1, 3, 9, 11])
    rest = torch.tensor([i for i in range(16) if i not in (1, 3, 9, 11)])
    assert torch.isnan(y[..., bad]).all()
    want, size = ref.rope(_f64(x), PLACES, np.where(np.isfinite(f), f, 0.0), "half", 1.0)
    check(y[..., rest].contiguous(), want[..., rest], size[..., rest], "f32", False)
