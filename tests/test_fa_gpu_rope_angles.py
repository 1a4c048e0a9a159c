"""fa_rope's sines and cosines in fp32, seen through the pair (1, 0), against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from exact_io_aware_30_gb300 import fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("direction", [1.0, -1.0])
def test_sines_and_cosines_over_the_whole_turn(layout, direction):
    """x = (1, 0) gives (cos, sin) with products that round nothing.  The angle is cut to 2^-32 turn and,
    an eighth of a turn off a quarter turn at most, rounded to fp32: 2^-27 of half a turn.  sincospi is
    off by at most a step, 2^-24 below 1 (and at 1 it is exact or a step below)."""
    from exact_io_aware_30_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    S, rot = 40000, 8
    plan = fa.rope_plan(rot, base=50.0)
    q = torch.zeros(1, 1, S, rot, device="cuda")
    q[..., :rot // 2 if layout == "half" else rot:1 if layout == "half" else 2] = 1.0
    call = fa.rope if direction > 0 else fa.rope_backward
    y = call(q, None, plan, offset=-1000, layout=layout)[0, 0].double().cpu().numpy()
    c, s = (y[:, :rot // 2], y[:, rot // 2:]) if layout == "half" else (y[:, 0::2], y[:, 1::2])
    freq = plan.freq.cpu().numpy().astype(np.uint64)
    n = (np.arange(S, dtype=np.int64) - 1000).astype(np.uint64)
    turns = (n[:, None] * freq).astype(np.int64).astype(np.float64) * 2.0 ** -64  # exact modulo a turn, then 2^-53
    theta = direction * 2 * np.pi * turns
    bound = 2.0 ** -24 + np.pi * (2.0 ** -27 + 2.0 ** -31)
    assert np.max(np.abs(c - np.cos(theta))) <= bound and np.max(np.abs(s - np.sin(theta))) <= bound
    # the quarter turns themselves
    quarter = fa.RopePlan(2, torch.tensor([1 << 62], dtype=torch.int64, device="cuda"), 1.0)
    y = call(torch.tensor([1.0, 0.0], device="cuda").expand(1, 1, 8, 2), None, quarter, offset=-4, layout=layout)[0, 0].tolist()
    up = 1.0 if direction > 0 else -1.0
    assert y == [[1.0, 0.0], [0.0, up], [-1.0, 0.0], [0.0, -up]] * 2
