"""The angles of rotary positions on the GPU: within 2^-34 of a turn at every 32-bit position, seen where a sine or cosine is nearly
zero and fp32 shows the angle's last bits."""
from fractions import Fraction

import numpy as np
import pytest

from tests.harness import torch_mod
from tests.test_rope_turns import turns_of

pytestmark = pytest.mark.gpu

torch = None


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = torch_mod()
    assert torch.cuda.is_available()


def sine_of_turns(a):
    """sin(2 pi a) of a small fraction a (|a| < 2^-9), to fp64: two terms of the series."""
    x = float(a) * 2 * np.pi
    return x - x ** 3 / 6


@pytest.mark.parametrize("rot,layout", [(32, "half"), (32, "interleaved"), (26, "half")])
def test_angles_within_a_34th_power_of_a_turn(rot, layout):
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(rot)
    pairs = rot // 2
    first = np.arange(pairs) if layout == "half" else 2 * np.arange(pairs)
    second = first + (pairs if layout == "half" else 1)
    worst, seen = 0.0, 0
    for p in [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -1999999973, 1 << 24, 77777, 1]:
        # Frequencies that turn by a few quarters and a little at this position (whole turns a position beside them: f may be large).
        quarters = rng.integers(1, 4000, pairs)
        little = np.exp2(rng.uniform(-33, -10, pairs)) * rng.choice([-1, 1], pairs)
        f = (quarters / 4 + little) / p * 2 * np.pi
        f[: pairs // 4] += 2 * np.pi * rng.integers(-1000, 1000, pairs // 4)
        rope = Rope(head_dim=32, rot_dim=rot, layout=layout, freqs=f)
        x = np.zeros((1, 1, 32), np.float32)
        x[..., first] = 1.0
        dx, out = torch.from_numpy(x).cuda(), torch.empty((1, 1, 32), device="cuda")
        pos = torch.tensor([p], dtype=torch.int32, device="cuda")
        rope.apply(1, dx.data_ptr(), out.data_ptr(), 1, "f32", positions_ptr=pos.data_ptr(), stream=torch.cuda.current_stream().cuda_stream)
        y = out.double().cpu().numpy()[0, 0]
        for i in range(pairs):
            turns = turns_of(float(f[i])) * p
            q = round(turns * 4)                      # quarters, and the small rest a
            a = turns - Fraction(q, 4)
            if abs(a) > Fraction(1, 1 << 9):          # far positions times the rounding of a large f: no small rest
                continue
            # (cos, sin) of q quarters + a: the one of them that is nearly zero is +- sin(2 pi a)
            small = {0: y[second[i]], 1: -y[first[i]], 2: -y[second[i]], 3: y[first[i]]}[q % 4]
            want = sine_of_turns(a)
            # what the series' arguments, the sum x + e, the product and the amplitude round: 4 steps of 2^-24 of it
            tol = 2 * np.pi * 2.0 ** -34 + 4 * 2.0 ** -24 * abs(want)
            worst, seen = max(worst, abs(small - want) / tol), seen + 1
            assert abs(small - want) <= tol, (p, i, q % 4, (small - want) / (2 * np.pi) * 2.0 ** 34)
    assert seen > 4 * pairs and worst > 0
