"""GPU tests of the rotary positions' cos and sin themselves, on both sides of the
borders at which they are put together.

Bound.  The angle's rest beyond the nearest quarter turn is a whole number of 2^-32
turns (the table's product rounded: 2^-33 turns, 2^-30 rad), converted to fp32 (2^-24
of itself), times a constant (2^-25) with a rounding (2^-24): at most 2.5 x 2^-24 of pi / 4,
2^-23.02 rad, which moves a cos or sin by at most 0.71 of that, 1.4 x 2^-24.  The series up to x^9
and x^8 leave off below 2^-29 and 2^-25.2; their last two sums round by 2^-25 each:
together below 1.4 + 0.9 + 1 (x 2^-24) < 2^-22.  The product with m rounds once more, and
a sum of two products twice."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def turned(step, positions, x, transpose=False, mscale=1.0):
    """Pairs x [n, 2] at `positions` of a one-pair table whose frequency is step / 2^64 turns, and their exact angles."""
    t = api().RopeTable(2, mscale=mscale)
    t.data.step[0] = step
    pos = torch.from_numpy(positions.astype(np.int32)).cuda()
    y = api().rope(x[:, None].contiguous(), pos, t, transpose=transpose)[:, 0]
    turn = np.array([(int(p) * step % (1 << 64)) / 2.0 ** 64 for p in positions])
    return y.double().cpu().numpy(), 2 * np.pi * turn


# eighths of a turn a position (each border between two quarters' halves), a little more and less, and odd ones
STEPS = [1 << 61, (1 << 61) + (1 << 33), (1 << 61) - (1 << 33), (1 << 61) + (1 << 31), (1 << 62) + 1, (1 << 64) // 3,
         11400714819323198485, 1 << 40]


@pytest.mark.parametrize("step", STEPS)
def test_cos_and_sin(step):
    pos = np.concatenate([np.arange(-600, 600), np.random.default_rng(61).integers(-2 ** 31, 2 ** 31, 4000)])
    one = torch.tensor([[1.0, 0.0]], device="cuda").expand(len(pos), 2)
    got, angle = turned(step, pos, one)
    assert np.abs(got[:, 0] - np.cos(angle)).max() <= 2.0 ** -22 and np.abs(got[:, 1] - np.sin(angle)).max() <= 2.0 ** -22
    back, _ = turned(step, pos, one, transpose=True)
    assert np.array_equal(back[:, 0], got[:, 0]) and np.array_equal(back[:, 1], -got[:, 1])
    m, _ = turned(step, pos, one, mscale=1.25)
    assert np.abs(m[:, 0] - 1.25 * np.cos(angle)).max() <= 1.25 * 2.0 ** -22 + 2.0 ** -24
    print("largest error, 2^-24:", max(np.abs(got[:, 0] - np.cos(angle)).max(), np.abs(got[:, 1] - np.sin(angle)).max()) * 2 ** 24)


def test_quarter_turns_are_exact():
    pos = np.arange(-8, 9)
    x = torch.tensor([[3.0, -5.0]], device="cuda").expand(17, 2)
    got, _ = turned(1 << 62, pos, x)
    want = np.array([[[3, -5], [5, 3], [-3, 5], [-5, -3]][p % 4] for p in pos], float)
    assert np.array_equal(got, want)
