"""The frequencies of YaRN over its whole range of arguments (host only): the
ramp's ends lie where the pairs' numbers of turns say, also past the last pair
and before the first."""
import math

import pytest

import adaptive_vector_quantized_b200 as avq


def ramp_of(rot, base, factor, trained, turns_low, turns_high, axes=1):
    """How far each pair is from kept (0) to divided by the factor (1), and its turns over the trained range."""
    f, _ = avq.avq_rotary_freqs(rot, base=base, axes=axes, scaling="yarn", factor=factor, trained=trained,
                                turns_low=turns_low, turns_high=turns_high)
    f = f.tolist()
    pairs = rot // 2 // axes
    assert f[:pairs] * axes == f
    plain = [base ** (-i / pairs) for i in range(pairs)]
    return ([(1 - y / x) / (1 - 1 / factor) for x, y in zip(plain, f)], [trained * x / (2 * math.pi) for x in plain])


# rot, base, factor, trained, turns_low, turns_high
ARGS = [(64, 10000.0, 8.0, 4096, 1.0, 32.0), (64, 10000.0, 8.0, 65536, 1.0, 32.0), (64, 10000.0, 8.0, 131072, 1.0, 32.0),
        (64, 500.0, 8.0, 4096, 1.0, 32.0), (128, 10000.0, 4.0, 200000, 0.5, 40.0), (16, 100.0, 2.0, 100000, 1.0, 32.0),
        (64, 10000.0, 8.0, 1, 1.0, 32.0), (64, 10000.0, 8.0, 4096, 1000.0, 2000.0), (8, 1.5, 3.0, 1 << 30, 1.0, 2.0),
        (32, 10000.0, 8.0, 40, 1.0, 32.0)]


@pytest.mark.parametrize("axes", [1, 2])
@pytest.mark.parametrize("args", ARGS)
def test_pairs_are_kept_or_divided_by_their_turns(args, axes):
    rot, base, factor, trained, low, high = args
    ramp, turns = ramp_of(rot * axes, base, factor, trained, low, high, axes)
    for i, (r, t) in enumerate(zip(ramp, turns)):
        if t < low * (1 - 1e-12):
            assert abs(r - 1) < 1e-12, (i, t, r)
        elif t > high * (1 + 1e-12):
            assert abs(r) < 1e-12, (i, t, r)
        elif t > low * (1 + 1e-12):
            assert r < 1 - 1e-9, (i, t, r)
    assert all(b >= a - 1e-12 for a, b in zip(ramp, ramp[1:]))


@pytest.mark.parametrize("args", [a for a in ARGS if a[3] >= 4096 and a[4] < 100])
def test_ramp_ends_at_the_rotated_size(args):
    """Linear in the pair index from max(floor(i(high)), 0) to min(ceil(i(low)), rot - 1), with i(r) the
    index of the pair that would make r turns."""
    rot, base, factor, trained, low, high = args
    ramp, _ = ramp_of(*args)

    def index(r):
        return rot * math.log(trained / (2 * math.pi * r)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
    for i, r in enumerate(ramp):
        want = 0.0 if i <= lo else 1.0 if i >= hi else (i - lo) / (hi - lo)
        assert abs(r - want) < 1e-12, (i, r, want)


def test_slowest_pair_that_turns_more_than_once_is_not_divided_in_full():
    f, _ = avq.avq_rotary_freqs(64)
    y, _ = avq.avq_rotary_freqs(64, scaling="yarn", factor=8.0, trained=65536)
    assert 1.3 < 65536 * f[-1] / (2 * math.pi) < 1.4
    assert abs(f[-1] / y[-1] - 3.85) < 0.01
