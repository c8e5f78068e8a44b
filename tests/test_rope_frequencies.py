"""Frequencies of the scaled rotary positions against their definitions, every pair, at the defaults (CPU only)."""
import math

import pytest

from sparse_kv_cache_landmark_gb300 import kvo


def turns(t):
    return [(x % 2 ** 64) / 2.0 ** 64 for x in t.tolist()]


def wavelength(i, rot, base):
    return 2 * math.pi * base ** (2.0 * i / rot)


def banded(rot, base, factor, length, low=1.0, high=4.0):
    """By wavelengths: those shorter than length / high stay, those longer than length / low grow by the factor, and between
    the two the frequencies blend linearly in the number of turns within the length."""
    out = []
    for i in range(rot // 2):
        w = wavelength(i, rot, base)
        if w < length / high:
            out.append(1 / w)
        elif w > length / low:
            out.append(1 / (factor * w))
        else:
            s = (length / w - low) / (high - low)
            out.append((1 - s) / (factor * w) + s / w)
    return out


def ramp(rot, base, factor, length, low=1.0, high=32.0):
    """By pairs: up to the pair (rounded down) that turns `high` times within the length they stay, from the one (rounded
    up) that turns `low` times they are divided, and between the two they blend linearly in the pair's number."""
    pair = lambda n: (rot / 2) * math.log(length / (2 * math.pi * n), base)
    a, b = max(0, math.floor(pair(high))), min(rot - 1, math.ceil(pair(low)))
    out = []
    for i in range(rot // 2):
        divided = min(1.0, max(0.0, (i - a) / (b - a)))
        f = 1 / wavelength(i, rot, base)
        out.append(f * (1 - divided) + f / factor * divided)
    return out


@pytest.mark.parametrize("rot,base,factor,length", [(64, 10000.0, 8.0, 8192), (128, 500000.0, 8.0, 8192), (128, 10000.0, 4.0, 4096),
                                                    (64, 1000000.0, 40.0, 32768), (32, 10000.0, 2.0, 2048)])
def test_scaled_frequencies_at_the_defaults(rot, base, factor, length):
    for kind, want in (("banded", banded(rot, base, factor, length)), ("ramp", ramp(rot, base, factor, length))):
        f, amp = kvo.rope_frequencies(rot, base, kind, factor, original_len=length, device="cpu")
        got = turns(f)
        blended = [i for i, w in enumerate(want) if 1.001 * w < 1 / wavelength(i, rot, base) < 0.999 * factor * w]
        assert blended
        for i, (x, y) in enumerate(zip(got, want)):
            assert math.isclose(x, y, rel_tol=1e-10), (kind, i, x, y)
        assert math.isclose(amp, 0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0)


def test_bounds_given_are_taken():
    for kind, form in (("banded", banded), ("ramp", ramp)):
        f, _ = kvo.rope_frequencies(128, 10000.0, kind, 4.0, original_len=4096, low=2.0, high=16.0, device="cpu")
        for x, y in zip(turns(f), form(128, 10000.0, 4.0, 4096, 2.0, 16.0)):
            assert math.isclose(x, y, rel_tol=1e-10)
    with pytest.raises(kvo.KvoError, match="high > low"):
        kvo.rope_frequencies(128, 10000.0, "ramp", 4.0, low=40.0, device="cpu")
    with pytest.raises(kvo.KvoError, match="high > low"):
        kvo.rope_frequencies(128, 10000.0, "banded", 4.0, low=5.0, device="cpu")
