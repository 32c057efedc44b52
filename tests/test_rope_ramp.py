"""The ramp of rotary frequencies by index, pinned against the published
method (YaRN: Peng et al., 2023) written out here: index i(r) = rot ln(len /
(2 pi r)) / (2 ln base) makes r turns over len positions; the part that stays
falls from 1 at max(floor(i(high)), 0) to 0 at min(ceil(i(low)), rot - 1), an
end that may lie beyond the table's rot/2 pairs (CPU only)."""
import math

import numpy as np
import pytest

from verify_matvec_gb300 import build, cbq


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def _method(rot, base, factor, length, low, high):
    at = lambda r: rot * math.log(length / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
    table = []
    for i in range(rot // 2):
        whole = base ** (-2 * i / rot) / (2 * math.pi)
        ramp = min(max((i - first) / (last - first), 0.0), 1.0)
        table.append(whole / factor * ramp + whole * (1 - ramp))
    return np.array(table)


@pytest.mark.parametrize("rot,base,factor,length,low,high", [
    (64, 1e4, 16.0, 65536.0, 1.0, 32.0),    # ends at 33 of 32 pairs
    (64, 1e4, 40.0, 4096.0, 1.0, 32.0),     # ends inside the table
    (128, 1e4, 4.0, 131072.0, 1.0, 32.0),   # ends far beyond it
    (128, 1e6, 4.0, 32768.0, 1.0, 32.0),
    (32, 1e4, 8.0, 262144.0, 2.0, 64.0),
    (64, 1e4, 16.0, 1e8, 1.0, 32.0),        # its start lies beyond the pairs, too: all of them stay
])
def test_ramp(rot, base, factor, length, low, high):
    got = cbq.cbq_rope_turns(rot, base=base, scaling="index", factor=factor, orig_len=length, low=low, high=high, device="cpu")
    np.testing.assert_allclose(got.numpy(), _method(rot, base, factor, length, low, high), rtol=1e-13)


def test_ramp_past_the_table():
    """Worked out by hand: over 65,536 positions the slowest of 32 pairs still makes 1.4 turns and keeps a part of its
    rate.  i(32) = 20.1 and i(1) = 32.1, so the ramp falls from pair 20 to 33: pair 31 keeps 2/13, pair 24 9/13."""
    got = cbq.cbq_rope_turns(64, scaling="index", factor=16.0, orig_len=65536.0, low=1.0, high=32.0, device="cpu").numpy()
    rate = got * (2 * math.pi) / 1e4 ** (-np.arange(32) / 32)
    np.testing.assert_allclose(rate[:21], 1.0, rtol=1e-13)
    np.testing.assert_allclose(rate[[24, 31]], [9 / 13 + 4 / 13 / 16, 2 / 13 + 11 / 13 / 16], rtol=1e-12)
