"""Which of the two ramps in use rotary_freqs' "yarn" is: linear in a pair's turns, not in its index."""
import math

import torch

from delta_rule_linear_gated_amd import binding as B


def test_the_ramp_is_linear_in_the_turns():
    rot, factor, trained = 128, 8.0, 4096
    plain, f = B.rotary_freqs(rot)[0], B.rotary_freqs(rot, scaling="yarn", factor=factor, trained=trained)[0]
    turns = trained * plain / (2 * math.pi)
    kept = (f - plain / factor) / (plain - plain / factor)   # 1: as trained, 0: divided by the factor
    between = (turns > 1) & (turns < 32)
    assert torch.allclose(kept[between], (turns[between] - 1) / 31, rtol=0, atol=1e-12)
    assert torch.allclose(kept[turns >= 32], torch.ones(()).double()) and float(kept[turns <= 1].abs().max()) < 1e-12

    def pair(n):   # the index of a pair that turns n times, as a real number
        return rot * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(10000.0))

    low, high = math.floor(pair(32)), math.ceil(pair(1))
    ramp = 1 - ((torch.arange(rot // 2).double() - low) / (high - low)).clamp(0, 1)
    other = plain * ramp + plain / factor * (1 - ramp)
    off = (f / other - 1).abs()
    assert int((off > 1e-9).sum()) == 25 and 0.56 < float(off.max()) < 0.57   # what the docstring says of it
