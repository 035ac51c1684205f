"""The rotary table against frequencies in 60 digits.  No GPU."""
from decimal import Decimal, getcontext

import math
import pytest

from sparse_attention_lightning_score_b200 import api

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def _turns(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """2^64 f_i / (2 pi) by the definition; the ends of YaRN's ramp are whole pairs."""
    getcontext().prec = 60
    if scaling == "yarn":
        pair = [rot * math.log(original_len / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (beta_fast, beta_slow)]
        lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
    out = []
    for i in range(rot // 2):
        f = (-Decimal(2 * i) / rot * Decimal(base).ln()).exp()
        if scaling == "linear":
            f /= Decimal(factor)
        if scaling == "yarn":
            ramp = min(max(Decimal(i - lo) / (hi - lo), Decimal(0)), Decimal(1))
            f = f / Decimal(factor) * ramp + f * (1 - ramp)
        out.append(f / (2 * PI) * 2 ** 64)
    return out


@pytest.mark.parametrize("rot,kw", [
    (64, {}), (128, {}), (1024, {}), (2, dict(base=500000.0)), (36, dict(base=1.0625)), (64, dict(base=1e29)),
    (128, dict(scaling="linear", factor=8.0)), (96, dict(scaling="linear", factor=3.7)),
    (64, dict(scaling="yarn", factor=40.0, original_len=4096)), (128, dict(scaling="yarn", factor=1.9, original_len=32768)),
    (32, dict(scaling="yarn", factor=2.0, original_len=77, beta_fast=8.0, beta_slow=0.5))])
def test_table_is_within_two_units_of_the_fixed_point(rot, kw):
    """Half a unit of 2^-64 turns from the last rounding.  Before it a value below 2^61.4 units in 64 significant bits:
    power (2^-63 of it), its exponent (ln(base) e 2^-64, times base^-e at most 0.06 units), division, 2 pi and YaRN's four
    steps (2^-64 each): below 2^61.4 (2^-63 + 6 * 2^-64) + 0.06 + 0.5 = 1.9 units."""
    got = api.li_rope_table(rot, device="cpu", **kw).tolist()
    for g, w in zip(got, _turns(rot, **kw)):
        assert abs(Decimal(g % 2 ** 64) - w) <= 2
