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


def test_yarn_needs_a_pair_that_makes_beta_slow_turns():
    """Over fewer than 2 pi beta_slow positions every pair makes fewer than beta_slow turns and would be divided by the
    factor, but the ramp, which starts at pair 0, would leave that one as it is: refused."""
    kw = dict(scaling="yarn", factor=40.0, device="cpu")
    for short, enough, slow in [(1, 7, 1.0), (6, 7, 1.0), (12, 13, 2.0), (3, 4, 0.5)]:
        with pytest.raises(api.LiError):
            api.li_rope_table(64, original_len=short, beta_slow=slow, **kw)
        got = api.li_rope_table(64, original_len=enough, beta_slow=slow, **kw).tolist()
        plain = api.li_rope_table(64, device="cpu").tolist()
        assert got[0] == plain[0] and abs(got[31] - plain[31] / 40) <= 1 + plain[31] * 2.0 ** -52
