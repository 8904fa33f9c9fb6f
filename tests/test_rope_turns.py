"""The rotation's table against arithmetic of 60 digits: entries are whole units of
2^-64 turns, so that a product with a position of 32 bits is within 2^-33 turns."""
from decimal import Decimal, localcontext

import pytest

from speculative_decoding_tree_best_gb300 import binding
from tests.test_chain_args import lib  # noqa: F401

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def exact(rot, base, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    n, y = rot // 2, []
    base, factor = Decimal(base), Decimal(factor)
    slow, fast = Decimal(beta_slow), Decimal(beta_fast)
    if scaling == "ntk":
        base *= (factor.ln() * rot / (rot - 2)).exp()
    for j in range(n):
        f = (-base.ln() * j / n).exp()
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            g = min(Decimal(1), max(Decimal(0), (orig_len * f / TWO_PI - slow) / (fast - slow)))
            f = (1 - g) * f / factor + g * f
        y.append(f / TWO_PI * 2 ** 64)
    return y


@pytest.mark.parametrize("rot", [16, 64, 112, 128])
@pytest.mark.parametrize("base", [1.0, 1.5, 1e4, 1e6, 5e6, 1e300])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.7),
                                dict(scaling="ntk", factor=7.3),
                                dict(scaling="yarn", factor=4.0, orig_len=32768),
                                dict(scaling="yarn", factor=32.1, orig_len=8191, beta_fast=31.7,
                                     beta_slow=0.3)])
def test_entries_are_whole_units(lib, rot, base, kw):  # noqa: F811
    turns, _ = binding.spec_rope_turns(rot, base, **kw)
    with localcontext() as ctx:
        ctx.prec = 60
        for got, want in zip(turns, exact(rot, base, **kw)):
            assert abs(got - want) <= Decimal("0.50001")


def test_the_farthest_position(lib):  # noqa: F811
    """What the kernel makes of an entry: the upper 32 bits of position times entry,
    modulo a turn.  Half a unit of the entry at 2^31 - 1 is 2^-34 turns, and the bits
    that are left out less than 2^-32."""
    turns, _ = binding.spec_rope_turns(128, 1e6)
    p = 2 ** 31 - 1
    with localcontext() as ctx:
        ctx.prec = 60
        for got, want in zip(turns, exact(128, 1e6)):
            angle = Decimal(((p * got) % 2 ** 64) >> 32) / 2 ** 32
            off = (angle - (p * want / 2 ** 64) % 1 + Decimal("0.5")) % 1 - Decimal("0.5")
            assert -(Decimal(2) ** -32 + Decimal(2) ** -34) <= off <= Decimal(2) ** -34


def test_entries_of_given_frequencies(lib):  # noqa: F811
    """A caller's own frequencies: to the nearest unit, modulo a turn."""
    f = [1.0, 0.1, 1e4 ** (-31 / 32), -0.1, 0.1 + 40.0, 0.0, 5e-20]
    with localcontext() as ctx:
        ctx.prec = 60
        for got, x in zip(binding.rope_turns_of(f), f):
            off = (got - Decimal(x) / TWO_PI * 2 ** 64) % 2 ** 64
            assert min(off, 2 ** 64 - off) <= Decimal("0.50001") and 0 <= got < 2 ** 64
    # those of a scaling that the library has, up to the rounding of their doubles
    mine, _ = binding.spec_rope_turns(64, 1e4)
    for a, b in zip(binding.rope_turns_of([1e4 ** (-j / 32) for j in range(32)]), mine):
        assert abs(a - b) <= 2 ** 10
