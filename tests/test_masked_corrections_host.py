"""The bounds that the gradients' corrections are tested with: the arithmetic with its roundings
stays inside them, and each mistake that a kernel could make there leaves them (no GPU)."""
import pytest
import torch

from oracle import block_ops, masked_rounding

from .masked_correction_cases import CASES, make, spoiled

FULL = ("no correction", "wrong sign", "half of e", "first half of e")


def arithmetic(case, spoil, mistake=None):
    q, k, v, d_out, opts = make(case)
    fwd = {n: opts[n] for n in opts}
    out = block_ops.masked(q, k, v, **fwd)["out"].float().bfloat16()
    if spoil:
        out = spoiled(out, d_out)
    return masked_rounding.gradients(q, k, v, d_out, out, fine=case[-1], mistake=mistake, **opts)


def share(r, name):
    return float(masked_rounding.outside(r[name].float().bfloat16(), r, name).double().mean())


SMALL = [c for c in CASES if c[1] * c[2] * c[3] <= 2_000_000]


@pytest.mark.parametrize("spoil", [False, True])
@pytest.mark.parametrize("case", SMALL, ids=str)
def test_the_arithmetic_is_within_its_bound(case, spoil):
    r = arithmetic(case, spoil)
    assert all(share(r, n) == 0 for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("mistake", FULL + ("a tile of the sum", "half of the sum"))
@pytest.mark.parametrize("case", SMALL, ids=str)
def test_a_mistake_in_the_correction_shows(case, mistake):
    r = arithmetic(case, True, mistake)
    if mistake == "half of e" and case[2] // case[6].get("docs", 1) <= 64:
        assert share(r, "dq") == 0  # no columns behind the first 64
        return
    assert share(r, "dq") > 0.1
    if mistake in FULL:
        assert share(r, "dk") > 0.1


@pytest.mark.parametrize("case", [c for c in SMALL if c[-1]], ids=str)
def test_lost_low_halves_show(case):
    r = arithmetic(case, False, "low halves")
    assert all(share(r, n) > 0.01 for n in ("dq", "dk", "dv"))
