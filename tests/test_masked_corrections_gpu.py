"""The corrections that masked attention's gradients carry, each held to a bound that a kernel
without it breaks (test_masked_corrections_host.py shows that): gradients from an `out` that is
far off, which the sum e has to take off again, and operands of two bf16 values (needs a B200).
"""
import ctypes

import pytest
import torch

from joint_audio_video_flash_b200 import build, ltxattn
from oracle import masked_rounding

from .masked_correction_cases import CASES, make, spoiled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    ltxattn.create()


def cuda(opts):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in opts.items()}


def partial_bytes(q, k, v, out, lse, opts):
    """Workspace of the backward call beside its statistics: partial gradients."""
    call = ltxattn._masked_call(
        torch.cuda.current_device(), q, k, v, out, lse, opts.get("scale"),
        opts.get("softcap", 0.0), opts.get("slopes"), opts.get("causal", False), None,
        opts.get("q_starts"), opts.get("kv_starts"))
    need = ctypes.c_ulonglong(0)
    assert ltxattn.load().ltxattn_masked_workspace(call, 1, need) == ltxattn.OK
    return need.value - (8 * lse.numel() + 15) // 16 * 16


@pytest.mark.parametrize("spoil", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients_are_within_the_bound(case, spoil):
    q, k, v, d_out, opts = make(case)
    dev, o = [t.cuda() for t in (q, k, v, d_out)], cuda(opts)
    out, lse = ltxattn.masked_forward(*dev[:3], **o)
    if case[-2]:
        assert partial_bytes(*dev[:3], out, lse, o) > 0
    if spoil:
        out = spoiled(out, dev[3])
    got = ltxattn.masked_backward(dev[3], *dev[:3], out, lse, **o)
    ltxattn.check()
    r = masked_rounding.gradients(q, k, v, d_out, out.cpu(), fine=case[-1], **opts)
    for name, x in zip(("dq", "dk", "dv"), got):
        bad = masked_rounding.outside(x, r, name)
        off = (x.cpu().double() - r[name + "_true"]).abs() / (r[name + "_tol"] + 1e-30)
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, {float(off[bad].max())}"
