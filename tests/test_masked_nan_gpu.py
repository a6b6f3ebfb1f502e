"""Attention with masked scores: what is not finite in a visible row shows in every result that
reads it, however the keys were split (needs a B200)."""
import ctypes
import math

import pytest
import torch

from joint_audio_video_flash_b200 import build, ltxattn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    ltxattn.create()


def make(batch, q_len, kv_len, heads, kv_heads, dim):
    g = torch.Generator().manual_seed(q_len + kv_len)
    return [torch.randn(batch, n, h, dim, generator=g).bfloat16().cuda()
            for n, h in ((q_len, heads), (kv_len, kv_heads), (kv_len, kv_heads), (q_len, heads))]


def in_parts(q, k, v, **opts):
    """Whether the forward call splits the keys (it needs a workspace then)."""
    lse = torch.empty(q.shape[0], q.shape[2], q.shape[1], device="cuda")
    call = ltxattn._masked_call(torch.cuda.current_device(), q, k, v, torch.empty_like(q), lse,
                                None, opts.get("softcap", 0.0), None, opts.get("causal", False),
                                None, None, None)
    need = ctypes.c_ulonglong(0)
    assert ltxattn.load().ltxattn_masked_workspace(call, 0, need) == ltxattn.OK
    return need.value > 0


CASES = [
    # batch, q_len, kv_len, heads, kv_heads, dim, options, key parts
    (2, 1, 9000, 8, 2, 128, {}, True),
    (1, 3, 5000, 4, 4, 64, dict(causal=True), True),
    (2, 1, 9000, 4, 4, 64, dict(softcap=10.0), True),   # capped, without a running maximum
    (1, 100, 2000, 2, 2, 64, dict(softcap=10.0), True),
    (2, 1, 100, 4, 4, 64, {}, False),
    (1, 300, 300, 4, 2, 128, dict(causal=True), False),
    (1, 200, 200, 2, 2, 64, dict(softcap=10.0), False),
]


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_a_query_that_is_not_finite(case, bad):
    batch, q_len, kv_len, heads, kv_heads, dim, opts, parts = case
    q, k, v, d_out = make(*case[:6])
    assert in_parts(q, k, v, **opts) == parts
    want, want_lse = ltxattn.masked_forward(q, k, v, **opts)
    q[0, q_len - 1, 1, 5] = bad
    out, lse = ltxattn.masked_forward(q, k, v, **opts)
    ltxattn.check()
    if bad == math.inf and opts.get("softcap"):  # a cap makes scores of infinities finite
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        return
    assert torch.isnan(out[0, q_len - 1, 1]).all() and torch.isnan(lse[0, 1, q_len - 1])
    want[0, q_len - 1, 1], out[0, q_len - 1, 1] = 0, 0
    want_lse[0, 1, q_len - 1], lse[0, 1, q_len - 1] = 0, 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse = ltxattn.masked_forward(q, k, v, **opts)
    dq, _, _ = ltxattn.masked_backward(d_out, q, k, v, out, lse, **opts)
    ltxattn.check()
    assert torch.isnan(dq[0, q_len - 1, 1]).all()


@pytest.mark.parametrize("at", [0, 70])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_a_key_that_is_not_finite(case, at):
    batch, q_len, kv_len, heads, kv_heads, dim, opts, parts = case
    q, k, v, _ = make(*case[:6])
    assert in_parts(q, k, v, **opts) == parts
    k[0, at, 1, 3] = math.nan
    out, lse = ltxattn.masked_forward(q, k, v, **opts)
    ltxattn.check()
    group = heads // kv_heads
    place = torch.arange(q_len) + kv_len - q_len
    sees = place >= at if opts.get("causal") else torch.ones(q_len, dtype=torch.bool)
    for b in range(batch):
        for h in range(heads):
            hit = sees if b == 0 and h // group == 1 else torch.zeros(q_len, dtype=torch.bool)
            assert torch.equal(torch.isnan(lse[b, h].cpu()), hit)
            assert torch.equal(torch.isnan(out[b, :, h].cpu()).all(-1), hit)
            assert torch.equal(torch.isnan(out[b, :, h].cpu()).any(-1), hit)


def test_the_only_part_that_sees_keys_is_not_finite():
    # documents of one key part's worth of keys among longer ones: the other parts see none
    q, k, v, _ = make(1, 4, 6000, 2, 2, 64)
    q_starts = torch.tensor([[0, 2, 4]], dtype=torch.int32, device="cuda")
    kv_starts = torch.tensor([[0, 40, 6000]], dtype=torch.int32, device="cuda")
    k[0, 7, 0, 0] = math.nan
    out, lse = ltxattn.masked_forward(q, k, v, q_starts=q_starts, kv_starts=kv_starts)
    ltxattn.check()
    assert torch.isnan(out[0, :2, 0]).all() and torch.isnan(lse[0, 0, :2]).all()
    assert torch.isfinite(out[0, 2:]).all() and torch.isfinite(out[0, :, 1]).all()
    assert torch.isfinite(lse[0, 0, 2:]).all() and torch.isfinite(lse[0, 1]).all()
