"""Masked attention's gradients where a query sees one key: its weight is 1 whatever the score
is, so the score has no gradient at all, and dq (and dk, where that key is a document's only
one) is 0, not the rounding of two sums that cancel (needs a B200)."""
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


def gradients(batch, q_len, kv_len, heads, kv_heads, dim, bias=False, seed=0, **opts):
    g = torch.Generator().manual_seed(seed + q_len + kv_len)
    q, k, v, d_out = (torch.randn(batch, n, h, dim, generator=g).bfloat16().cuda()
                      for n, h in ((q_len, heads), (kv_len, kv_heads), (kv_len, kv_heads),
                                   (q_len, heads)))
    if bias:
        opts["slopes"] = torch.linspace(-0.4, 0.5, heads).cuda()
    opts = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in opts.items()}
    out, lse = ltxattn.masked_forward(q, k, v, **opts)
    grads = ltxattn.masked_backward(d_out, q, k, v, out, lse, **opts)
    ltxattn.check()
    return grads


@pytest.mark.parametrize("cap", [0.0, 10.0, 50.0, 500.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1, 64), (2, 1, 1, 8, 8, 128), (2, 16, 1, 5, 1, 128),
                                  (1, 24, 1, 16, 4, 64), (2, 300, 1, 32, 8, 128),
                                  (1, 5000, 1, 8, 8, 64)], ids=str)
def test_one_key(case, bias, cap):
    dq, dk, dv = gradients(*case, bias=bias, softcap=cap, scale=4 * case[-1] ** -0.5)
    assert not dq.any() and not dk.any()
    assert torch.isfinite(dv).all() and dv.any()


@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_documents_of_one_key(cap):
    # documents of 1, 0, 1, 200 and 1 keys
    ks = torch.tensor([[0, 1, 1, 2, 202, 203]], dtype=torch.int32)
    qs = torch.tensor([[0, 9, 9, 150, 300, 301]], dtype=torch.int32)
    dq, dk, dv = gradients(1, 301, 203, 4, 2, 64, softcap=cap, q_starts=qs, kv_starts=ks)
    rows, keys = torch.zeros(301, dtype=torch.bool), torch.zeros(203, dtype=torch.bool)
    rows[150:300] = True
    keys[2:202] = True
    assert not dq[:, ~rows].any() and not dk[:, ~keys].any()
    assert dq[:, rows].any(-1).all() and dk[:, keys].any(-1).all()


@pytest.mark.parametrize("kv_len", [300, 5000])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_the_first_row_of_a_causal_call(cap, kv_len):
    # with key parts (few rows), without, and with a prefix of one key that the early rows share
    for q_len, prefix in ((kv_len, None), (kv_len + 70, 1)):
        opts = {} if prefix is None else dict(prefix=torch.tensor([[prefix]], dtype=torch.int32))
        dq, _, _ = gradients(1, q_len, kv_len, 2, 1, 128, softcap=cap, causal=True, **opts)
        one = 1 if prefix is None else 71
        assert not dq[:, :one].any()
        assert dq[:, one:].any(-1).all()
