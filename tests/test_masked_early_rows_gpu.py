"""The early rows of long causal calls, which see few keys although the call's rows see many on
average (needs a B200)."""
import pytest
import torch

from joint_audio_video_flash_b200 import build, ltxattn
from oracle import block_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    ltxattn.create()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("opts", [
    {}, dict(softcap=20.0),
    dict(softcap=20.0, slopes=torch.tensor([0.3, -0.01])),
    dict(softcap=40.0, q_starts=torch.tensor([[0, 3, 3000]], dtype=torch.int32),
         kv_starts=torch.tensor([[0, 3, 3000]], dtype=torch.int32))],
    ids=["plain", "cap", "cap-bias", "cap-documents"])
def test_early_rows(opts, dim):
    g = torch.Generator().manual_seed(dim)
    n = 5000 if "q_starts" not in opts else 3000
    q, k, v, d_out = (torch.randn(1, n, 2, dim, generator=g).bfloat16() for _ in range(4))
    opts = dict(opts, causal=True)
    dev = {a: t.cuda() if isinstance(t, torch.Tensor) else t for a, t in opts.items()}
    x = [t.cuda() for t in (q, k, v, d_out)]
    out, lse = ltxattn.masked_forward(*x[:3], **dev)
    dq, _, _ = ltxattn.masked_backward(x[3], *x[:3], out, lse, **dev)
    ltxattn.check()
    # rows 0 .. 63 need the first 64 keys only, whatever comes behind them
    cut = {a: t.clamp(max=64) if a.endswith("starts") else t for a, t in opts.items()}
    ref = block_ops.masked(*(t[:, :64] for t in (q, k, v)), d_out=d_out[:, :64], **cut)
    for name, got, want, err in (("out", out[:, :64], ref["out"], ref["out_err"]),
                                 ("lse", lse[:, :, :64], ref["lse"], ref["lse_err"]),
                                 ("dq", dq[:, :64], ref["dq"], ref["dq_err"])):
        off = (got.cpu().double() - want).abs() / (err + 1e-30)
        assert float(off.max()) <= 1, name
    # a row that sees one key: its weight and the result are rounded, 2^-8 each
    far = (out[:, 0].cpu().double() - v[:, 0].double()).abs()
    assert torch.all(far <= 2 * 2.0 ** -8 * 1.01 * v[:, 0].double().abs())
    assert not dq[:, 0].any()
