"""The workspace of layer norm's gradients, and the wide rows that need most of it (needs a
B200)."""
import ctypes

import pytest
import torch

from joint_audio_video_flash_b200 import build, ltxattn
from oracle import block_ops

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    ltxattn.load()


def workspace(rows, cols, groups, code):
    need = ctypes.c_ulonglong(0)
    assert ltxattn.load().ltxattn_layer_norm_workspace(rows, cols, groups, code, need) == \
        ltxattn.OK
    return need.value


@pytest.mark.parametrize("code", [ltxattn.BF16, ltxattn.FP32])
@pytest.mark.parametrize("rows,cols,groups", [
    (30720, 4096, 1), (30720, 4096, 2), (1 << 20, 100, 1), (2000, 16384, 1), (100000, 16384, 1),
    (5000, 1 << 20, 1), (1 << 30, 1 << 20, 1), (6000, 1 << 20, 3000), (3 << 20, 8192, 1 << 20),
    (1 << 30, 1, 1)])
def test_partials_are_a_few_megabytes(rows, cols, groups, code):
    # a CTA of the row kernels holds 2 * cols floats of them: 8192 columns at most on one CTA per
    # SM, 10 MB; the column kernel's are less
    assert workspace(rows, cols, groups, code) <= 16 << 20


@pytest.mark.parametrize("case", [(700, 9000, 1, BF), (301, 16384, 1, BF), (300, 8200, 3, FP),
                                  (3000, 4097, 2, FP), (40, 100000, 2, BF), (5, 1 << 20, 1, HF)],
                         ids=str)
@pytest.mark.parametrize("apart", [False, True])
def test_wide_rows(case, apart):
    """apart: x and dy lie differently on 16-byte boundaries, which the column kernel takes."""
    rows, cols, groups, dtype = case
    g = torch.Generator().manual_seed(rows + cols)
    x, dy = ((torch.randn(rows, cols, generator=g) + m).to(dtype) for m in (0.5, 0.0))
    w = (1 + 0.2 * torch.randn((cols,) if groups == 1 else (groups, cols), generator=g)).to(dtype)
    wide = torch.zeros(rows, cols + 24, dtype=dtype, device="cuda")
    xd = wide[:, 3:3 + cols] if apart else wide[:, :cols]
    xd.copy_(x)
    _, mean, rstd = ltxattn.layer_norm(xd, w.cuda(), return_stats=True)
    got = ltxattn.layer_norm_backward(dy.cuda(), xd, mean, rstd, w.cuda())
    ref = block_ops.layer_norm_backward(dy, x, mean.cpu(), rstd.cpu(), w)
    for n, (want, bound) in enumerate(ref):
        bound = block_ops.rounded(want, bound, dtype) if n == 0 else bound
        err = (got[n].cpu().double().reshape(want.shape) - want).abs()
        assert torch.all(err <= bound), float((err / bound).max())
    again = ltxattn.layer_norm_backward(dy.cuda(), xd, mean, rstd, w.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, again))
