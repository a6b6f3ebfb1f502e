"""Rotary axes: the channels behind the last axis keep their bits (needs a B200)."""
import math

import pytest
import torch

from joint_audio_video_flash_b200 import build, ltxattn

pytestmark = pytest.mark.gpu

BITS = {torch.bfloat16: torch.int16, torch.float16: torch.int16, torch.float32: torch.int32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    ltxattn.load()


def unrotated(dim, dims, layout):
    """Channels of a head that no axis has."""
    pairs = sum(dims) // 2
    left = torch.ones(dim, dtype=torch.bool)
    if layout == "pairs":
        left[:2 * pairs] = False
    else:
        left[:pairs] = False
        left[dim // 2:dim // 2 + pairs] = False
    return left


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("dim,dims", [(64, (2,)), (64, (24, 16, 16)), (128, (44, 42)), (80, (10, 16)),
                                      (128, (126,)), (16, (14,)), (512, (100, 6))])
@pytest.mark.parametrize("inverse", [False, True])
def test_channels_of_no_axis_keep_their_bits(dtype, layout, dim, dims, inverse):
    g = torch.Generator().manual_seed(dim + sum(dims))
    q, k = (torch.randn(2, 9, h, dim, generator=g).to(dtype).cuda() for h in (3, 1))
    pos = (torch.rand(2, 9, len(dims), generator=g) * 100).cuda()
    freq = ltxattn.rope_frequencies(dims)
    opts = dict(layout=layout, inverse=inverse)
    left = unrotated(dim, dims, layout).cuda()
    want_q, want_k = ltxattn.rope_axes(q, k, pos, freq, dims, **opts)
    # every second one of them is a value that a product or a sum would change or spread
    odd = torch.nonzero(left).flatten()
    odd = odd[torch.randperm(len(odd), generator=g)[:max(1, len(odd) // 2)].cuda()]
    values = torch.tensor([math.nan, math.inf, -math.inf, -0.0]).to(dtype).cuda()
    for x in (q, k):
        pick = torch.randint(0, 4, (*x.shape[:3], len(odd)), generator=g).cuda()
        x[..., odd] = values[pick]
        x.view(BITS[dtype])[0, 0, 0, odd[0]] |= 1  # a NaN or an infinity's neighbour: its bits
    for in_place in (False, True):
        a, b = (q.clone(), k.clone()) if in_place else (q, k)
        got_q, got_k = ltxattn.rope_axes(a, b, pos, freq, dims, a if in_place else None,
                                         b if in_place else None, **opts)
        for got, x, want in ((got_q, q, want_q), (got_k, k, want_k)):
            assert torch.equal(got[..., left].view(BITS[dtype]), x[..., left].view(BITS[dtype]))
            assert torch.equal(got[..., ~left], want[..., ~left])
