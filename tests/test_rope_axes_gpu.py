"""Rotary positions with several axes against their fp64 definition (needs a B200).

Bounds: the output's rounding (half a unit in the last place) and 2^-21 of the rotated pair
for the sine, the cosine and the angle (oracle/block_ops.py).
"""
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
    ltxattn.load()


def grid_positions(batch, length, axes, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(batch, length, axes, generator=g) * 2000 - 300) * scale


def check(got, x, positions, freq, dims, layout, inverse):
    ref, bound = block_ops.rope_axes(x.cpu(), positions.cpu(), freq, dims, layout, inverse)
    err = (got.cpu().double() - ref).abs()
    bound = block_ops.rounded(ref, bound, x.dtype)
    assert torch.all(err <= bound), float((err / bound).max())


CASES = [
    # batch, len, heads, kv_heads, dim, axes, dtype, layout, inverse, positions per batch row
    (1, 1, 1, 1, 8, (8,), torch.bfloat16, "pairs", False, True),
    (2, 1, 32, 32, 64, (24, 20, 20), torch.bfloat16, "pairs", False, False),
    (2, 37, 8, 2, 128, (44, 42, 42), torch.bfloat16, "pairs", False, True),
    (2, 37, 8, 2, 128, (44, 42, 42), torch.bfloat16, "halves", True, True),
    (1, 300, 5, 1, 96, (32, 0, 30), torch.float16, "pairs", False, True),
    (3, 129, 3, 3, 80, (16, 16, 16, 16), torch.float16, "halves", True, False),
    (1, 513, 40, 8, 64, (64,), torch.float32, "pairs", True, True),
    (2, 65, 2, 1, 512, (172, 170, 170), torch.float32, "halves", False, True),
    (1, 19, 1, 1, 16, (2,), torch.float32, "halves", False, True),
    (1, 700, 2, 1, 40, (20, 20), torch.bfloat16, "pairs", False, True),  # 5 chunks a head
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_matches_definition(case):
    batch, length, heads, kv_heads, dim, dims, dtype, layout, inverse, own = case
    g = torch.Generator().manual_seed(length + heads)
    q = torch.randn(batch, length, heads, dim, generator=g).to(dtype).cuda()
    k = torch.randn(batch, length, kv_heads, dim, generator=g).to(dtype).cuda()
    pos = grid_positions(batch if own else 1, length, len(dims), 3).cuda()
    freq = ltxattn.rope_frequencies(dims)
    qo, ko = ltxattn.rope_axes(q, k, pos, freq, dims, layout=layout, inverse=inverse)
    for got, x in ((qo, q), (ko, k)):
        check(got, x, pos, freq, dims, layout, inverse)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 400.0, 8000.0])
def test_far_positions_keep_their_angles(scale):
    # positions to 1.6e7 (angles of 2.5 million turns): fp32 angles would be off by radians
    pos = grid_positions(1, 200, 2, 5, scale).cuda()
    q = torch.randn(1, 200, 2, 64, generator=torch.Generator().manual_seed(1)).cuda()
    freq = ltxattn.rope_frequencies((32, 32))
    got, none = ltxattn.rope_axes(q, None, pos, freq, (32, 32))
    assert none is None
    check(got, q, pos, freq, (32, 32), "pairs", False)


@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_views_in_place_and_back(layout):
    # queries and keys are parts of one projection's rows; the rest of it stays as it is
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(2, 50, 8 + 2 * 4, 64, generator=g).bfloat16().cuda()
    before = qkv.clone()
    q, k = qkv[:, :, :8], qkv[:, :, 8:12]
    pos = grid_positions(2, 50, 3, 4).cuda()
    dims, freq = (24, 20, 20), ltxattn.rope_frequencies((24, 20, 20))
    qo, ko = ltxattn.rope_axes(q, k, pos, freq, dims, layout=layout)
    ltxattn.rope_axes(q, k, pos, freq, dims, q_out=q, k_out=k, layout=layout)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, :, 12:], before[:, :, 12:])
    # head-major tensors
    qh = before[:, :, :8].transpose(1, 2).contiguous().transpose(1, 2)
    kh = before[:, :, 8:12].transpose(1, 2).contiguous().transpose(1, 2)
    a, b = ltxattn.rope_axes(qh, kh, pos, freq, dims, layout=layout)
    assert torch.equal(a, qo) and torch.equal(b, ko)
    # turning back gives the input to two roundings
    back, _ = ltxattn.rope_axes(qo, ko, pos, freq, dims, layout=layout, inverse=True)
    lim = 2 ** -8 * 3 * before[:, :, :8].float().abs().amax()
    assert (back.float() - before[:, :, :8].float()).abs().max() <= lim


def test_gradient_against_differences():
    # L = sum(w * rope(x)): its gradient is the inverse rotation of w
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(2, 1, 9, 2, 32, generator=g)
    pos = grid_positions(1, 9, 2, 8, 0.01).cuda()
    dims, freq = (16, 16), ltxattn.rope_frequencies((16, 16))
    grad, _ = ltxattn.rope_axes(w.cuda(), None, pos, freq, dims, inverse=True)
    direction = torch.randn(x.shape, generator=g)

    def loss(t):
        y, _ = ltxattn.rope_axes(t.float().cuda(), None, pos, freq, dims)
        return float((y.cpu().double() * w.double()).sum())

    # the rotation is linear: a difference of any step is exact but for fp32 rounding
    diff = (loss(x + direction) - loss(x - direction)) / 2
    exact = float((grad.cpu().double() * direction.double()).sum())
    assert abs(diff - exact) <= 2 ** -20 * float((w.abs() * 4).sum())


def test_other_stream_and_graph():
    q = torch.randn(1, 64, 4, 64).bfloat16().cuda()
    pos = grid_positions(1, 64, 1, 9).cuda()
    freq = ltxattn.rope_frequencies((64,))
    ref, _ = ltxattn.rope_axes(q, None, pos, freq, (64,))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = ltxattn.rope_axes(q, None, pos, freq, (64,), stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = ltxattn.rope_axes(q, None, pos, freq, (64,))
    q.copy_(torch.randn(q.shape))
    graph.replay()
    assert torch.equal(out, ltxattn.rope_axes(q, None, pos, freq, (64,))[0])


def test_refusals():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 4, 1, device="cuda")
    freq = ltxattn.rope_frequencies((64,))
    with pytest.raises(TypeError):
        ltxattn.rope_axes(q.double(), None, pos, freq, (64,))
    with pytest.raises(TypeError):
        ltxattn.rope_axes(q.cpu(), None, pos, freq, (64,))
    with pytest.raises(ValueError):
        ltxattn.rope_axes(q, None, pos, freq[:-1], (64,))
    with pytest.raises(ValueError):
        ltxattn.rope_axes(q, None, pos[:, :3], freq, (64,))
    with pytest.raises(ValueError):
        ltxattn.rope_axes(q.transpose(2, 3), None, pos, freq, (64,))
    with pytest.raises(ValueError):
        ltxattn.rope_axes(q, q.float(), pos, freq, (64,))
    with pytest.raises(ValueError):
        ltxattn.rope_axes(q, None, pos, freq, (64,), layout="interleaved")
    for bad in (dict(q_out=q.expand(1, 4, 2, 64)[:, :1].expand(1, 4, 2, 64)),  # one row for all
                dict(k=q.clone(), k_out=q)):                              # k_out is q
        with pytest.raises(ltxattn.LtxAttnError) as e:
            ltxattn.rope_axes(q, bad.pop("k", None), pos, freq, (64,), **bad)
        assert e.value.status == ltxattn.ERR_INVALID_ARG
    wide = torch.zeros(1, 4, 2, 66, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ltxattn.LtxAttnError) as e:
        ltxattn.rope_axes(wide[..., :64], None, pos, freq, (64,))
    assert e.value.status == ltxattn.ERR_MISALIGNED
    with pytest.raises(ltxattn.LtxAttnError) as e:
        ltxattn.rope_axes(wide, None, pos, freq, (64,))
    assert e.value.status == ltxattn.ERR_UNSUPPORTED
