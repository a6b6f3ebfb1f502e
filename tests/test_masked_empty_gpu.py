"""Masked attention over documents that hold no key, or no query, at all (needs a B200)."""
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


@pytest.mark.parametrize("opts", [{}, dict(causal=True), dict(softcap=10.0)], ids=str)
@pytest.mark.parametrize("q_len,kv_len,heads,kv_heads,dim", [
    (200, 200, 4, 2, 64),      # no parts
    (200, 4000, 2, 2, 128),    # key parts forwards and for dq
    (4000, 200, 2, 1, 64),     # query parts for dk and dv
])
@pytest.mark.parametrize("no", ["keys", "queries", "either"])
def test_nothing_to_see(no, q_len, kv_len, heads, kv_heads, dim, opts):
    g = torch.Generator().manual_seed(q_len)
    q, k, v, d_out = (torch.randn(2, n, h, dim, generator=g).bfloat16().cuda() for n, h in
                      ((q_len, heads), (kv_len, kv_heads), (kv_len, kv_heads), (q_len, heads)))
    qs = [3, q_len // 3, q_len // 2, q_len - 5] if no == "keys" else [9] * 4
    ks = [2, kv_len // 2, kv_len // 2, kv_len - 3] if no == "queries" else [7] * 4
    opts = dict(opts, q_starts=torch.tensor([qs] * 2, dtype=torch.int32).cuda(),
                kv_starts=torch.tensor([ks] * 2, dtype=torch.int32).cuda())
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, heads, q_len), 5.0, device="cuda")
    grads = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]

    def step():
        ltxattn.masked_forward(q, k, v, out, lse, **opts)
        ltxattn.masked_backward(d_out, q, k, v, out, lse, *grads, **opts)
        return [t.clone() for t in (out, lse, *grads)]  # what follows in the stream

    inside = [torch.zeros(n, dtype=torch.bool) for n in (q_len, kv_len)]
    inside[0][qs[0]:qs[-1]] = True
    inside[1][ks[0]:ks[-1]] = True
    for graph in (None, torch.cuda.CUDAGraph()):
        for t, mark in zip((out, lse, *grads), (7, 5, 7, 7, 7)):
            t.fill_(mark)
        torch.cuda.synchronize()
        if graph is None:
            got = step()
        else:
            with torch.cuda.graph(graph):
                got = step()
            graph.replay()
        torch.cuda.synchronize()
        ltxattn.check()
        for t, rows, mark, empty in (
                (got[0], inside[0], 7, 0), (got[1].transpose(1, 2), inside[0], 5, -math.inf),
                (got[2], inside[0], 7, 0), (got[3], inside[1], 7, 0), (got[4], inside[1], 7, 0)):
            assert torch.all(t[:, rows] == empty) and torch.all(t[:, ~rows] == mark)
