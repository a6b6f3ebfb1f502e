"""Masked attention over more documents than a warp has lanes (needs a B200)."""
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


def offsets(lengths, gap, tail):
    line = torch.cat([torch.tensor([gap]), gap + lengths.cumsum(0)])
    return line.int(), int(line[-1]) + tail


CASES = [
    # batch, documents, longest, heads, kv_heads, dim, options
    (1, 33, 300, 2, 2, 64, dict(causal=True)),
    (2, 64, 150, 4, 1, 128, dict(softcap=5.0)),        # packed heads
    (1, 65, 40, 2, 1, 64, dict(causal=True, prefix=True)),
    (2, 300, 9, 2, 2, 64, dict(bias=True)),
    (1, 1100, 5, 2, 1, 64, {}),
    (1, 2500, 3, 1, 1, 128, dict(causal=True, prefix=True)),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_many_documents(case):
    batch, docs, longest, heads, kv_heads, dim, o = case
    g = torch.Generator().manual_seed(docs)
    qs, ks, q_len, kv_len = [], [], 0, 0
    for b in range(batch):  # a fifth of them without a query or without a key
        for starts in (qs, ks):
            n = torch.randint(1, longest + 1, (docs,), generator=g)
            n[torch.rand(docs, generator=g) < 0.2] = 0
            line, length = offsets(n, 5 * b + 130 * (starts is qs), 3 - b)
            starts.append(line)
            q_len, kv_len = (max(q_len, length), kv_len) if starts is qs else \
                (q_len, max(kv_len, length))
    q, k, v, d_out = (torch.randn(batch, n, h, dim, generator=g).bfloat16() for n, h in (
        (q_len, heads), (kv_len, kv_heads), (kv_len, kv_heads), (q_len, heads)))
    opts = dict(q_starts=torch.stack(qs), kv_starts=torch.stack(ks), causal=o.get("causal", False),
                softcap=o.get("softcap", 0.0))
    if o.get("bias"):
        opts["slopes"] = torch.linspace(0.1, 0.3, heads)
    if o.get("prefix"):
        opts["prefix"] = torch.randint(0, longest + 2, (batch, docs), generator=g).int()
    ref = block_ops.masked(q, k, v, d_out=d_out, **opts)
    dev = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in opts.items()}
    x = [t.cuda() for t in (q, k, v, d_out)]
    got = {"out": torch.full_like(x[0], 7.0),
           "lse": torch.full((batch, heads, q_len), 7.0, device="cuda")}
    ltxattn.masked_forward(*x[:3], got["out"], got["lse"], **dev)
    got.update({n: torch.full_like(t, 7.0) for n, t in zip(("dq", "dk", "dv"), x)})
    ltxattn.masked_backward(x[3], *x[:3], got["out"], got["lse"], got["dq"], got["dk"], got["dv"],
                            **dev)
    ltxattn.check()
    for b in range(batch):
        rows, keys = (torch.zeros(n, dtype=torch.bool) for n in (q_len, kv_len))
        rows[int(qs[b][0]):int(qs[b][-1])] = True
        keys[int(ks[b][0]):int(ks[b][-1])] = True
        for n, inside in (("out", rows), ("lse", rows), ("dq", rows), ("dk", keys), ("dv", keys)):
            t, want, err = (a[b].cpu().double() for a in (got[n], ref[n], ref[n + "_err"]))
            if n == "lse":
                t, want, err = t.T, want.T, err.T
            assert torch.all(t[~inside] == 7), n
            t, want, err = t[inside], want[inside], err[inside]
            assert torch.all(((t - want).abs() <= err + 1e-30) | (t == want)), n


def test_the_most_documents_end_soon():
    # one token each: out is v, and no CTA walks the documents ahead of its own (which took 370 ms
    # forwards and 630 ms backwards)
    docs = 65535
    q, k, v, d_out = (torch.randn(1, docs, 1, 64, device="cuda").bfloat16() for _ in range(4))
    s = torch.arange(docs + 1, dtype=torch.int32, device="cuda")[None].contiguous()
    opts = dict(q_starts=s, kv_starts=s)
    out, lse = ltxattn.masked_forward(q, k, v, **opts)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    events[0].record()
    ltxattn.masked_forward(q, k, v, **opts)
    dq, dk, dv = ltxattn.masked_backward(d_out, q, k, v, out, lse, **opts)
    events[1].record()
    torch.cuda.synchronize()
    ltxattn.check()
    assert torch.equal(out, v) and torch.equal(dv, d_out) and not dq.any() and not dk.any()
    assert events[0].elapsed_time(events[1]) < 100


def test_many_offsets_that_break_the_rules_stay_inside():
    # the kernels hold every offset inside the tensor; only that is checked here
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, 500, 2, 64, generator=g).bfloat16().cuda() for _ in range(3))
    s = torch.randint(-1000, 1500, (1, 201), generator=g).int().cuda()
    out, lse = ltxattn.masked_forward(q, k, v, q_starts=s, kv_starts=s.flip(1).contiguous())
    ltxattn.masked_backward(q, q, k, v, out, lse, q_starts=s, kv_starts=s.flip(1).contiguous())
    ltxattn.check()
