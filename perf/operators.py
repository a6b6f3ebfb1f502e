"""Timed cases of the operators around attention: rotary positions with several axes, attention
with masked, capped and distance-biased scores (and its gradients), layer norm and its gradients.

`run` computes a case in its plain form (elementary torch operations in 32 bits) or, with `own`
true, through the calls of the package.  Workload sizes are those of an LTX-2 block (15360 video
tokens at 768x1280x121, 27280 at 1280x704x241, 126 or 252 audio tokens, 4096 video and 2048 audio
channels, heads of 128 and 64) and of a rank's share of its heads.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ITEM = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------- cases
def _rope(name, batch, length, heads, kv_heads, dim, axes, dtype="bf16", layout="pairs",
          inverse=False, own_positions=False, fused=True):
    """axes: "t-y-x" channels of each axis; own_positions: a grid of its own per batch row."""
    return {"name": name, "kind": "rope", "batch": batch, "length": length, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "axes": axes, "dtype": dtype, "layout": layout,
            "inverse": inverse, "own_positions": own_positions, "fused": fused}


def _attend(name, batch, q_len, kv_len, heads, kv_heads, dim, docs=0, tail=0, causal=False,
            prefix=0, cap=0.0, distance=False, train=False):
    """docs: documents per batch row (0 = one, without offsets); tail: rows behind the last
    document; prefix: keys at a document's start that every query of it sees."""
    return {"name": name, "kind": "attend", "batch": batch, "q_len": q_len, "kv_len": kv_len,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "docs": docs, "tail": tail,
            "causal": causal, "prefix": prefix, "cap": cap, "distance": distance, "train": train}


def _norm(name, rows, cols, groups, dtype="bf16", grad=False):
    """groups: 0 = no weight and bias, 1 = one for all rows, n = one per n-th of the rows."""
    return {"name": name, "kind": "norm", "rows": rows, "cols": cols, "groups": groups,
            "dtype": dtype, "grad": grad}


def listed():
    return [
        # the queries and keys of one new token per stream: launch latency
        _rope("rope_one_token", 2, 1, 32, 32, 64, "64"),
        # a clip's queries and keys as they come out of the fused projection, (t, y, x) positions
        _rope("rope_video", 1, 15360, 32, 32, 128, "44-42-42"),
        # the gradient in 32 bits: shared key heads, some channels unrotated, odd length, halves
        _rope("rope_grad_halves", 2, 4099, 16, 4, 64, "24-16-16", "fp32", "halves", True, True,
              False),
        # one new query per sample over the long clip's keys
        _attend("attend_one_query", 2, 1, 27280, 32, 8, 128, causal=True),
        # the audio stream, two clips and padding in a row, nearer tokens weigh more
        _attend("attend_audio_distance", 2, 252, 252, 32, 32, 64, docs=2, tail=4, distance=True),
        # a text prefix that everybody sees, then tokens in order; capped scores
        _attend("attend_prefix_capped", 1, 4173, 4173, 16, 2, 128, causal=True, prefix=257,
                cap=30.0),
        # clips of several lengths packed into one sequence of 15360 tokens, a rank's 8 heads with
        # keys and values shared by pairs of them
        _attend("attend_packed_clips", 1, 15360, 15360, 8, 4, 128, docs=5),
        # a training step's attention over packed clips
        _attend("train_packed_clips", 1, 7680, 7680, 16, 16, 128, docs=3, train=True),
        # a training step with every option at a ragged length and heads of 64
        _attend("train_every_option", 2, 1003, 1003, 12, 4, 64, docs=4, tail=9, causal=True,
                prefix=33, cap=20.0, distance=True, train=True),
        # the audio stream's norm with its own scale and shift per sample
        _norm("norm_audio", 252, 2048, 2),
        # the video stream's norm, backwards, scale and shift per sample
        _norm("norm_grad_video", 30720, 4096, 2, grad=True),
        # an odd width in 32 bits, backwards, one weight
        _norm("norm_grad_odd", 5001, 1537, 1, "fp32", grad=True),
    ]


def _spread(rng, low, high):
    """A whole number, evenly spread over the logarithm of its range."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    kind = rng.choice(("rope", "attend", "attend", "attend", "norm"))
    if kind == "rope":
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        dim = rng.choice((64, 128))
        heads, kv_heads = rng.choice(((32, 32), (32, 8), (16, 4), (8, 8), (6, 2), (1, 1)))
        batch = rng.choice((1, 1, 2, 3))
        most = 15360 * 64 * 128 * 2 // (batch * (heads + kv_heads) * dim * ITEM[dtype])
        axes = rng.choice({64: ("64", "24-20-20", "16-24-16", "32-32"),
                           128: ("128", "44-42-42", "32-48-48", "64-64", "32-32-32-32")}[dim])
        return _rope("", batch, _spread(rng, 1, min(most, 27280)), heads, kv_heads, dim, axes,
                     dtype, rng.choice(("pairs", "halves")), rng.random() < 0.4,
                     rng.random() < 0.5, rng.random() < 0.6)
    if kind == "norm":
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        cols = rng.choice((2048, 4096, _spread(rng, 1, 8192)))
        groups = rng.choice((0, 1, 2, 3))
        rows = _spread(rng, 1, 30720 * 4096 * 2 // (cols * ITEM[dtype]))
        rows = min(rows, 200000)
        return _norm("", max(groups, 1) * max(1, rows // max(groups, 1)), cols, groups, dtype,
                     rng.random() < 0.6)
    train = rng.random() < 0.5
    dim = rng.choice((64, 128))
    heads, kv_heads = rng.choice(((8, 8), (16, 4), (12, 4), (32, 8), (6, 2), (5, 1), (1, 1)))
    batch = rng.choice((1, 1, 2))
    most = (7680 * 7680 * 16 if train else 15360 * 15360 * 8) // (batch * heads)
    shape = rng.choice(("self", "self", "cross", "few"))
    if shape == "few":
        q_len = rng.choice((1, 1, 2, 5, 16))
        kv_len = _spread(rng, 1, min(27280, most // q_len))
    else:
        q_len = _spread(rng, 1, min(15360, math.isqrt(most)))
        kv_len = q_len if shape == "self" else _spread(rng, 1, min(15360, most // q_len))
    docs = rng.choice((0, 1, 2, 5)) if min(q_len, kv_len) >= 16 else 0
    causal = rng.random() < 0.5
    return _attend("", batch, q_len, kv_len, heads, kv_heads, dim, docs=docs,
                   tail=rng.choice((0, 3)) if docs else 0, causal=causal,
                   prefix=_spread(rng, 1, kv_len) if causal and rng.random() < 0.5 else 0,
                   cap=rng.choice((0.0, 0.0, 10.0, 50.0)), distance=rng.random() < 0.3,
                   train=train)


def _lengths(total, docs, turn):
    """Lengths of `docs` documents that fill `total` rows: uneven, the third of four or more
    empty; every batch row (`turn`) has them in another order."""
    parts = [3 + (5 * i + 2 * turn) % 7 for i in range(docs)]
    if docs >= 4:
        parts[2] = 0
    lengths = [total * p // sum(parts) for p in parts]
    lengths[-1] += total - sum(lengths)
    return lengths


def _documents(case, b):
    """(query start, queries, key start, keys, prefix) of every document of batch row b."""
    if not case["docs"]:
        return [(0, case["q_len"], 0, case["kv_len"], min(case["prefix"], case["kv_len"]))]
    found, q0, k0 = [], 0, 0
    for nq, nk in zip(_lengths(case["q_len"] - case["tail"], case["docs"], b),
                      _lengths(case["kv_len"] - case["tail"], case["docs"], b)):
        found.append((q0, nq, k0, nk, min(case["prefix"], nk)))
        q0, k0 = q0 + nq, k0 + nk
    return found


def _visible_pairs(case):
    n = 0
    for b in range(case["batch"]):
        for _, nq, _, nk, prefix in _documents(case, b):
            if not case["causal"]:
                n += nq * nk
            else:
                i = torch.arange(nq, dtype=torch.int64)
                n += int((i + 1 + nk - nq).clamp(min=prefix, max=nk).clamp(min=0).sum())
    return n


def work(case):
    if case["kind"] == "rope":
        n = case["batch"] * case["length"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        axes = len(case["axes"].split("-"))
        rows = case["batch"] if case["own_positions"] else 1
        return {"bytes": 2 * n * ITEM[case["dtype"]] + 4 * rows * case["length"] * axes,
                "flops": 3 * n}
    if case["kind"] == "norm":
        n, item = case["rows"] * case["cols"], ITEM[case["dtype"]]
        affine = case["groups"] * case["cols"]
        if case["grad"]:  # x, dy, weight and statistics in; dx and the two gradients out
            return {"bytes": 3 * n * item + affine * (item + 8) + 8 * case["rows"],
                    "flops": 12 * n}
        return {"bytes": 2 * n * item + 2 * affine * item, "flops": 7 * n}
    q = case["batch"] * case["q_len"] * case["heads"] * case["dim"]
    kv = case["batch"] * case["kv_len"] * case["kv_heads"] * case["dim"]
    lse = 4 * case["batch"] * case["q_len"] * case["heads"]
    pairs = _visible_pairs(case) * case["heads"] * case["dim"]
    if case["train"]:  # q, k, v, d_out in; out, lse, dq, dk, dv out
        return {"bytes": 2 * (4 * q + 4 * kv) + lse, "flops": 14 * pairs}
    return {"bytes": 2 * (2 * q + 2 * kv) + lse, "flops": 4 * pairs}


# ---------------------------------------------------------------------------- inputs
def _frequencies(axes, base=10000.0):
    """Radians per position of every rotated channel pair, axis after axis."""
    return [base ** (-2.0 * i / d) for d in axes for i in range(d // 2)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if case["kind"] == "rope":
        dtype = DTYPES[case["dtype"]]
        b, n, h, hk, d = (case[x] for x in ("batch", "length", "heads", "kv_heads", "dim"))
        axes = [int(x) for x in case["axes"].split("-")]
        if case["fused"]:  # views of the fused projection's output
            qkv = normal(b, n, h + 2 * hk, d, dtype=dtype)
            q, k = qkv[:, :, :h], qkv[:, :, h:h + hk]
        else:
            q, k = normal(b, n, h, d, dtype=dtype), normal(b, n, hk, d, dtype=dtype)
        # frame times in seconds at 24 frames, rows and columns of a 24 x 40 grid; a clip of
        # its own per batch row starts elsewhere
        token = torch.arange(n, device="cuda")
        grid = [(token // 960) / 24.0, (token // 40) % 24, token % 40, token]
        start = torch.randint(0, 5000, (b if case["own_positions"] else 1, 1, len(axes)),
                              generator=g, device="cuda")
        positions = torch.stack([x.float() for x in grid[:len(axes)]], dim=-1)[None] + start
        freq = _frequencies(axes)
        return {"case": case, "q": q, "k": k, "positions": positions.float().contiguous(),
                "freq": freq, "axes": axes,
                "freq_gpu": torch.tensor(freq, dtype=torch.float64, device="cuda")}

    if case["kind"] == "norm":
        dtype = DTYPES[case["dtype"]]
        x = (normal(case["rows"], case["cols"], dtype=torch.float32) * 2 + 0.5).to(dtype)
        s = {"case": case, "x": x, "weight": None, "bias": None, "eps": 1e-6}
        if case["groups"]:
            shape = (case["cols"],) if case["groups"] == 1 else (case["groups"], case["cols"])
            s["weight"] = (1 + 0.2 * normal(*shape, dtype=torch.float32)).to(dtype)
            s["bias"] = (0.1 * normal(*shape, dtype=torch.float32)).to(dtype)
        if case["grad"]:  # what the forward pass has left
            s["dy"] = normal(case["rows"], case["cols"], dtype=dtype)
            s["mean"] = x.float().mean(dim=1)
            s["rstd"] = ((x.float() - s["mean"][:, None]).square().mean(dim=1) + 1e-6).rsqrt()
        return s

    b, h, hk, d = (case[x] for x in ("batch", "heads", "kv_heads", "dim"))
    nq, nk = case["q_len"], case["kv_len"]
    if nq == nk:  # self-attention: views of the fused projection's output
        qkv = normal(b, nq, h + 2 * hk, d)
        q, k, v = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
    else:
        q, k, v = normal(b, nq, h, d), normal(b, nk, hk, d), normal(b, nk, hk, d)
    s = {"case": case, "q": q, "k": k, "v": v, "scale": 1 / math.sqrt(d), "cap": case["cap"],
         "causal": case["causal"], "slopes": None, "q_starts": None, "kv_starts": None,
         "prefix": None}
    if case["cap"]:  # scores near the cap, where it bends
        s["scale"] *= 4.0
    if case["distance"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")
    rows = [_documents(case, i) for i in range(b)]
    if case["docs"]:
        s["q_starts"], s["kv_starts"] = (
            torch.tensor([[r[0][at]] + [x[at] + x[at + 1] for x in r] for r in rows],
                         dtype=torch.int32, device="cuda") for at in (0, 2))
    if case["prefix"]:
        s["prefix"] = torch.tensor([[x[4] for x in r] for r in rows], dtype=torch.int32,
                                   device="cuda")
    # what the program keeps for the results; rows of no document stay as they are here
    s["out"] = torch.zeros(b, nq, h, d, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.full((b, h, nq), -math.inf, device="cuda")
    if case["train"]:
        s["d_out"] = normal(b, nq, h, d)
        s["dq"] = torch.zeros_like(s["out"])
        s["dk"], s["dv"] = (torch.zeros(b, nk, hk, d, dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
    return s


# ---------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, layout):
    y = x.float()
    if layout == "pairs":
        a, c = y[..., 0::2], y[..., 1::2]
        return torch.stack((a * cos - c * sin, a * sin + c * cos), dim=-1).flatten(-2).to(x.dtype)
    a, c = y.chunk(2, dim=-1)
    return torch.cat((a * cos - c * sin, a * sin + c * cos), dim=-1).to(x.dtype)


def _plain_rope(s):
    case, half = s["case"], s["case"]["dim"] // 2
    axis = torch.repeat_interleave(torch.arange(len(s["axes"]), device="cuda"),
                                   torch.tensor(s["axes"], device="cuda") // 2)
    angle = s["positions"].double()[..., axis] * s["freq_gpu"]
    angle = torch.nn.functional.pad(angle, (0, half - angle.shape[-1]))[:, :, None]
    if case["inverse"]:
        angle = -angle
    cos, sin = angle.cos().float(), angle.sin().float()
    return {"q": _rotate(s["q"], cos, sin, case["layout"]),
            "k": _rotate(s["k"], cos, sin, case["layout"])}


def _place(starts, length, batch):
    """Document, place in it and the documents' lengths of every row; rows of none have -1."""
    i = torch.arange(length, device="cuda")[None].expand(batch, length).contiguous()
    if starts is None:
        return torch.zeros_like(i), i, torch.full((batch, 1), length, device="cuda")
    starts = starts.long()
    doc = torch.searchsorted(starts[:, 1:].contiguous(), i, right=True)
    inside = (i >= starts[:, :1]) & (doc < starts.shape[1] - 1)
    place = i - starts.gather(1, doc.clamp(max=starts.shape[1] - 2))
    return torch.where(inside, doc, -1), place, starts[:, 1:] - starts[:, :-1]


def _plain_attend(s):
    case = s["case"]
    b, h, hk, d = (case[x] for x in ("batch", "heads", "kv_heads", "dim"))
    nq, nk, group = case["q_len"], case["kv_len"], h // hk
    q_doc, q_at, q_n = _place(s["q_starts"], nq, b)
    k_doc, k_at, k_n = _place(s["kv_starts"], nk, b)
    doc = q_doc.clamp(min=0)
    at = q_at + (k_n - q_n).gather(1, doc)  # the last query stands at the last key
    seen = (q_doc[:, :, None] == k_doc[:, None, :]) & (q_doc >= 0)[:, :, None]
    if s["causal"]:
        early = k_at[:, None, :] <= at[:, :, None]
        if s["prefix"] is not None:
            early |= k_at[:, None, :] < s["prefix"].long().gather(1, doc)[:, :, None]
        seen &= early
    hidden = ~seen[:, None, None]
    # [batch, key head, query heads of it, rows, channels]
    qf = s["q"].float().view(b, nq, hk, group, d).permute(0, 2, 3, 1, 4)
    kf = s["k"].float().permute(0, 2, 1, 3)[:, :, None]
    vf = s["v"].float().permute(0, 2, 1, 3)[:, :, None]
    p = torch.matmul(qf * s["scale"], kf.transpose(-1, -2))
    bend = None
    if s["cap"]:
        p = torch.tanh(p.div_(s["cap"]))
        if case["train"]:
            bend = p.square().neg_().add_(1)
        p = p.mul_(s["cap"])
    if s["slopes"] is not None:
        far = (at[:, :, None] - k_at[:, None, :]).abs().float()
        p = p.sub_(s["slopes"].view(1, hk, group, 1, 1) * far[:, None, None])
    p.masked_fill_(hidden, -math.inf)
    top = p.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = ((total.log() + top) * math.log2(math.e))[..., 0].reshape(b, h, nq)
    p = p.div_(torch.where(total == 0, 1.0, total))
    out = torch.matmul(p, vf)

    def back(x, heads, length):
        return x.permute(0, 3, 1, 2, 4).reshape(b, length, heads, d).to(torch.bfloat16)

    r = {"out": back(out, h, nq), "lse": lse}
    if case["train"]:
        do = s["d_out"].float().view(b, nq, hk, group, d).permute(0, 2, 3, 1, 4)
        r["dv"] = back(torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True), hk, nk)
        ds = torch.matmul(do, vf.transpose(-1, -2))
        ds = ds.sub_((do * out).sum(dim=-1, keepdim=True)).mul_(p)
        del p
        if bend is not None:
            ds = ds.mul_(bend)
        r["dq"] = back(torch.matmul(ds, kf) * s["scale"], h, nq)
        r["dk"] = back(torch.matmul(ds.transpose(-1, -2), qf * s["scale"]).sum(2, keepdim=True),
                       hk, nk)
    return r


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    groups = max(case["groups"], 1)
    parts = (groups, case["rows"] // groups, case["cols"])
    if not case["grad"]:
        y = x - x.mean(dim=1, keepdim=True)
        y = y * torch.rsqrt(y.square().mean(dim=1, keepdim=True) + s["eps"])
        if s["weight"] is not None:
            y = y.view(parts) * s["weight"].float().view(groups, 1, -1) \
                + s["bias"].float().view(groups, 1, -1)
        return {"y": y.view(x.shape).to(s["x"].dtype)}
    dy = s["dy"].float()
    normed = (x - s["mean"][:, None]) * s["rstd"][:, None]
    r = {}
    if s["weight"] is not None:
        r["dweight"] = (dy * normed).view(parts).sum(dim=1).view(s["weight"].shape)
        r["dbias"] = dy.view(parts).sum(dim=1).view(s["weight"].shape)
        dy = (dy.view(parts) * s["weight"].float().view(groups, 1, -1)).view(x.shape)
    r["dx"] = (s["rstd"][:, None] * (dy - dy.mean(dim=1, keepdim=True)
                                     - normed * (dy * normed).mean(dim=1, keepdim=True))
               ).to(s["x"].dtype)
    return r


# ---------------------------------------------------------------------------- one pass
def _own(s):
    from joint_audio_video_flash_b200 import ltxattn

    ltxattn.create()  # a no-op after the first call
    case = s["case"]
    if case["kind"] == "rope":
        q, k = ltxattn.rope_axes(s["q"], s["k"], s["positions"], s["freq"], s["axes"],
                                 layout=case["layout"], inverse=case["inverse"])
        return {"q": q, "k": k}
    if case["kind"] == "norm":
        if not case["grad"]:
            return {"y": ltxattn.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"])}
        dx, dweight, dbias = ltxattn.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"],
                                                         s["weight"])
        return {"dx": dx} if dweight is None else {"dx": dx, "dweight": dweight, "dbias": dbias}
    options = {"scale": s["scale"], "softcap": s["cap"], "slopes": s["slopes"],
               "causal": s["causal"], "prefix": s["prefix"], "q_starts": s["q_starts"],
               "kv_starts": s["kv_starts"]}
    out, lse = ltxattn.masked_forward(s["q"], s["k"], s["v"], s["out"], s["lse"], **options)
    r = {"out": out, "lse": lse}
    if case["train"]:
        r["dq"], r["dk"], r["dv"] = ltxattn.masked_backward(
            s["d_out"], s["q"], s["k"], s["v"], out, lse, s["dq"], s["dk"], s["dv"], **options)
    return r


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "attend": _plain_attend, "norm": _plain_norm}[
        state["case"]["kind"]](state)


# ---------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        half = case["dim"] // 2
        sign = -1.0 if case["inverse"] else 1.0
        answer = {}
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            pair = 0
            for axis, channels in enumerate(s["axes"]):
                for _ in range(channels // 2):
                    angle = sign * s["freq"][pair] * s["positions"][:, :, axis].double()
                    i, j = (2 * pair, 2 * pair + 1) if case["layout"] == "pairs" \
                        else (pair, pair + half)
                    c, n = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
                    y[..., i] = c * x[..., i] - n * x[..., j]
                    y[..., j] = n * x[..., i] + c * x[..., j]
                    pair += 1
            answer[name] = y
        return answer
    if case["kind"] == "norm":
        x = s["x"].double()
        groups = max(case["groups"], 1)
        n = case["rows"] // groups
        if not case["grad"]:
            y = torch.empty_like(x)
            for g in range(groups):
                part = x[g * n:(g + 1) * n]
                var, mean = torch.var_mean(part, dim=1, unbiased=False, keepdim=True)
                part = (part - mean) / torch.sqrt(var + s["eps"])
                if s["weight"] is not None:
                    part = part * s["weight"].double().view(groups, -1)[g] \
                        + s["bias"].double().view(groups, -1)[g]
                y[g * n:(g + 1) * n] = part
            return {"y": y}
        dx, dw, db = torch.empty_like(x), [], []
        for g in range(groups):
            at = slice(g * n, (g + 1) * n)
            dy, rstd = s["dy"][at].double(), s["rstd"][at].double()[:, None]
            z = (x[at] - s["mean"][at].double()[:, None]) * rstd
            dw.append((dy * z).sum(0))
            db.append(dy.sum(0))
            if s["weight"] is not None:
                dy = dy * s["weight"].double().view(groups, -1)[g]
            dx[at] = rstd * (dy - dy.mean(1, keepdim=True) - z * (dy * z).mean(1, keepdim=True))
        if s["weight"] is None:
            return {"dx": dx}
        shape = s["weight"].shape
        return {"dx": dx, "dweight": torch.stack(dw).view(shape), "dbias": torch.stack(db).view(shape)}
    # attention: one document, one query head at a time, a stretch of its queries
    h, group, cap = case["heads"], case["heads"] // case["kv_heads"], case["cap"]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    out = torch.zeros(s["out"].shape, **f64)
    lse = torch.full(s["lse"].shape, -math.inf, **f64)
    if case["train"]:
        dq = torch.zeros(s["dq"].shape, **f64)
        dk, dv = torch.zeros(s["dk"].shape, **f64), torch.zeros(s["dv"].shape, **f64)
    for b in range(case["batch"]):
        for q0, nq, k0, nk, prefix in _documents(case, b):
            if nq == 0 or nk == 0:
                continue
            j = torch.arange(nk, device="cuda")
            for head in range(h):
                k = s["k"][b, k0:k0 + nk, head // group].double()
                v = s["v"][b, k0:k0 + nk, head // group].double()
                for first in range(0, nq, 4096):
                    last = min(first + 4096, nq)
                    at = slice(q0 + first, q0 + last)
                    i = torch.arange(first, last, device="cuda")[:, None] + (nk - nq)
                    q = s["q"][b, at, head].double()
                    score = q @ k.T * s["scale"]
                    slope = torch.ones((), **f64)
                    if cap:
                        bent = torch.tanh(score / cap)
                        score, slope = bent * cap, 1 - bent * bent
                    if s["slopes"] is not None:
                        score = score - s["slopes"][head].double() * (i - j).abs()
                    if case["causal"]:
                        score[(j > i) & (j >= prefix)] = -math.inf
                    line = torch.logsumexp(score, dim=1)
                    weight = torch.nan_to_num(torch.exp(score - line[:, None]), nan=0.0)
                    out[b, at, head] = o = weight @ v
                    lse[b, head, at] = line / math.log(2.0)
                    if case["train"]:
                        do = s["d_out"][b, at, head].double()
                        dv[b, k0:k0 + nk, head // group] += weight.T @ do
                        g = weight * (do @ v.T - (do * o).sum(1, keepdim=True)) * slope
                        dq[b, at, head] = g @ k * s["scale"]
                        dk[b, k0:k0 + nk, head // group] += g.T @ q * s["scale"]
    r = {"out": out, "lse": lse}
    return {**r, "dq": dq, "dk": dk, "dv": dv} if case["train"] else r
