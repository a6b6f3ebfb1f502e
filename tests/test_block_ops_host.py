"""Rotary axes, layer norm and masked attention: arguments that the C ABI refuses on the host,
before any CUDA call, and the structs' layout (no GPU needed)."""
import ctypes
import re

import pytest

from joint_audio_video_flash_b200 import build, ltxattn

INVALID, UNSUPPORTED, MISALIGNED = (ltxattn.ERR_INVALID_ARG, ltxattn.ERR_UNSUPPORTED,
                                    ltxattn.ERR_MISALIGNED)
# fake, never dereferenced device addresses, 256 MB apart
A, B, C, D, E, F, G, H = ((i + 1) << 28 for i in range(8))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ltxattn.load()


def reaches_cuda(lib, status):
    """No device here: a call whose arguments pass ends at its first CUDA call."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-only expectation: no CUDA device")
    return status in (ltxattn.ERR_CUDA, ltxattn.ERR_NOT_INITIALIZED)


@pytest.mark.parametrize("struct,name", [
    (ltxattn._RopeCall, "ltxattn_rope_call"), (ltxattn._MaskedCall, "ltxattn_masked_call"),
    (ltxattn._MaskedGrad, "ltxattn_masked_grad")])
def test_struct_fields_follow_the_header(struct, name):
    with open(ltxattn.HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
    declared = []
    for line in body.split(";"):
        line = re.sub(r"\[\d+\]", "", line.strip()).replace("*", " ")
        if line:
            first, *rest = line.split(",")
            declared += [first.split()[-1]] + [x.strip() for x in rest]
    assert [f[0] for f in struct._fields_] == declared


def rope(lib, **kw):
    shape = dict(batch=2, len=16, heads=4, kv_heads=2, head_dim=64)
    shape.update({k: kw.pop(k) for k in list(kw) if k in shape})
    n, h, hk, d = (shape[x] for x in ("len", "heads", "kv_heads", "head_dim"))
    dims = kw.pop("axis_dims", (24, 20, 20))
    freq = kw.pop("freq", [1.0] * max(1, sum(x // 2 for x in dims if x > 0)))
    a = dict(q=A, k=B, q_out=C, k_out=D, q_stride=(n * h * d, h * d, d),
             k_stride=(n * hk * d, hk * d, d), q_out_stride=(n * h * d, h * d, d),
             k_out_stride=(n * hk * d, hk * d, d), positions=E,
             inv_freq=(ctypes.c_double * len(freq))(*freq) if freq else None,
             axis_dims=tuple(dims) + (0,) * (4 - len(dims)), axes=len(dims), positions_batch=1,
             dtype=0, layout=0, inverse=0)
    a.update(shape)
    a.update(kw)
    return lib.ltxattn_rope_axes(ctypes.byref(ltxattn._RopeCall(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k_out=None), INVALID),
    (dict(k=None), INVALID), (dict(positions=None), INVALID), (dict(inv_freq=None), INVALID),
    (dict(batch=0), INVALID), (dict(len=0), INVALID), (dict(heads=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(dtype=3), INVALID), (dict(layout=2), INVALID),
    (dict(positions_batch=3), INVALID), (dict(axes=0), INVALID), (dict(axes=5), UNSUPPORTED),
    (dict(axis_dims=(3, 20)), INVALID), (dict(axis_dims=(-2, 20)), INVALID),
    (dict(axis_dims=(0, 0)), INVALID), (dict(axis_dims=(64, 2)), INVALID),
    (dict(freq=[float("nan")] * 32), INVALID), (dict(freq=[float("inf")] * 32), INVALID),
    (dict(head_dim=60, axis_dims=(24, 20)), UNSUPPORTED), (dict(head_dim=72, layout=1), UNSUPPORTED),
    (dict(head_dim=520), UNSUPPORTED), (dict(heads=1025), UNSUPPORTED),
    (dict(batch=1025), UNSUPPORTED), (dict(len=(1 << 24) + 1), UNSUPPORTED),
    (dict(batch=1024, len=1 << 24), UNSUPPORTED),
    (dict(q=A + 8), MISALIGNED), (dict(k_out=D + 2), MISALIGNED),
    (dict(positions=E + 2), MISALIGNED), (dict(q_stride=(4096, 256, 68)), MISALIGNED),
    (dict(q_stride=(-4096, 256, 64)), INVALID),            # backwards
    (dict(q_out_stride=(0, 256, 64)), INVALID),            # batch rows on one another
    (dict(q_out=A + 4096), INVALID),                       # overlaps q
    (dict(q_out=B), INVALID), (dict(k_out=C), INVALID), (dict(k_out=A), INVALID),
    (dict(q_out=E), INVALID),                              # positions would change
])
def test_rope_refusals(lib, kw, status):
    assert rope(lib, **kw) == status


def test_rope_accepts_views(lib):
    assert reaches_cuda(lib, rope(lib))
    assert reaches_cuda(lib, rope(lib, q_out=A, k_out=B))                       # in place
    assert reaches_cuda(lib, rope(lib, k=None, k_out=None))
    # parts of one projection's rows of 8 heads, in place
    row, d = 8 * 64, 64
    view = dict(q_stride=(16 * row, row, d), q_out_stride=(16 * row, row, d),
                k_stride=(16 * row, row, d), k_out_stride=(16 * row, row, d))
    assert reaches_cuda(lib, rope(lib, q_out=A, k=A + 4 * d * 2, k_out=A + 4 * d * 2, **view))
    # ... but not parts that run into one another
    assert rope(lib, q_out=A, k=A + 3 * d * 2, k_out=A + 3 * d * 2, **view) == INVALID


def norm(lib, x=A, w=B, b=C, out=D, mean=None, rstd=None, rows=8, cols=64, groups=1, xs=64,
         os_=64, eps=1e-6, dtype=0):
    return lib.ltxattn_layer_norm(x, w, b, out, mean, rstd, rows, cols, groups, xs, os_, eps,
                                  dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(w=None), INVALID),
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(groups=0), INVALID),
    (dict(groups=3), INVALID), (dict(xs=63), INVALID), (dict(os_=10), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(dtype=7), INVALID),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(cols=(1 << 20) + 1, xs=1 << 21, os_=1 << 21), UNSUPPORTED),
    (dict(x=A + 1), MISALIGNED), (dict(dtype=2, w=B + 2), MISALIGNED),
    (dict(mean=E + 2), MISALIGNED),
    (dict(out=A + 2), INVALID), (dict(out=A, os_=72), INVALID), (dict(out=B), INVALID),
    (dict(mean=A), INVALID), (dict(mean=E, rstd=E + 4), INVALID), (dict(rstd=C), INVALID),
])
def test_layer_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def test_layer_norm_accepts(lib):
    for kw in (dict(), dict(w=None, b=None), dict(b=None), dict(out=A), dict(x=A + 2),
               dict(mean=E, rstd=F, groups=8)):
        assert reaches_cuda(lib, norm(lib, **kw))


def norm_grad(lib, dy=A, x=B, w=C, mean=D, rstd=E, dx=F, dw=G, db=G + 4096, rows=8, cols=64,
              groups=1, dys=64, xs=64, dxs=64, dtype=0, ws=H, bytes_=1 << 20):
    return lib.ltxattn_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, rows, cols, groups,
                                           dys, xs, dxs, dtype, ws, bytes_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dx=None), INVALID), (dict(rows=0), INVALID),
    (dict(groups=5), INVALID), (dict(dys=1), INVALID), (dict(dxs=63), INVALID),
    (dict(dtype=-1), INVALID), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(dy=A + 1), MISALIGNED), (dict(dw=G + 1), MISALIGNED), (dict(ws=H + 2), MISALIGNED),
    (dict(dx=A + 2), INVALID), (dict(dx=A, dxs=128), INVALID), (dict(dw=A), INVALID),
    (dict(db=G + 8), INVALID), (dict(dw=D), INVALID), (dict(ws=B), INVALID), (dict(dx=C), INVALID),
])
def test_layer_norm_grad_refusals(lib, kw, status):
    assert norm_grad(lib, **kw) == status


def test_norm_workspace_refusals(lib):
    n = ctypes.c_ulonglong(0)
    assert lib.ltxattn_layer_norm_workspace(8, 64, 1, 0, None) == INVALID
    assert lib.ltxattn_layer_norm_workspace(8, 64, 3, 0, ctypes.byref(n)) == INVALID
    assert lib.ltxattn_layer_norm_workspace(8, 64, 1, 9, ctypes.byref(n)) == INVALID


def masked_call(**kw):
    shape = dict(batch=2, q_len=16, kv_len=24, heads=4, kv_heads=2, head_dim=64)
    shape.update({k: kw.pop(k) for k in list(kw) if k in shape})
    nq, nk, h, hk, d = (shape[x] for x in ("q_len", "kv_len", "heads", "kv_heads", "head_dim"))
    sq, sk = (nq * h * d, h * d, d), (nk * hk * d, hk * d, d)
    a = dict(q=A, k=B, v=C, out=D, lse=E, q_stride=sq, k_stride=sk, v_stride=sk, out_stride=sq,
             scale=0.125, softcap=0.0, slopes=None, prefix=None, q_starts=None, kv_starts=None,
             docs=0, causal=0)
    a.update(shape)
    a.update(kw)
    return ltxattn._MaskedCall(**a), sq, sk


def masked(lib, **kw):
    ws = kw.pop("ws", F)
    return lib.ltxattn_masked_forward(ctypes.byref(masked_call(**kw)[0]), ws, 1 << 28, None)


MASKED = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(batch=0), INVALID), (dict(q_len=0), INVALID),
    (dict(kv_len=0), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("nan")), INVALID),
    (dict(softcap=1e-44), INVALID), (dict(softcap=3e38), INVALID), (dict(scale=3e38), INVALID),
    (dict(docs=-1), INVALID),
    (dict(docs=2), INVALID),                                   # no offsets
    (dict(q_starts=G, kv_starts=G + 256), INVALID),            # offsets of no document
    (dict(docs=2, q_starts=G), INVALID),
    (dict(prefix=G), INVALID),                                 # not causal
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(q_len=(1 << 24) + 1), UNSUPPORTED), (dict(heads=1026), UNSUPPORTED),
    (dict(batch=1025), UNSUPPORTED),
    (dict(docs=65536, q_starts=G, kv_starts=H), UNSUPPORTED),
    (dict(q=A + 8), MISALIGNED), (dict(out=D + 4), MISALIGNED), (dict(lse=E + 2), MISALIGNED),
    (dict(slopes=G + 1), MISALIGNED), (dict(k_stride=(3200 + 4, 128, 64)), MISALIGNED),
    (dict(k_stride=(0, 128, 64)), INVALID), (dict(v_stride=(3200, -128, 64)), INVALID),
]


@pytest.mark.parametrize("kw,status", MASKED, ids=str)
def test_masked_refusals(lib, kw, status):
    assert masked(lib, **kw) == status
    g = ltxattn._MaskedGrad(d_out=F, dq=G + (1 << 20), dk=G + (2 << 20), dv=G + (3 << 20))
    call, g.d_out_stride, g.dk_stride = masked_call(**dict(kw))
    g.dq_stride, g.dv_stride = g.d_out_stride, g.dk_stride
    assert lib.ltxattn_masked_backward(ctypes.byref(call), ctypes.byref(g), H, 1 << 28,
                                       None) == status


@pytest.mark.parametrize("kw", [dict(out=A), dict(out=B + 64), dict(out=C), dict(lse=A),
                                dict(lse=D), dict(slopes=D), dict(lse=G, slopes=G)], ids=str)
def test_masked_outputs_do_not_overlap(lib, kw):
    assert masked(lib, **kw) == INVALID


def test_masked_grad_refusals(lib):
    def back(call_kw=None, **kw):
        call, sq, sk = masked_call(**(call_kw or {}))
        a = dict(d_out=F, dq=G + (1 << 20), dk=G + (2 << 20), dv=G + (3 << 20), d_out_stride=sq,
                 dq_stride=sq, dk_stride=sk, dv_stride=sk)
        a.update(kw)
        return lib.ltxattn_masked_backward(ctypes.byref(call),
                                           ctypes.byref(ltxattn._MaskedGrad(**a)), H, 1 << 28, None)

    for n in ("d_out", "dq", "dk", "dv"):
        assert back(**{n: None}) == INVALID
        assert back(**{n: G + (5 << 20) + 8}) == MISALIGNED
        assert back(**{n + "_stride": (0, 0, 0)}) == INVALID
    assert back(dict(lse=None)) == INVALID
    for kw in (dict(dq=A), dict(dk=B), dict(dv=C), dict(dq=D), dict(dk=E), dict(dq=F),
               dict(dk=G + (1 << 20)), dict(dv=G + (2 << 20))):
        assert back(**kw) == INVALID
    assert reaches_cuda(lib, back())


def test_masked_accepts(lib):
    for kw in (dict(), dict(lse=None), dict(causal=1, prefix=G), dict(softcap=30.0, slopes=G),
               dict(docs=3, q_starts=G, kv_starts=G + 256, causal=1, prefix=H)):
        assert reaches_cuda(lib, masked(lib, **kw))
    n = ctypes.c_ulonglong(0)
    assert lib.ltxattn_masked_workspace(ctypes.byref(masked_call()[0]), 0, None) == INVALID
    assert reaches_cuda(lib, lib.ltxattn_masked_workspace(ctypes.byref(masked_call()[0]), 1,
                                                          ctypes.byref(n)))
