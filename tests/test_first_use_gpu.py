"""What a process pays for its first calls (needs a B200): ltxattn_create and the
allocation-free call load none of the masked attention's kernels, a first call works inside a
capture, and a context that was destroyed and made again works."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import torch
from joint_audio_video_flash_b200 import build, ltxattn
build.build()
q, k = (torch.randn(1, n, 4, 64, device="cuda").bfloat16() for n in (64, 2048))
out = torch.empty_like(q)
torch.cuda.synchronize()

def taken():  # MB of device memory, torch's own apart
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return (total - free - torch.cuda.memory_reserved()) / 2 ** 20

def masked_calls():  # of every kind that q and k select
    for dim in (64, 128):
        for n, keys in ((60, 60), (300, 300), (300, 2600)):
            x, y = (torch.randn(1, m, 2, dim, device="cuda").bfloat16() for m in (n, keys))
            for cap in (0.0, 20.0):
                for slopes in (None, torch.ones(2, device="cuda")):
                    o = dict(softcap=cap, slopes=slopes)
                    a, lse = ltxattn.masked_forward(x, y, y, **o)
                    ltxattn.masked_backward(a, x, y, y, a, lse, **o)
    ltxattn.check()
"""


def fresh(code):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    run = subprocess.run([sys.executable, "-c", HEAD + code], cwd=ROOT, capture_output=True,
                         text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    return run.stdout.split()


@pytest.mark.parametrize("first", [
    "ltxattn.create()",
    "ltxattn.forward_split_noalloc(q, k, k, out, kv_valid_len=2000, num_splits=2)"])
def test_masked_kernels_load_with_their_first_call(first):
    # kernels are loaded in steps of 2 MB; those of masked_calls take more than one
    before, after = map(float, fresh(f"""
ltxattn.load()
{first}
ltxattn.create()
a = taken()
masked_calls()
print(a, taken())
"""))
    assert after - before >= 2, (before, after)


@pytest.mark.parametrize("call", [
    "ltxattn.rope_axes(q, None, torch.zeros(1, 64, 1, device='cuda'), [1.0] * 32, (64,))[:1]",
    "(ltxattn.layer_norm(q),)",
    "ltxattn.layer_norm_backward(q, q, m, m, q[0, 0, 0].clone())",
    "ltxattn.masked_forward(q, k, k)",
    "ltxattn.masked_backward(q, q, q, q, q, m.transpose(1, 2).contiguous())"])
def test_a_first_call_inside_a_capture(call):
    assert fresh(f"""
ltxattn.create()
m = torch.ones(1, 64, 4, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = {call}
graph.replay()
torch.cuda.synchronize()
ltxattn.check()
print(all(torch.equal(a, b) for a, b in zip(got, {call})))
""") == ["True"]


def test_a_context_made_again():
    assert fresh("""
ltxattn.create()
a, _ = ltxattn.masked_forward(q, k, k)
torch.cuda.synchronize()
ltxattn.destroy()
try:
    ltxattn.masked_forward(q, k, k)
    print("no error")
except ltxattn.LtxAttnError as e:
    print(e.status == ltxattn.ERR_NOT_INITIALIZED)
ltxattn.create()
b, _ = ltxattn.masked_forward(q, k, k)
ltxattn.check()
print(torch.equal(a, b))
""") == ["True", "True"]
