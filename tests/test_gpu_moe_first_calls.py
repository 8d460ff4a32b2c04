"""What the first calls in a process prepare (GPU; each case in a process of its own)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import time
import torch
import q6_int8_mmq_gb300 as q6
q6.load()
x = torch.randn(2, 512, device="cuda")
raw = torch.zeros(2 * 8 * 2 * 144, device="cuda", dtype=torch.uint8)
ids = torch.zeros(2, device="cuda", dtype=torch.int32)
A, B = torch.ones(2, 8, 512, device="cuda").half(), torch.ones(2, 16, 8, device="cuda").half()
ad = q6.LoraAdapters(A, B, torch.ones(2, device="cuda"))
Y = torch.zeros(2, 16, device="cuda")

def timed(call):
    torch.cuda.synchronize()
    t = time.perf_counter()
    result = call()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) * 1e3, result
"""


def run(code):
    # kernels are loaded when they are first named, as by default
    env = dict(os.environ, CUDA_MODULE_LOADING="LAZY")
    r = subprocess.run([sys.executable, "-c", SETUP + code], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_the_shared_projections_do_not_pay_for_the_experts():
    """The first call raises the kernels' limits of shared memory, which loads them (measured: 2.1 ms
    for the shared projections, 1.7 ms for the experts and adapters). Those of the experts and of the
    adapters are loaded by the first call that runs them, so together the two cost more than a
    quarter of the first call of all; had that call loaded them they would cost about a twentieth."""
    out = run("""
first, _ = timed(lambda: q6.quantize_act(x))
w = q6.pack_experts(raw, "q4_K", 2, 8, 512)
g = q6.group_rows(ids, 2)
experts, _ = timed(lambda: q6.experts_mmq(w, x.half(), g))
adapters, _ = timed(lambda: q6.lora_add(ad, x, g, Y))
print(first, experts + adapters)
""")
    first, own = map(float, out.split()[-2:])
    assert own > 0.25 * first, out


def test_first_calls_may_be_captured():
    """A graph may hold the first product and the first adapter of a process that has made another
    call before."""
    run("""
q6.quantize_act(x)
w = q6.pack_experts(raw, "q4_K", 2, 8, 512)
h = torch.ones(2, 512, device="cuda").half()
g = q6.group_rows(ids, 2)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out, _ = q6.experts_mmq(w, h, g)
    y = q6.lora_add(ad, h, g, Y, out=torch.empty_like(Y))
graph.replay()
torch.cuda.synchronize()
assert not out.any() and (y == 512 * 8).all(), y
""")
