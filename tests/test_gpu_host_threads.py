"""Calls from host threads.  A thread that has made no CUDA call of its own yet
(an autograd worker, a server's handler) has no current context, and the calls
have to work there all the same."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FRESH = """
import threading, torch
from activation_sparse_decode_gemv_b200 import binding as pb
from activation_sparse_decode_gemv_b200 import inputs
T, d, f = %d, 264, 1032
g = torch.Generator(device="cuda").manual_seed(0)
n = lambda *s: torch.randn(*s, generator=g, device="cuda")
w = [(n(f, d) * 0.05).half() for _ in range(3)]
u, dy, x = n(T, d).half(), n(T, d).half(), n(T, 272)
wq = torch.randint(-128, 128, (96, 272), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
one = torch.ones(96, device="cuda")
lt = inputs.make_layer(inputs.CONFIGS["opt7b_f16"].scaled(d=512, f=2048, r=128), 0, seed=1).to(torch.device("cuda"))
us = n(16, 512).half()
ws_bytes = 1 << 24
def buffers():
    h = torch.half
    return {"y": torch.empty(T, d, dtype=h, device="cuda"), "gate": torch.empty(T, f, dtype=h, device="cuda"),
            "up": torch.empty(T, f, dtype=h, device="cuda"), "du": torch.empty(T, d, dtype=h, device="cuda"),
            "dw": [torch.empty(f, d, dtype=h, device="cuda") for _ in range(3)],
            "q": torch.empty(T, 272, dtype=torch.int8, device="cuda"), "s": torch.empty(T, device="cuda"),
            "z": torch.empty(T, 96, device="cuda"), "ys": torch.empty(16, 512, device="cuda"),
            "ws": [torch.zeros(ws_bytes, dtype=torch.uint8, device="cuda") for _ in range(3)]}
def run(b):
    dense, sparse = pb.GatedFfnLayer(*w), pb.FfnLayer.from_tensors(lt)
    pb.pi_gated_ffn_forward(dense, u, b["y"], b["ws"][0], gate=b["gate"], up=b["up"])
    pb.pi_gated_ffn_backward(dense, u, b["gate"], b["up"], dy, b["ws"][0], b["du"], *b["dw"])
    pb.pi_quantize_i8(x, b["q"], b["s"])
    pb.pi_matmul_i8(b["q"], b["s"], wq, one, b["z"], b["ws"][1])
    pb.pi_decode_ffn(sparse, us, b["ys"], b["ws"][2])
here, there, errors = buffers(), buffers(), []
torch.cuda.synchronize()
pb.lib()
def thread():
    try:
        run(there)
    except Exception as e:
        errors.append(e)
t = threading.Thread(target=thread)
t.start(), t.join()
assert not errors, errors
run(here)
torch.cuda.synchronize()
for k in ("y", "gate", "up", "du", "z", "ys"):
    assert torch.equal(here[k], there[k]), k
assert all(torch.equal(p, q) for p, q in zip(here["dw"], there["dw"]))
assert all(pb.pi_get_device_status(s) == 0 for s in here["ws"] + there["ws"])
print("threads agree")
"""


def _child(code):
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "threads agree" in out.stdout, out.stderr[-2000:]


@pytest.mark.parametrize("T", [2, 300])
def test_layers_made_and_called_in_a_thread_without_a_context(cuda_device, T):
    _child(FRESH % T)


MANY = """
import threading, torch
from activation_sparse_decode_gemv_b200 import binding as pb
N, d, f, k = 12, 264, 1032, 272
g = torch.Generator(device="cuda").manual_seed(0)
n = lambda *s: torch.randn(*s, generator=g, device="cuda")
pb.lib()
jobs = []
for i in range(N):
    T = (1, 3, 40, 200)[i % 4]
    w = [(n(f, d) * 0.05).half() for _ in range(3)]
    layer = pb.GatedFfnLayer(*w)
    j = {"layer": layer, "ws": pb.make_gated_ffn_workspace(layer, T, True), "u": n(T, d).half(), "dy": n(T, d).half(),
         "x": n(T, k), "q": torch.empty(T, k, dtype=torch.int8, device="cuda"), "s": torch.empty(T, device="cuda"),
         "wq": torch.randint(-128, 128, (96, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8),
         "one": torch.ones(96, device="cuda"), "iws": pb.make_matmul_i8_workspace(T, 96, k)}
    j["out"] = [torch.empty(T, m, dtype=torch.half, device="cuda") for m in (d, f, f, d)] + \\
        [torch.empty(f, d, dtype=torch.half, device="cuda") for _ in range(3)] + [torch.empty(T, 96, device="cuda")]
    jobs.append(j)
torch.cuda.synchronize()
def run(j):
    y, gate, up, du, *dw, z = j["out"]
    pb.pi_gated_ffn_forward(j["layer"], j["u"], y, j["ws"], gate=gate, up=up)
    pb.pi_gated_ffn_backward(j["layer"], j["u"], gate, up, j["dy"], j["ws"], du, *dw)
    pb.pi_quantize_i8(j["x"], j["q"], j["s"])
    pb.pi_matmul_i8(j["q"], j["s"], j["wq"], j["one"], z, j["iws"])
start, errors = threading.Barrier(N), []
def thread(j):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for _ in range(3):
                run(j)
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        errors.append(e)
ts = [threading.Thread(target=thread, args=(j,)) for j in jobs]
[t.start() for t in ts], [t.join() for t in ts]
assert not errors, errors
for j in jobs:
    got = [t.clone() for t in j["out"]]
    for t in j["out"]:
        t.zero_()
    run(j)
    assert all(torch.equal(a, b) for a, b in zip(got, j["out"]))
    assert pb.pi_get_device_status(j["ws"]) == 0 and pb.pi_get_device_status(j["iws"]) == 0
print("threads agree")
"""


def test_first_calls_of_many_threads_at_once(cuda_device):
    """Each on a stream of its own: what a first call sets up for the device is set up once and read by the
    others, and every thread's results are those of a call alone."""
    _child(MANY)
