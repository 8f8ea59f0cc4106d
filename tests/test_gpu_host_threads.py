"""Calls from host threads: a thread that has made no CUDA call of its own yet
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
