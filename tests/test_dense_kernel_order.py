"""Orders that the kernels of the dense operators rely on, read from their source
on the CPU.

A block may touch another block's shared memory only once that block has
started, which a cluster barrier that every block has passed shows (being
launched together does not): in each kernel that reaches a peer's shared
memory, a cluster barrier is waited for before the first such access."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "activation_sparse_decode_gemv_b200", "csrc")
# what reaches a peer: remote sums, remote partial tiles, a peer's barriers
REMOTE = re.compile(r"\brow_sum<|\bld_cluster_f32x4\(|\bmbar_arrive_cluster\(|\btma_load_2d_pair\(|\bmma_commit_pair\(")
WAIT = re.compile(r"\bcluster_sync\(\)|\bpeer_started_wait<CL>\(\)")


def _kernels(name):
    """{kernel: its body without comments}"""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    found = {}
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\(", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if not depth:
                break
        found[m.group(1)] = text[at:end]
    return found


@pytest.mark.parametrize("name,kernels", [("pi_norm.cuh", {"norm_fwd_kernel", "norm_bwd_kernel"}),
                                          ("pi_gemm.cuh", {"pair_gemm_kernel", "split_gemm_kernel"})])
def test_peers_have_started_before_their_memory_is_touched(name, kernels):
    bodies = {k: b for k, b in _kernels(name).items() if REMOTE.search(b)}
    assert set(bodies) == kernels
    for k, body in bodies.items():
        wait = WAIT.search(body)
        assert wait and wait.start() < REMOTE.search(body).start(), f"{k}: no cluster barrier before the first remote access"


def test_the_wait_has_its_arrival():
    """Split barriers: the arrival comes first, once each, and outside of any loop over rows."""
    for k, body in _kernels("pi_norm.cuh").items():
        assert body.count("peer_started_wait<CL>()") == body.count("peer_started_arrive<CL>()") <= 1, k
        if "peer_started_wait<CL>()" in body:
            assert body.index("peer_started_arrive<CL>()") < body.index("peer_started_wait<CL>()") \
                < body.index("for (int t = t0; t < t1; ++t)"), k


@pytest.mark.parametrize("name", ["pi_norm.cuh", "pi_gemm.cuh"])
def test_no_non_coherent_loads(name):
    """These kernels start under the one before them, which may still be writing what they read after their wait
    (factors, scales).  A non-coherent load is for memory that nothing writes while the kernel lives."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert "__ldg(" not in text and "ld.global.nc" not in text and "ld_stream" not in text and "ld_keep" not in text
