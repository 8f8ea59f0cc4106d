"""What the binding of the dense block operators refuses because the C ABI
cannot see it: numbers beyond a C int (ctypes would take them modulo 2^32), on
the CPU."""
import os

import pytest
import torch

from activation_sparse_decode_gemv_b200 import binding as pb


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.environ.get("PI_FFN_LIB"):  # another build given: use it as is
        from activation_sparse_decode_gemv_b200 import build
        build.build()
    return pb.lib()


BIG = 2 ** 32 + 5  # 5 modulo 2^32


def test_numbers_beyond_a_c_int():
    w = torch.zeros(128, 64, dtype=torch.float16)
    layer = pb.GatedFfnLayer(w, w, w)
    gate = torch.zeros(8, 64)
    with pytest.raises(ValueError, match="tokens_per_gate"):
        pb.BlockNorm(64, gate=gate, tokens_per_gate=BIG)
    norm = pb.BlockNorm(64, gate=gate, tokens_per_gate=2 ** 31 - 1)  # the largest: one row for all tokens
    assert norm.desc.tokens_per_gate == 2 ** 31 - 1
    for n in (BIG, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="max_tokens"):
            pb.pi_gated_ffn_workspace_size(layer, n)
        with pytest.raises(ValueError, match="max_tokens"):
            pb.pi_block_norm_workspace_size(norm, n)
        for at in range(3):
            a = [4, 96, 64]
            a[at] = n
            with pytest.raises(ValueError, match=("tokens", "n", "k")[at]):
                pb.pi_matmul_i8_workspace_size(*a)


def test_tensors_of_more_rows_than_a_c_int():
    """On the meta device: nothing is allocated, and the row count is refused before the device is looked at."""
    e = lambda *s, dt: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    norm = pb.BlockNorm(8, y_dtype=torch.float16, u_dtype=torch.float16)
    x, q, s = e(BIG, 8, dt=torch.float32), e(BIG, 16, dt=torch.int8), e(BIG, dt=torch.float32)
    wide = e(BIG, 16, dt=torch.float32)
    w = torch.zeros(8, 8, dtype=torch.float16)
    layer, h, ws = pb.GatedFfnLayer(w, w, w), e(BIG, 8, dt=torch.float16), torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: pb.pi_block_norm_forward(norm, x, None, x, None),
                 lambda: pb.pi_block_norm_backward(norm, x, None, None, s, None, x, x, None, ws),
                 lambda: pb.pi_gated_ffn_forward(layer, h, h, ws),
                 lambda: pb.pi_gated_ffn_backward(layer, h, h, h, h, ws),
                 lambda: pb.pi_quantize_i8(wide, q, s),
                 lambda: pb.pi_matmul_i8(q, s, e(8, 16, dt=torch.int8), e(8, dt=torch.float32), x, ws),
                 lambda: pb.pi_matmul_i8(e(1, 16, dt=torch.int8), e(1, dt=torch.float32), q, s,
                                         e(1, BIG, dt=torch.float32), ws)):
        with pytest.raises(ValueError, match="over 2147483647"):
            call()


def test_weights_and_parameters_whose_memory_moved():
    """A layer and a norm hold addresses.  A tensor given other memory since (w.data = ..., set_) would be read where
    it was: freed memory.  New values in the same memory are fine."""
    h = torch.float16
    u, ws = torch.zeros(4, 64, dtype=h), torch.zeros(65536, dtype=torch.uint8)
    g, f, s = torch.zeros(4, 128, dtype=h), torch.zeros(4, 64), torch.zeros(4)
    for at, name in enumerate(("w_gate", "w_up", "w_down_t")):
        w = [torch.zeros(128, 64, dtype=h) for _ in range(3)]
        layer = pb.GatedFfnLayer(*w)
        w[at].add_(1)
        with pytest.raises(ValueError, match="must be a CUDA tensor"):  # nothing else is wrong
            pb.pi_gated_ffn_forward(layer, u, u.clone(), ws)
        w[at].data = w[at].data.clone()
        with pytest.raises(ValueError, match=f"{name}: .*moved"):
            pb.pi_gated_ffn_forward(layer, u, u.clone(), ws)
        with pytest.raises(ValueError, match=f"{name}: .*moved"):
            pb.pi_gated_ffn_backward(layer, u, g, g, u, ws)
    for name in ("w_post", "w_pre", "gate"):
        p = {"w_post": torch.ones(64), "w_pre": torch.ones(64), "gate": torch.ones(4, 64)}
        norm = pb.BlockNorm(64, post_norm=True, **p, tokens_per_gate=1)
        p[name].add_(1)
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            pb.pi_block_norm_forward(norm, f, u, f, u.clone())
        p[name].data = p[name].data.clone()
        with pytest.raises(ValueError, match=f"{name}: .*moved"):
            pb.pi_block_norm_forward(norm, f, u, f, u.clone())
        with pytest.raises(ValueError, match=f"{name}: .*moved"):
            pb.pi_block_norm_backward(norm, f, u, s, s, u.clone(), None, f.clone(), u.clone(), ws)
