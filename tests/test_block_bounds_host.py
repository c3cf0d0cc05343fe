"""Sizes whose index arithmetic would leave 32 bits, and operands of a later launch, are refused before any launch (no
GPU needed)."""
import struct

import pytest


@pytest.fixture(scope="module")
def B():
    from mixed_precision_decode_b200 import build
    build.build()
    from mixed_precision_decode_b200 import bitsmoe
    return bitsmoe


@pytest.mark.parametrize("T, K", [(2 ** 27 - 1, 16), (2 ** 30 + 1, 1), (2 ** 31 - 1, 1), (2 ** 26, 31), (2 ** 28 + 1, 4)])
def test_routing_of_more_than_2_30_pairs(B, T, K):
    """A pair's index plus a CTA's 1024 threads, and a token's plus the 8192 x 32 whose bits are kept, stay below 2^31."""
    args = struct.pack("@7PQq6ifi", 256, 512, 1024, 2048, 4096, 256, 0, 1 << 40, 64, T, 64, K, 0, 0, 1, 1.0, 0)
    assert B.lib().bitsmoe_topk_route(args, None) == B.EINVAL
    assert B.topk_route_workspace_bytes(T, 64, K) == 0
    assert B.topk_route_workspace_bytes(2 ** 30 // K, 64, K) > 0


@pytest.mark.parametrize("T, K", [(2 ** 27 - 1, 16), (2 ** 30 + 1, 1)])
def test_dense_ffn_of_more_than_2_30_pairs(B, T, K):
    d = B.ffn_dims(64, 32, 4, K)
    assert B.dense_ffn_workspace_bytes(d, T) == 0 and B.dense_ffn_workspace_bytes(d, 2 ** 30 // K) > 0
    args = struct.pack("@6i11PQq", 64, 32, 4, K, T, 1, *[256] * 10, 0, 1 << 60, 64)
    assert B.lib().bitsmoe_dense_ffn_forward(args, None) == B.EINVAL


@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 1])
def test_grouped_product_of_more_than_2_30_rows(B, n):
    args = struct.pack("@7Pq10i", 256, 512, 0, 1024, 2048, 4096, 0, 16, n, n, 8, 16, 2, 1, 1, 1, 0, 0)
    assert B.lib().bitsmoe_grouped_matmul(args, None) == B.EINVAL


@pytest.mark.parametrize("bad", [dict(wd=264), dict(d_model=1 << 20, E=4096)])
def test_dense_ffn_refuses_the_down_product_before_the_first_launch(B, bad):
    """A misaligned W_down, or more rows of it than a tensor map counts, is refused as such: not after the gate and up
    products were launched (which here, without a GPU, would answer with a CUDA error)."""
    ok = dict(d_model=64, d_ff=32, E=4, K=2, tokens=3, type=1, x=256, wg=256, wu=256, wd=256, ids=256, gw=256, off=256,
              od=256, out=256, ws=512, st=0, nb=1 << 60, xs=1 << 20)
    assert B.lib().bitsmoe_dense_ffn_forward(struct.pack("@6i11PQq", *{**ok, **bad}.values()), None) == B.EINVAL


@pytest.mark.parametrize("d", [2 ** 30 + 1, 2 ** 31 - 1])
def test_norm_of_more_than_2_30_columns(B, d):
    args = struct.pack("@7P5q6i2f", 256, 512, 0, 0, 256, 1024, 2048, d, d, 0, d, d, 1, d, 0, 0, 1, 0, 1.0, 1e-6)
    assert B.lib().bitsmoe_norm_residual(args, None) == B.EINVAL


@pytest.mark.parametrize("k", [2 ** 30 + 8, 2 ** 31 - 8])
def test_grouped_product_over_more_than_2_30_columns(B, k):
    args = struct.pack("@7Pq10i", 256, 512, 0, 1024, 0, 2048, 0, k, 4, 4, 8, k, 2, 1, 1, 1, 0, 0)
    assert B.lib().bitsmoe_grouped_matmul(args, None) == B.EINVAL
