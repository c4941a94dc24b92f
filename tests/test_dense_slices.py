"""Slices that do not start on 16 bytes, without a GPU: the binding gives the library copies that do, alive while the call is made, and
leaves all others where they are."""
import ctypes

import pytest
import torch

from test_attn_binding import on
from test_dense_binding import calls  # noqa: F401
from weight_only_int4_route_gb300 import dense

F32, I32 = torch.float32, torch.int32
VECTORS = {"moe_rmsnorm": [4], "moe_linear_w8a8": [2, 5, 6], "moe_token_logprobs": [6]}     # their places among the arguments
TYPES = {"moe_rmsnorm": ctypes.c_float, "moe_linear_w8a8": ctypes.c_float, "moe_token_logprobs": ctypes.c_int32}


@pytest.mark.parametrize("first", range(9))
def test_slices_are_copied_where_they_must_be(calls, monkeypatch, first):  # noqa: F811
    seen = {}

    class Library:
        def __getattr__(self, name):
            def call(*a):
                if name in VECTORS:      # what lies there during the call
                    seen[name] = [(a[i], list((TYPES[name] * 4).from_address(a[i]))) for i in VECTORS[name]]
                return 0
            return call

    monkeypatch.setattr(dense, "lib", Library)
    n = 4
    f32 = [on(torch.arange(16.0) + 100 * i)[first:first + n] for i in range(4)]
    ids = on(torch.arange(16, dtype=I32))[first:first + n]
    dense.rmsnorm(on(torch.zeros(n, n)), f32[0])
    dense.linear_w8a8(on(torch.zeros((n, 16), dtype=torch.int8)), f32[1], on(torch.zeros((n, 16), dtype=torch.int8)), f32[2], f32[3])
    dense.token_logprobs(on(torch.zeros(n, 40)), ids, k=1)
    given = {"moe_rmsnorm": [f32[0]], "moe_linear_w8a8": f32[1:], "moe_token_logprobs": [ids]}
    assert sorted(seen) == sorted(given)
    for name, tensors in given.items():
        for (address, values), t in zip(seen[name], tensors):
            assert address % 16 == 0 and values == t.tolist()
            assert (address == t.data_ptr()) == (t.data_ptr() % 16 == 0)
