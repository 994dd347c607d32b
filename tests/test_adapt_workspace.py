"""Workspaces of the adapters for many tokens: what a call has to keep (one
fp32 sum of each token and rank, its 16-bit parts and exponent, and in the
backward pass dT, the laid out factors and the gradients' partial sums), and
at most 256 MB beside it."""

import os

import pytest

from int8_quantized_matmul_amd import _native

MB = 2 ** 20


def _lib():
    if not os.path.exists(_native.LIB_PATH):
        from int8_quantized_matmul_amd.build import build
        build()
    return _native.load()


@pytest.mark.parametrize("r", [1, 16, 33, 64, 65, 128])
@pytest.mark.parametrize("s", [257, 4096, 16384, 65536, 262144, 2 ** 20, 2 ** 24])
def test_forward_workspace_is_a_few_sums_a_token(s, r):
    ranks = -(-r // 16) * 16
    need = 4 * s * r + 4 * s * ranks + 4 * s
    assert need <= _lib().i8mm_lora_forward_workspace_bytes(s, 36864, 12288, r) <= need + 256 * MB


@pytest.mark.parametrize("r", [1, 16, 33, 64, 65, 128])
@pytest.mark.parametrize("s", [257, 4096, 65536, 2 ** 20, 2 ** 24])
def test_backward_workspace_is_a_few_sums_a_token(s, r):
    h, o, G = 4096, 12288, 8
    ranks = -(-r // 16) * 16
    need = 8 * s * r + 4 * s * ranks + 4 * s + 2 * (s + 32 * 9) * ranks * 6 + 8 * s * ranks // 32
    # partial sums: chunks of 32768 tokens at most, 128 at least, twice as many as fit
    sums = (2 * s // min(32768, max(128, s // 8 // 128 * 128)) + 2) * 4 * r * (h + o)
    assert 8 * s * r <= _lib().i8mm_lora_backward_workspace_bytes(s, h, o, r, G) <= need + sums + 256 * MB
