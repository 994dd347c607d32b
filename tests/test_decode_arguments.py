"""Arguments that the Python calls of decoding refuse before they look at a device (CPU)."""

import pytest
import torch

import int8_quantized_matmul_amd as i8


def test_a_history_to_write_without_one_to_read_is_refused():
    with pytest.raises(ValueError, match="history"):
        i8.beam_select(torch.zeros((2, 9)), torch.zeros((1, 2)), 2, history_out=torch.zeros((2, 1), dtype=torch.int32))
