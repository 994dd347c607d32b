"""The adapters for so many tokens that a tile's later adapters have fewer
parts, and then none of their own: test_gpu_lora.py's bounds."""

import pytest
import torch

import int8_quantized_matmul_amd as i8
from gpu_util import say
from test_gpu_lora import BF16, F16, _case, _check_backward, _check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,h,o,r,G,kind", [(66000, 576, 64, 40, 3, "mixed"), (140000, 64, 576, 70, 50, "runs"),
                                            (270000, 64, 128, 66, 2, "mixed")])
def test_forward_and_backward(s, h, o, r, G, kind, dtype):
    say(f"  launch: lora s={s} h={h} o={o} r={r} G={G} {kind} {dtype}")
    c = _case(s, h, o, r, G, kind, dtype)
    Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"], base=c["base"])
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], base=c["gbase"])
    torch.cuda.synchronize()
    _check_forward(c, Y, T, c["base"])
    _check_backward(c, T, dX, dA, dB, c["gbase"])
