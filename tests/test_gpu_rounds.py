"""Layer norm's and the adapters' gradients where a block goes through several
rounds of rows, and in every variant that the width chooses: carried column
sums, the next row's loads, both halves of the rows' sums; several rounds of
four tiles, and chunks with partial sums. Bounds: test_gpu_layer_norm.py's and
test_gpu_lora.py's.
"""

import pytest
import torch

import int8_quantized_matmul_amd as i8
from gpu_util import say
from test_gpu_layer_norm import TYPES, _check_backward as _check_norm_backward, _check_forward as _check_norm, _inputs
from test_gpu_lora import BF16, F16, _case, _check_backward, _check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("s,h", [(1100, 768), (2049, 100), (700, 5120), (530, 12296), (3, 12289), (300, 12289),
                                 (3, 14000), (300, 14000), (3, 16384), (600, 16384), (300, 16400)])
def test_norm_gradients_over_rounds(s, h, xt, wt):
    say(f"  launch: layer_norm s={s} h={h} {xt} {wt}")
    X, w, b, dY = _inputs(s, h, xt, wt, s + h)
    Y, mean, rstd = i8.layer_norm(X, w, b, 1e-5)
    dX, dw, db = i8.layer_norm_backward(dY, X, w, mean, rstd)
    dX1, _, _ = i8.layer_norm_backward(dY, X, w, mean, rstd, param_grads=False)
    torch.cuda.synchronize()
    _check_norm(X, w, b, 1e-5, Y, mean, rstd)
    _check_norm_backward(dY, X, w, mean, rstd, dX, dw, db)
    _check_norm_backward(dY, X, w, mean, rstd, dX1, None, None)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,h,o,r,G,kind", [(512, 256, 320, 64, 1, "one"), (500, 320, 256, 40, 1, "one"),
                                            (512, 320, 192, 16, 1, "one"), (450, 64, 256, 100, 1, "one"),
                                            (1500, 4160, 12352, 64, 2, "runs"), (1300, 8256, 8192, 24, 2, "mixed"),
                                            (1100, 8192, 8256, 90, 1, "one")])
def test_adapter_gradients_over_rounds(s, h, o, r, G, kind, dtype):
    say(f"  launch: lora s={s} h={h} o={o} r={r} G={G} {kind} {dtype}")
    c = _case(s, h, o, r, G, kind, dtype)
    Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"], base=c["base"])
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], base=c["gbase"])
    torch.cuda.synchronize()
    _check_forward(c, Y, T, c["base"])
    _check_backward(c, T, dX, dA, dB, c["gbase"])
