"""GPU tests of the state space layer calls at their edges: batches without sequences,
states in place, calls close behind one another.  Bounds as in test_ssm_gpu.py."""
import pytest
import torch

import linear_attention_sequence_gb300 as kda
from linear_attention_sequence_gb300 import _ssm
from test_ssm_gpu import BF16, DEV, F32, conv_inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows, but no sequence

@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("first", [0, 7, 200, -3])
def test_conv_of_rows_without_sequences(first, dtype, packed):
    """A padded buffer whose batch is empty: no row is written, and the parameters'
    gradients are 0."""
    T, D, W = 200, 40, 4
    x = conv_inputs(T, D, W, 0, dtype, 501)
    cu = torch.tensor([first], dtype=torch.int32, device=DEV)
    out = torch.full((T, D), 7.0, device=DEV, dtype=dtype)
    _, last = kda.kda_ssm_conv(x["x"], x["weight"], x["bias"], cu, x["state"], out=out)
    assert last.shape == (0, W - 1, D) and bool((out == 7).all())
    xi, sc = kda.kda_act_pack8(x["x"]) if packed else (x["x"], None)
    g = kda.kda_ssm_conv_backward(xi, x["weight"], x["d_out"], x["bias"], cu, x["state"], x_scales=sc,
                                  d_conv_state_out=x["d_state"])
    assert not g["dweight"].any() and not g["dbias"].any() and g["d_conv_state"].shape == (0, W - 1, D)
    # the C call, for the rows of dx
    dx, dw = torch.full((T, D), 7.0, device=DEV, dtype=dtype), torch.full((D, W), 7.0, device=DEV)
    rows = lambda t: _ssm._ROWS.pack(t.data_ptr(), t.stride(0), 0)  # noqa: E731
    dims = _ssm._DIMS.pack(0, T, D, W, *[_ssm._code(dtype, "x")] * 2)
    _ssm._run("kda_ssm_conv_backward", torch.cuda.current_device(), dims, rows(x["x"]), x["weight"].data_ptr(), 0, 0,
              cu.data_ptr(), 1, rows(x["d_out"]), 0, dx.data_ptr(), dw.data_ptr(), 0, 0, 0, 0)
    assert bool((dx == 7).all()) and not dw.any()
    assert kda.kda_get_last_device_error() == 0
