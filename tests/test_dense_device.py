"""Layer norm, the gated feed-forward block and the 4-bit calls run on their
tensors' device, also where another one is current (the library and the device
calls are stand-ins, so this needs no GPU)."""

import pytest
import torch

from gaussian_splatting_differentiable_ewa_amd import _lib as L
from test_tokens_device import Stand, machine  # noqa: F401  (a fixture)

BF16, U8 = torch.bfloat16, torch.uint8


def calls(device, stream):
    def t(*shape, dtype=torch.float32):
        return Stand(*shape, dtype=dtype, device=device)

    x, w, ws = t(9, 64, dtype=BF16), t(64), t(1000)
    up, down, kept = t(128, 64, dtype=BF16), t(64, 128, dtype=BF16), t(5760, dtype=U8)
    h = t(9, 128, dtype=BF16)
    codes, scales = t(40, 32, dtype=U8), t(40, 4, dtype=U8)
    L.gs_layer_norm_fwd(x, w, w, x, t(2, 9), stream=stream)
    L.gs_layer_norm_bwd(x, x, w, t(2, 9), x, w, w, ws, stream=stream)
    L.gs_gated_ff_fwd(x, up, up, down, L.GS_SILU, h, kept, x, ws, stream=stream)
    L.gs_gated_ff_bwd(x, x, up, up, down, h, kept, L.GS_SILU, x, up, up, down, ws, stream=stream)
    L.gs_quantise_fp4(x, codes, scales, stream=stream)
    L.gs_dequantise_fp4(codes, scales, t(40, 64), stream=stream)
    L.gs_linear_fp4(x, codes, scales, t(9, 40, dtype=BF16), ws, stream=stream)


@pytest.mark.parametrize("device", [0, 1])
def test_launches_are_on_the_tensors_device(machine, device):  # noqa: F811
    log, _ = machine
    calls(device, None)
    assert len(log) == 7
    assert all(at == device and stream == 1000 + device for _, at, stream in log), log
    assert torch.cuda.current_device() == 0


def test_a_given_stream_is_used_there(machine):  # noqa: F811
    log, stream = machine
    calls(1, stream)
    assert len(log) == 7 and all(at == 1 and s == 77 for _, at, s in log), log
