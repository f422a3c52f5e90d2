"""CPU checks of the 8-bit serving operators' binding and example: what they refuse, what they size.  Nothing here
launches a kernel."""
import importlib.util
import os

import pytest
import torch

import block_quantized_weight_affine_amd as qg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("codes", [torch.uint8, torch.bool, torch.float8_e4m3fn, torch.float8_e5m2, torch.int16])
def test_w8a8_takes_int8_codes_only(codes):
    w, ws, x, y = torch.zeros(16, 32, dtype=codes), torch.ones(16), torch.zeros(1, 32), torch.zeros(1, 16)
    with pytest.raises(qg.QGError) as e:
        qg.qgemm_w8a8(w, ws, x, y, 16, 32, 1, stream=0)
    assert e.value.status == qg.QG_EINVAL


@pytest.mark.parametrize("scales", [torch.int32, torch.float64, torch.float16, torch.bfloat16])
def test_w8a8_takes_f32_scales_only(scales):
    w, ws, x, y = torch.zeros(16, 32, dtype=torch.int8), torch.ones(32).to(scales), torch.zeros(1, 32), torch.zeros(1, 16)
    with pytest.raises(qg.QGError) as e:
        qg.qgemm_w8a8(w, ws, x, y, 16, 32, 1, stream=0)
    assert e.value.status == qg.QG_EINVAL
