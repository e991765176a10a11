"""The serving example: drafts checked by chunk attention agree with single-token decodes."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("scheme", ["int8_dither", "int8_rtn", "fp8_e4m3", "kivi2"])
def test_drafts_agree_with_decodes(scheme):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("draft_and_verify", os.path.join(ROOT, "examples", "draft_and_verify.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out, meters, diff = ex.serve(scheme, n_layers=2, prompts=(70, 5, 200), steps=3, draft=3, chunk=96)
    assert torch.isfinite(out.float()).all()
    # two layers of x + Wo o with |x| of a few units: the attention outputs differ by a few 2^-8 of |o| <= 5
    # (bf16 rounding of either, the chunk path's fp16 operands), and the sums round to bf16, 2^-8 of 8
    assert diff <= 4 * 2.0 ** -8 * 5 + 3 * 2.0 ** -8 * 8
    if meters is not None:
        assert meters.shape == (2, 3, 28) and ((meters >= 0) & (meters <= 1)).all()
