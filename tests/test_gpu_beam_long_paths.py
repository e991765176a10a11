"""Paths of as many steps as an int counts."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 9])
def test_steps_up_to_the_largest(T):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    rows = torch.zeros(T, 1, 1, dtype=torch.int32, device="cuda")
    tokens = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1, 1)
    out = torch.empty(1, 1, T, dtype=torch.int32, device="cuda")
    wc.witcert_beam_paths(rows, tokens, out=out)
    assert torch.equal(out.view(-1), tokens.view(-1))
    wc.witcert_beam_paths(rows, tokens, length=torch.tensor([3], dtype=torch.int32, device="cuda"), pad=-7, out=out)
    assert out[0, 0, :3].tolist() == [0, 1, 2] and int(out[0, 0, 3:].max()) == -7 == int(out[0, 0, 3:].min())
