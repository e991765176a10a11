"""Outputs given to the beam selection and to paths are checked like the other arguments (CPU only: tensors that say
they are on a device, refused before anything looks at their memory)."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc


class There(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


@pytest.fixture(autouse=True)
def _device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def there(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(There)


@pytest.mark.parametrize("at, bad, text", [
    (0, [[0.0] * 4] * 2, "out scores"), (1, None, "rows"), (2, there(2, 4, dtype=torch.int64), "tokens"),
    (3, there(2, 3, dtype=torch.bool), "out finished"), (3, "no", "out finished"), (1, torch.zeros(2, 4, dtype=torch.int32), "rows")])
def test_one_of_them(at, bad, text):
    x, s = there(2, 4, 10, dtype=torch.float32), there(2, 4, dtype=torch.float32)
    out = [there(2, 4, dtype=t) for t in (torch.float32, torch.int32, torch.int32, torch.bool)]
    out[at] = bad
    with pytest.raises(ValueError, match=text):
        wc.witcert_beam_select(x, s, out=tuple(out))


@pytest.mark.parametrize("out", [7, (), there(4, 2, 4, dtype=torch.int32), "four"])
def test_all_of_them(out):
    x, s = there(2, 4, 10, dtype=torch.float32), there(2, 4, dtype=torch.float32)
    with pytest.raises(ValueError, match="four tensors"):
        wc.witcert_beam_select(x, s, out=out)


@pytest.mark.parametrize("out", [[1], 7, there(2, 4, 4, dtype=torch.int32), there(2, 4, 5, dtype=torch.int64),
                                 torch.zeros(2, 4, 5, dtype=torch.int32)])
def test_paths(out):
    r = there(5, 2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="out"):
        wc.witcert_beam_paths(r, r, out=out)
