"""Gradients and copies of AdamW with as many elements as their parameter but another shape are refused: element by
element, they are another matrix.  States may have any.  Without a GPU."""
import pytest
import torch

if torch.cuda.is_available():
    pytest.skip("host tensors: without a GPU only", allow_module_level=True)

from bit_gradient_compression_amd import loco  # noqa: E402

F8, U8, BF = torch.float8_e4m3fn, torch.uint8, torch.bfloat16


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    """Host tensors: what passes the checks is refused for its memory, and says so."""
    monkeypatch.setattr(loco, "_device", lambda: 0)


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("kw,match", [
    (dict(), "device memory"), (dict(grad=z(96)), "device memory"), (dict(grad=z(8, 1, 12)), "device memory"),
    (dict(param=z(96)), "device memory"), (dict(grad=z(12, 8)), "grad has the shape"), (dict(grad=z(4, 24)), "grad has the shape"),
    (dict(grad=z(2, 4, 12)), "grad has the shape"), (dict(copy=z(12, 8, dtype=BF)), "param_bf16 has the shape"),
    (dict(m=z(12, 8), v=z(2, 48)), "device memory"),
    (dict(m=(z(2, 48, dtype=F8), z(1, dtype=U8)), v=(z(96, dtype=U8), z(1, dtype=U8))), "device memory"),
])
def test_tensors(kw, match):
    a = dict(param=z(8, 12), grad=z(8, 12), m=z(8, 12), v=z(96), copy=z(8, 12, dtype=BF))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        loco.AdamwTensors([tuple(a.values())])

