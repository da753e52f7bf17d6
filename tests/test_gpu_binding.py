"""GPU tests of the Python binding's checks that need GPU tensors."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _z(*s, dt=BF16):
    return torch.zeros(*s, dtype=dt, device="cuda")


def test_codes_only_where_codes_belong():
    """Tensors of e4m3 codes are taken as codes of the 8-bit calls and nowhere
    else: not as a workspace, not as an operand."""
    say("binding, codes")
    e = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda").view(L.E4M3)
    x, w, d, u = _z(8, 32), _z(16, 32), _z(4, 32), _z(16, 4)
    wq, ws, wqt = L.fp8_quantize_weight(w, transposed=True)
    q, s = L.fp8_quantize_rows(x)
    calls = [lambda: L.linear(x, w, workspace=e), lambda: L.lora_linear(x, w, d, u, 1.0, workspace=e),
             lambda: L.lora_merge(w, d, u, 1.0, workspace=e), lambda: L.lora_linear_backward(x, w, d, u, 1.0, _z(8, 16), workspace=e),
             lambda: L.fp8_linear(q, s, wq, ws, workspace=e), lambda: L.fp8_lora_linear(x, wq, ws, d, u, 1.0, workspace=e),
             lambda: L.fp8_lora_linear_backward(x, wqt, ws, d, u, 1.0, _z(8, 16), workspace=e),
             lambda: L.orthogonalize(w, workspace=e)]
    for call in calls:
        with pytest.raises(TypeError, match="unsupported dtype"):
            call()
    for call in (lambda: L.linear(q, w), lambda: L.orthogonalize(q), lambda: L.fp8_quantize_rows(q)):
        with pytest.raises(TypeError):
            call()
    raw = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    assert torch.equal(L.fp8_linear(q, s, wq, ws, workspace=raw), _z(8, 16))
    with pytest.raises(ValueError, match="w_q has dtype"):
        L.fp8_linear(q, s, wq.view(torch.uint8), ws)
