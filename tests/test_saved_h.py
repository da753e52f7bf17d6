"""Where the binding finds the h that a forward left, on the CPU: at the byte
the layout names, whatever the workspace tensor's dtype."""
import pytest
import torch

import lora_bypass_linear_amd as L

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("ws_dtype", [torch.uint8, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("adt", [BF16, F32])
@pytest.mark.parametrize("fp8", [True, False])
def test_saved_h_in_any_workspace(ws_dtype, adt, fp8):
    M, N, K, r = 48, 64, 128, 20
    x, d, u = torch.zeros(M, K, dtype=BF16), torch.zeros(r, K, dtype=adt), torch.zeros(N, r, dtype=adt)
    w = torch.zeros(N, K, dtype=BF16)
    n = L.fp8_lora_workspace_size(M, N, K, r, *(L.dtype_code(x), 0, L.dtype_code(d), L.dtype_code(u))) if fp8 else \
        L.lora_workspace_size(M, N, K, r, L.dtype_code(x), L.dtype_code(w), 0, L.dtype_code(d), L.dtype_code(u))
    raw = torch.randint(0, 256, (-(-n // 8) * 8,), dtype=torch.uint8)
    get = (lambda ws: L.fp8_lora_saved_h(ws, x, d, u)) if fp8 else (lambda ws: L.lora_saved_h(ws, x, w, d, u))
    want, got = get(raw), get(raw.view(ws_dtype))
    assert got.dtype == want.dtype and got.shape == want.shape == (M, 32)
    assert got.data_ptr() == want.data_ptr()
    shaped = get(raw.view(ws_dtype).view(2, -1))
    assert shaped.data_ptr() == want.data_ptr()
