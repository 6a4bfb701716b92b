"""Refusals of the 8-bit operators' Python calls that need no GPU: tensors in host memory, and arguments that are no
tensors, are refused with ValueError and the argument's name before anything touches the runtime."""
import pytest
import torch

nf4 = pytest.importorskip("quantized_lora_fine_amd", reason="libnf4lora.so not built")

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16
X = torch.zeros(8, 272)
B = X.to(BF16)
A, S = torch.zeros(8, 272, dtype=torch.uint8).view(E4M3), torch.zeros(8, 3)
W, WS = torch.zeros(144, 272, dtype=torch.uint8).view(E4M3), torch.zeros(2, 3)
W3, WS3, OFF = torch.zeros(2, 144, 272, dtype=torch.uint8).view(E4M3), torch.zeros(2, 2, 3), torch.zeros(3, dtype=torch.int32)
w, rstd = torch.ones(272, dtype=BF16), torch.ones(8)

CALLS = [
    ("X", lambda: nf4.fp8_quantize(X)), ("X", lambda: nf4.fp8_quantize(B, 128)), ("X", lambda: nf4.fp8_quantize(None)),
    ("codes", lambda: nf4.fp8_dequantize(A, S)), ("codes", lambda: nf4.fp8_dequantize(None, S)),
    ("W", lambda: nf4.fp8_matmul(A, S, W, WS)), ("W", lambda: nf4.fp8_matmul(A, S, W, WS, True)),
    ("W", lambda: nf4.fp8_matmul(None, None, None, None)),
    ("W", lambda: nf4.fp8_matmul_grouped(A, S, W3, WS3, OFF)), ("W", lambda: nf4.fp8_matmul_grouped(A, S, W, WS, OFF)),
    ("X", lambda: nf4.rmsnorm_fwd(B, w)), ("X", lambda: nf4.rmsnorm_fwd(None, w)),
    ("dY", lambda: nf4.rmsnorm_bwd(B, B, w, rstd)), ("dY", lambda: nf4.rmsnorm_bwd(None, B, w, rstd)),
]


@pytest.mark.parametrize("i", range(len(CALLS)))
def test_refused_without_a_gpu(i):
    name, call = CALLS[i]
    with pytest.raises(ValueError, match=f"^{name}: "):
        call()
