"""Refusals of the Python calls around a shared projection that need no GPU: tensors in host memory, and arguments that
are no tensors, are refused with ValueError and the argument's name before anything touches the runtime."""
import pytest
import torch

nf4 = pytest.importorskip("quantized_lora_fine_amd", reason="libnf4lora.so not built")

BF16 = torch.bfloat16
X, w, stat = torch.zeros(8, 272, dtype=BF16), torch.ones(272, dtype=BF16), torch.ones(8)
L1, L2, s = torch.zeros(2, 272, 16, dtype=BF16), torch.zeros(2, 16, 144, dtype=BF16), torch.ones(2)
T, dY, OFF = torch.zeros(8, 16), torch.zeros(8, 144, dtype=BF16), torch.zeros(3, dtype=torch.int32)

CALLS = [
    ("X", lambda: nf4.layernorm_fwd(X, w)), ("X", lambda: nf4.layernorm_fwd(None, w)),
    ("X", lambda: nf4.layernorm_fwd(w, w)),
    ("dY", lambda: nf4.layernorm_bwd(X, X, w, stat, stat)), ("dY", lambda: nf4.layernorm_bwd(None, X, w, stat, stat)),
    ("ids", lambda: nf4.route(OFF, 2)), ("ids", lambda: nf4.route(None, 2)), ("ids", lambda: nf4.route(X, 2)),
    ("X", lambda: nf4.adapters_fwd(X, L1, L2, s, OFF)), ("X", lambda: nf4.adapters_fwd(None, L1, L2, s, OFF)),
    ("X", lambda: nf4.adapters_fwd(L1, L1, L2, s, OFF)),
    ("dY", lambda: nf4.adapters_bwd(dY, X, T, L1, L2, s, OFF)),
    ("dY", lambda: nf4.adapters_bwd(None, X, T, L1, L2, s, OFF)),
]


@pytest.mark.parametrize("i", range(len(CALLS)))
def test_refused_without_a_gpu(i):
    name, call = CALLS[i]
    with pytest.raises(ValueError, match=f"^{name}: "):
        call()


def test_workspaces_without_a_gpu():
    assert nf4.layernorm_workspace_bytes(8, 272) > 0 and nf4.route_workspace_bytes(8, 4) == 0
    for call in (lambda: nf4.layernorm_workspace_bytes(8, 24), lambda: nf4.route_workspace_bytes(8, 0),
                 lambda: nf4.adapters_workspace_bytes(nf4.NF4_OP_BWD, 8, 144, 272, 4, 12)):
        with pytest.raises(RuntimeError):
            call()
