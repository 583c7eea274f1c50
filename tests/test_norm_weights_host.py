"""Weights of HeadNorm that change after it was made: each call looks at them anew (no GPU needed)."""
import pytest
import torch

from attention_backward_flashattention_gb300 import binding


def _set(w, data):
    w.data = data


CHANGES = [
    lambda w: _set(w, w.data.to(torch.bfloat16)),
    lambda w: _set(w, w.data.double()),
    lambda w: _set(w, torch.ones(64, 2)[:, 0]),
    lambda w: _set(w, torch.ones(1, 64)),
    lambda w: _set(w, torch.ones(32)),
    lambda w: _set(w, torch.ones(())),
]


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("change", range(len(CHANGES)))
def test_changed_weights_are_refused(side, change):
    w = torch.nn.Parameter(torch.ones(64))
    norm = binding.HeadNorm(*((w, None) if side == 0 else (None, w)))
    norm.check(64)
    CHANGES[change](w)
    with pytest.raises(ValueError):
        norm.check(64)
    x = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: binding.norm_rope(x, x, norm),
                 lambda: binding.norm_rope_backward(x, x, x, x, norm)):
        with pytest.raises(ValueError, match="weight"):
            call()


def test_module_turned_to_another_type():
    module = torch.nn.Module()
    module.w = torch.nn.Parameter(torch.ones(128))
    norm = binding.HeadNorm(module.w, module.w)
    module.to(torch.bfloat16)
    with pytest.raises(ValueError, match="weight"):
        norm.check(128)
    module.to(torch.float32)
    norm.check(128)
    assert norm.struct.q_weight == norm.struct.k_weight == module.w.data_ptr()
