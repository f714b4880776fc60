"""What the autograd operators keep for a backward pass, without a GPU (the calls below them are replaced)."""
import contextlib

import pytest
import torch

import self_attention_gb300 as sa


@pytest.fixture
def kept(monkeypatch):
    asked = []

    def forward(x, w, bias=None, residual=None, activation="none", keep_z=False):
        asked.append(keep_z)
        y = x.detach() @ w.detach()
        return (y, y.clone()) if keep_z else y

    monkeypatch.setattr(sa, "linear_forward", forward)
    return asked


@pytest.mark.parametrize("mode,kept_there", [(contextlib.nullcontext, True), (torch.enable_grad, True),
                                             (torch.no_grad, False), (torch.inference_mode, False)])
def test_the_pre_activation_is_kept_for_a_graph_alone(kept, mode, kept_there):
    """Serving a trained model without a graph writes no z: weights that require gradients do not ask for it."""
    x, w, res = torch.ones(3, 8), torch.ones(8, 8, requires_grad=True), torch.ones(3, 8, requires_grad=True)
    with mode():
        y = sa.linear(x, w, None, None, "gelu")
        assert kept == [kept_there] and y.requires_grad == kept_there
        sa.linear(x, w)                                     # z is not needed without an activation,
        sa.linear(x, w.detach(), None, res, "gelu")         # nor for the residual's gradient
    assert kept == [kept_there, False, False]
