"""The gated delta rule's binding where it needs no GPU."""
import pytest
import torch

from selective_state_space_05_gb300 import delta


@pytest.mark.parametrize("grad,leaf,want", [(True, True, True), (True, False, False),
                                            (False, True, False), (False, False, False)])
def test_kept_only_for_a_backward(monkeypatch, grad, leaf, want):
    """Without grad mode nothing is kept, learned initial states or not."""
    asked = []

    def fwd(q, k, v, g, beta, *, save, **kw):
        asked.append(save)
        return (torch.zeros_like(v), torch.zeros(1, 1, 4, 8)) + ((torch.zeros(1),) if save else ())
    monkeypatch.setattr(delta, "delta_scan_fwd", fwd)
    q, v, g = torch.zeros(1, 2, 1, 8), torch.zeros(1, 2, 1, 4), torch.zeros(1, 2, 1)
    init = torch.zeros(1, 1, 4, 8, requires_grad=leaf)
    with torch.set_grad_enabled(grad):
        out, fin = delta.delta_scan(q, q, v, g, g, initial_states=init, return_final_states=True)
    assert asked == [want] and out.requires_grad == fin.requires_grad == want
