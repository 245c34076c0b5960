"""The binding of the paged cache operators without a GPU."""

import pytest
import torch

from host_transfer_gb300 import kv


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_gradient_for_attention_is_an_error(which):
    """The operators have no backward pass; a backward that reaches one says so."""
    args = [torch.randn(2, 3) for _ in range(3)]
    args[which].requires_grad_()
    out, lse = torch.randn(2, 3), torch.randn(2)
    got = kv._results("ibp_tree_attention", out, lse, *args)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    for x in got:
        with pytest.raises(RuntimeError, match="ibp_tree_attention has no backward"):
            x.sum().backward(retain_graph=True)
    assert args[which].grad is None
    with torch.no_grad():
        assert kv._results("", out, lse, *args)[0] is out
    assert kv._results("", out, lse, *(a.detach() for a in args))[0] is out
