"""The binding of the paged cache operators without a GPU."""

import contextlib
import types

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


class OnDevice(contextlib.AbstractContextManager):
    """Stands for the context that makes the tensors' device current."""

    inside = False

    def __enter__(self):
        OnDevice.inside = True

    def __exit__(self, *exc):
        OnDevice.inside = False


class Library:
    """Stands for the library: says in which context its functions were called."""

    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        def call(*args):
            self.seen.append((name, OnDevice.inside))
            return 64 if name.endswith("workspace") else 0

        return call


def test_scratch_is_sized_with_the_tensors_device_current(monkeypatch):
    """Scratch goes by the SMs of the device that is current when its size is asked for."""
    lib = Library()
    monkeypatch.setattr(kv, "_load", lambda: lib)
    monkeypatch.setattr(kv, "_for", lambda stream, device: (0, OnDevice()))
    monkeypatch.setattr(kv, "_status", lambda status, device: 0)
    monkeypatch.setattr(kv, "_on_device", lambda name, t: None)
    monkeypatch.setattr(kv, "_given", lambda name, t, *form: t)
    monkeypatch.setattr(kv, "_checked", kv._Checked())
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    table, lens, refs = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    codes, scales = torch.zeros((4, 2, 2, 64), dtype=torch.int8), torch.zeros((4, 2))
    kv.ibp_tree_attention(q, k, k, table, lens)
    kv.ibp_sparse_attention(q, k, k, table, lens, codes, scales, 2)
    kv.ibp_kv_fork(table, lens, refs, lens, 16)
    kv.ibp_kv_compact(table, refs, 16)
    sized = [inside for name, inside in lib.seen if name.endswith("workspace")]
    assert len(sized) == 4 and all(sized), lib.seen


def test_kept_checks_are_of_one_device():
    """Alike tensors of two GPUs, which may differ in their SMs, share no entry."""
    t = torch.zeros((2, 3))

    def on(index):
        return types.SimpleNamespace(shape=t.shape, stride=t.stride, dtype=t.dtype, is_cuda=True,
                                     device=torch.device("cuda", index))

    assert kv._form(on(0)) == kv._form(on(0)) != kv._form(on(1))
