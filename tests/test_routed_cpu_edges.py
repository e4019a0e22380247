"""Host behaviour around the align buffer's description: copies, and what a backward pass keeps."""
import copy
import os
import pickle

import pytest
import torch

import expert_adapter_gemms_gb300 as m


@pytest.fixture(scope="session")
def L():
    from expert_adapter_gemms_gb300 import build as b
    if not os.path.exists(b.LIB_PATH):
        b.build()
    return m.lib()


def fake_align(T=4, k=1, E=1, L=2):
    return m.Align(torch.zeros(1 << 12, dtype=torch.uint8), T, k, E, L, 256, 16)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda al: pickle.loads(pickle.dumps(al))],
                         ids=["copy", "deepcopy", "pickle"])
def test_a_used_align_can_be_copied(L, how):
    """As before its first use: nothing that the calls keep with it stands in the way, and the copy
    describes its own buffer."""
    al = fake_align()
    al.buf[:4] = torch.arange(4, dtype=torch.uint8)
    first, size = al.ref(), al.linear_workspace_size(64, 64, 8, 0, 0)
    other = how(al)
    assert type(other) is m.Align
    assert torch.equal(other.buf, al.buf)
    assert all(getattr(other, f) == getattr(al, f) for f in ("T", "k", "E", "L", "bm_base", "bm_lora"))
    assert (other.buf is al.buf) == (how is copy.copy)
    assert other.ref()._obj.buf == other.buf.data_ptr() and other.ref()._obj.T == 4
    assert other.linear_workspace_size(64, 64, 8, 0, 0) == size
    other.T = 300
    assert al.T == 4 and al.ref() is first and al.linear_workspace_size(64, 64, 8, 0, 0) == size
    assert other.ref()._obj.T == 300 and other.linear_workspace_size(64, 64, 8, 0, 0) > size


def functions(monkeypatch, seen):
    """The differentiable calls with their kernels' launches replaced: what the backward passes are
    given goes into `seen`. Each takes the leaf that the result hangs on and the align."""
    from expert_adapter_gemms_gb300 import routed
    monkeypatch.setattr(routed, "stream_handle", lambda: 0)
    monkeypatch.setattr(routed, "_permute", lambda x, al, out, stream: x.repeat_interleave(al.k, 0))

    def unpermute(o, al, w, out, stream):
        seen.append(al)
        return o.view(-1, 2, o.shape[1]).sum(1)

    def unpermute_backward(dy, o, al, w, need_do, need_dw):
        seen.append(al)
        return dy.repeat_interleave(2, 0), None

    def linear_backward(dy, x, W, A, B, al, **kw):
        seen.append(al)
        return dy, None, None

    monkeypatch.setattr(routed, "_unpermute", unpermute)
    monkeypatch.setattr(routed, "moe_unpermute_backward", unpermute_backward)
    monkeypatch.setattr(routed, "_linear", lambda x, *args: x.clone())
    monkeypatch.setattr(routed, "moe_lora_linear_backward", linear_backward)
    other = torch.zeros(1)
    return {"permute": (4, lambda x, al: routed._Permute.apply(x, al)),
            "unpermute": (8, lambda x, al: routed._Unpermute.apply(x, None, al)),
            "linear": (8, lambda x, al: routed._LoraLinear.apply(x, other, other, other, al, True, None))}


@pytest.mark.parametrize("op", ["permute", "unpermute", "linear"])
@pytest.mark.parametrize("hooks", [False, True], ids=["kept", "packed"])
def test_backward_keeps_the_forward_order(monkeypatch, op, hooks):
    """One description serves batch after batch: a program gives it the next batch's sizes and buffer
    before it goes back through this one. The backward pass still has this one's; with the next one's
    it would read past the rows that it is given."""
    seen = []
    rows, call = functions(monkeypatch, seen)[op]
    al = fake_align(T=4, k=2, E=4, L=2)
    buf = al.buf
    buf[:8] = torch.arange(8, dtype=torch.uint8)
    x = torch.ones(rows, 16, requires_grad=True)
    if hooks:  # as when activations are put elsewhere meanwhile
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone(), lambda t: t):
            y = call(x, al)
        buf[:8] = 0
    else:
        y = call(x, al)
    al.T, al.k, al.E, al.L, al.buf = 4096, 8, 64, 16, torch.zeros(1 << 13, dtype=torch.uint8)
    seen.clear()
    y.sum().backward()
    used, = seen
    assert (used.T, used.k, used.E, used.L, used.bm_base, used.bm_lora) == (4, 2, 4, 2, 256, 16)
    assert used.buf[:8].tolist() == list(range(8)) and (hooks or used.buf is buf)
    assert al.T == 4096 and al.buf is not used.buf


@pytest.mark.parametrize("op", ["permute", "unpermute", "linear"])
def test_backward_uses_the_kept_description(L, monkeypatch, op):
    """The plain case makes nothing anew: buffer, description and sizes are those of the forward call."""
    seen = []
    rows, call = functions(monkeypatch, seen)[op]
    al = fake_align(T=4, k=2, E=4, L=2)
    ref = al.ref()
    y = call(torch.ones(rows, 16, requires_grad=True), al)
    seen.clear()
    y.sum().backward()
    assert seen[0].buf is al.buf and seen[0].ref() is ref


def test_align_refuses_ids_that_end_before_its_slots(L, monkeypatch):
    """A buffer made for more tokens, or more experts a token, would be aligned from what lies behind the
    ids. (The look at the device is left out: what is not refused fails for want of a GPU.)"""
    from expert_adapter_gemms_gb300 import api
    monkeypatch.setattr(api, "_need", lambda t, *args: t)
    monkeypatch.setattr(api, "stream_handle", lambda: 0)
    monkeypatch.setattr(api, "lib", lambda: pytest.fail("not refused"))
    ids = lambda T, k: torch.zeros((T, k), dtype=torch.int32)  # noqa: E731
    for al, args in ((fake_align(T=9, k=2), (ids(8, 2), None)), (fake_align(T=8, k=3), (ids(8, 2), None)),
                     (fake_align(T=8, k=1), (ids(4, 2), torch.zeros(4, dtype=torch.int32)))):
        with pytest.raises(ValueError, match="align buffer is for"):
            m.moe_lora_align(*args, al.E, al.L, al=al)
