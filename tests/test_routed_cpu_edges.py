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
