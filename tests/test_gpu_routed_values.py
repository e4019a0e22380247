"""The operators around the experts' products at values, states and sizes that the other tests leave
out."""
import pytest
import torch
from torch.autograd import forward_ad

import gpu_util as gu
from test_gpu_routed import normal

pytestmark = pytest.mark.gpu


def test_router_refuses_forward_mode_derivatives():
    """A tangent is refused, not dropped."""
    m = gu.need_gpu()
    logits, dw = normal(1, (5, 8), torch.float32), normal(2, (5, 2), torch.float32)
    ids, w = m.moe_topk_softmax(logits, 2)
    with forward_ad.dual_level():
        dual, dual_dw, dual_w = (forward_ad.make_dual(t, torch.ones_like(t)) for t in (logits, dw, w))
        for call in (lambda: m.moe_topk_softmax(dual, 2),
                     lambda: m.moe_topk_softmax(forward_ad.make_dual(logits.clone().requires_grad_(), logits), 2),
                     lambda: m.moe_topk_softmax_backward(dual_dw, ids, w, 8),
                     lambda: m.moe_topk_softmax_backward(dw, ids, dual_w, 8)):
            with pytest.raises(NotImplementedError, match="forward"):
                call()
        ids2, w2 = m.moe_topk_softmax(logits, 2)  # no tangent: as ever
        assert torch.equal(ids2, ids) and torch.equal(w2, w)
        m.moe_topk_softmax_backward(dw, ids, w, 8)
