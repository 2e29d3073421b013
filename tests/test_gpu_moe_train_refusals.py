"""MoETrainLayer.backward: weights and gradients of another shape, order or type are refused before anything is launched."""
from __future__ import annotations

import pytest
import torch

from combine_get_dispatch_notify_gb300 import ep
from test_gpu_moe_train import make, step

pytestmark = pytest.mark.gpu


def test_backward_refuses_weights_and_gradients_of_another_shape():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    args = make("tiny")
    shape, route, F, cap = args[:4]
    x, logits, bias, w13, w2, grad = (t.cuda() for t in args[4:])
    layer = ep.MoETrainLayer(shape, route, F, cap)
    step(layer, x, logits, bias, w13, w2, grad)
    gl = torch.full_like(logits, 7.0)
    g13, g2 = (torch.full_like(t, 7.0, dtype=torch.float32) for t in (w13, w2))
    swapped = lambda t: t.transpose(1, 2).contiguous()  # noqa: E731
    good = dict(w13=w13, w2=w2, grad_w13=g13, grad_w2=g2)
    before = layer.grad_x.clone()
    layer.grad_x.fill_(7.0)
    for name, bad in (("w13", swapped(w13)), ("w13", w13.float()), ("w13", None), ("w2", swapped(w2)),
                      ("grad_w13", swapped(g13)), ("grad_w13", g13.transpose(1, 2)), ("grad_w13", g13.half()),
                      ("grad_w13", None), ("grad_w2", swapped(g2)), ("grad_w2", g2.double())):
        a = dict(good, **{name: bad})
        with pytest.raises(ValueError, match=name):
            layer.backward(grad, logits, a["w13"], a["w2"], gl, a["grad_w13"], a["grad_w2"])
    torch.cuda.synchronize()
    for t in (layer.grad_x, gl, g13, g2):
        assert (t == 7.0).all()
    assert torch.equal(layer.backward(grad, logits, w13, w2, gl, g13, g2), before)
