"""The differentiable operators have no forward-mode derivative: an argument that
carries a tangent is refused, so that none is lost."""
import pytest
import torch
from torch.autograd import forward_ad

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu


def calls(x, weight, bias, ids, labels, teacher):
    return {
        "embed": lambda: og.embed(x, labels),
        "layer_norm": lambda: og.layer_norm(x, weight, bias),
        "layer_norm_out": lambda: og.layer_norm(x, weight, bias, out=torch.empty(6, 24,
                                                                                 device="cuda")),
        "distill_loss": lambda: og.distill_loss(x, ids, teacher, labels, hard_weight=0.5),
    }


def arguments():
    rand = lambda *s: torch.randn(*s, device="cuda")
    return dict(x=rand(6, 24), weight=rand(24), bias=rand(24),
                ids=torch.randint(24, (6, 3), device="cuda"),
                labels=torch.arange(6, device="cuda"), teacher=rand(6, 3))


@pytest.mark.parametrize("call,name", [
    ("embed", "x"), ("layer_norm", "x"), ("layer_norm", "weight"), ("layer_norm", "bias"),
    ("layer_norm_out", "x"), ("distill_loss", "x"), ("distill_loss", "teacher")])
@pytest.mark.parametrize("grad", [True, False])
def test_an_argument_with_a_tangent_is_refused(call, name, grad):
    args = arguments()
    with forward_ad.dual_level():
        dual = dict(args)
        dual[name] = forward_ad.make_dual(args[name], torch.randn_like(args[name]))
        with torch.set_grad_enabled(grad), pytest.raises(RuntimeError, match="forward"):
            calls(**dual)[call]()
        # Arguments without one go through, within the level too.
        result = calls(**args)[call]()
        assert forward_ad.unpack_dual(result).tangent is None
    assert torch.equal(result, calls(**args)[call]())


@pytest.mark.parametrize("call", ["embed", "layer_norm", "distill_loss"])
def test_an_argument_with_a_tangent_and_a_gradient_is_refused(call):
    args = arguments()
    args["x"].requires_grad_()
    with forward_ad.dual_level():
        args["x"] = forward_ad.make_dual(args["x"], torch.randn(6, 24, device="cuda"))
        with pytest.raises(RuntimeError, match="forward"):
            calls(**args)[call]()
