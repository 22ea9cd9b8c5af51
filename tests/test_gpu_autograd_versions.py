"""Tensors that the operators write to through their addresses count as changed for
autograd: a graph that saved one of them refuses its backward pass instead of going
on with what stands there now.  Tensors that are only read do not count."""
import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

N, DIM = 12, 64


def rand(*shape):
    return torch.randn(*shape, device="cuda")


def logits_overwritten(z, keep):
    og.distill_loss_grad(z.detach(), None, None, keep["labels"], hard_weight=1.0, out=z.detach())


def y_overwrites(x, keep):
    og.layer_norm(x.detach(), out=x.detach())


def x_grad_overwrites_x(x, keep):
    og.layer_norm_grad(keep["dy"], x.detach(), None, keep["stats"], x_grad=x.detach())


def x_grad_overwrites_grad_out(x, keep):
    og.layer_norm_grad(x.detach(), keep["x"], None, keep["stats"], x_grad=x.detach())


def weight_grad_overwrites(x, keep):
    og.layer_norm_grad(keep["dy"], keep["x"], None, keep["stats"], weight_grad=x.detach()[0])


def bias_grad_adds(x, keep):
    og.layer_norm_grad(keep["dy"], keep["x"], None, keep["stats"], weight_grad=False,
                       bias_grad=x.detach()[1], accumulate=True)


def lookup_overwrites(x, keep):
    og.embed(keep["x"], keep["ids"], out=x.detach())


def table_grad_overwrites(x, keep):
    og.embed_grad(keep["dy"], keep["ids"], out=x.detach())


WRITES = [logits_overwritten, y_overwrites, x_grad_overwrites_x, x_grad_overwrites_grad_out,
          weight_grad_overwrites, bias_grad_adds, lookup_overwrites, table_grad_overwrites]


def others():
    x = rand(N, DIM)
    return dict(x=x, dy=rand(N, DIM), stats=og.layer_norm(x, stats=True)[1],
                ids=torch.arange(N, device="cuda"), labels=torch.arange(N, device="cuda"))


GRAPHS = [lambda z: og.distill_loss(z, None, None, torch.arange(N, device="cuda"),
                                    hard_weight=1.0).sum(),
          lambda z: og.layer_norm(z).square().sum(),
          lambda z: z.square().sum()]


@pytest.mark.parametrize("write", WRITES, ids=lambda f: f.__name__)
@pytest.mark.parametrize("graph", range(len(GRAPHS)))
def test_a_graph_that_saved_what_was_overwritten_refuses(write, graph):
    leaf = rand(N, DIM).requires_grad_()
    z = leaf * 1.0
    total = GRAPHS[graph](z)
    keep = others()
    read = {k: t._version for k, t in keep.items()}
    write(z, keep)
    assert {k: t._version for k, t in keep.items()} == read   # what is only read
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        total.backward()


@pytest.mark.parametrize("graph", range(len(GRAPHS)))
def test_new_results_and_norms_leave_graphs_alone(graph):
    leaf = rand(N, DIM).requires_grad_()
    z = leaf * 1.0
    total = GRAPHS[graph](z)
    keep, d = others(), z.detach()
    og.distill_loss_grad(d, None, None, keep["labels"], hard_weight=1.0)
    _, stats = og.layer_norm(d, stats=True)
    og.layer_norm_grad(d, d, None, stats)
    og.embed(d, keep["ids"])
    og.embed_grad(d, keep["ids"], n_rows=N)
    with og.GradClip([d.view(-1)]) as clip:
        clip.norm()
    total.backward()
    assert bool(leaf.grad.isfinite().all())


@pytest.mark.parametrize("write", WRITES, ids=lambda f: f.__name__)
def test_tensors_of_inference_mode_have_no_versions(write):
    """They are written to as before, within that mode and outside."""
    with torch.inference_mode():
        x = rand(N, DIM)
        was = x.clone()
        write(x, others())
        assert not torch.equal(x, was)
    was = x.clone()
    write(x, others())
    assert not torch.equal(x, was)
