"""Which sizes of layer norm's gradients go to one cluster, which needs no workspace."""
import ctypes

import pytest

import optimizer_step_gb300 as og


def workspace(n, dim):
    need = ctypes.c_int64()
    assert og.load().train_layer_norm_grad_workspace(n, dim, ctypes.byref(need)) == 0
    return need.value


@pytest.mark.parametrize("n,dim", [(14000, 9), (26214, 5), (131072, 1), (4097, 1), (8192, 16)])
def test_many_short_rows_are_spread_over_the_gpu(n, dim):
    assert workspace(n, dim) > 0


@pytest.mark.parametrize("n,dim", [(1, 1), (512, 256), (128, 1024), (4096, 32), (4096, 1)])
def test_few_rows_need_no_workspace(n, dim):
    assert workspace(n, dim) == 0
