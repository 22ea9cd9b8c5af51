"""Temperatures and weights of the distillation loss whose exponents or shares fp32 does
not hold are refused before anything touches a GPU."""
import pytest

import optimizer_step_gb300 as og
from optimizer_step_gb300 import _lib
from test_train_ops_model_abi import distill_args


@pytest.mark.parametrize("change", [
    dict(temperature=3e-39),                       # log2(e) / T
    dict(temperature=4.2e-39),
    dict(temperature=1e30, soft_weight=1e9),       # soft_weight T
    dict(temperature=3e38, soft_weight=-2.0),
    dict(temperature=2.0, soft_weight=3e38),
])
@pytest.mark.parametrize("labels", [4096, None])
def test_products_past_fp32_are_refused(change, labels):
    lib = og.load()
    change = dict(change, labels=labels, hard_weight=1.0 if labels else 0.0)
    assert lib.train_distill(*distill_args(**change)) == _lib.LAMB_ERR_INVALID
    assert b"temperature" in lib.lamb_last_error()


@pytest.mark.parametrize("change", [dict(temperature=3e-39),
                                    dict(temperature=2.0, soft_weight=3e38)])
def test_without_a_teacher_they_do_not_matter(change):
    """Without rows nothing is launched."""
    for less in (dict(top_k=0), dict(soft_weight=0.0)):
        args = distill_args(**{**change, **less, "n_rows": 0})
        assert og.load().train_distill(*args) == _lib.LAMB_OK
