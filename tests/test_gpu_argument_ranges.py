"""Token numbers at the ends of their range: right, or refused."""
import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

LAST = 2 ** 63 - 1


@pytest.mark.parametrize("beyond", [2 ** 63, 2 ** 64, 2 ** 64 + 3, -2 ** 63 - 1])
def test_token_numbers_beyond_64_bits_are_refused(beyond):
    """They would else count modulo 2^64."""
    table = torch.ones(10, 8, device="cuda")
    ids = torch.arange(4, device="cuda")
    with pytest.raises(ValueError):
        og.embed(table, ids, first_row=beyond)
    with pytest.raises(ValueError):
        og.embed_grad(table[:4], ids, n_rows=10, first_row=beyond)
    with pytest.raises(ValueError):
        og.embed_grad(table[:4], ids, n_rows=10, padding_id=beyond)


def test_a_slice_that_ends_at_the_last_token():
    table = torch.arange(3.0, device="cuda")[:, None] + torch.ones(3, 8, device="cuda")
    ids = torch.tensor([LAST, LAST - 2, -LAST - 1, -LAST, 0, LAST - 3], device="cuda")
    out = og.embed(table, ids, first_row=LAST - 2)
    assert out[:, 0].tolist() == [3.0, 1.0, 0.0, 0.0, 0.0, 0.0]
    for repeat in (1, 1000):
        grad = og.embed_grad(torch.ones(6 * repeat, 8, device="cuda"), ids.repeat(repeat),
                             n_rows=3, first_row=LAST - 2)
        assert grad[:, 0].tolist() == [repeat, 0.0, repeat]
