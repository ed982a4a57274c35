"""Python arguments that the rotary entries refuse rather than take for something else (no GPU needed)."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg


def test_rows_that_want_a_gradient_are_refused():
    # the entry keeps no graph: the output would silently be a constant of the loss
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16, requires_grad=True)
    table, pos = pkg.rope_table(8, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="gradient"):
        pkg.sdpa_rope(x, table, pos)
    for x_ in (x.detach(), x):  # (what is next to refuse: no CUDA device)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
            pkg.sdpa_rope(x_, table, pos)


@pytest.mark.parametrize("rot_dims", [0, -16, 17, 63, 24])
def test_tables_of_other_than_whole_pairs_are_refused(rot_dims):
    # 17 would be 8 pairs with the angles of 17 dims, which the entries cannot tell from 16
    with pytest.raises(ValueError, match="rot_dims"):
        pkg.rope_table(4, rot_dims)
