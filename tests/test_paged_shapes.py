"""Shapes that the binding of the exact paged cache refuses on the host: a
tensor with entries besides the ones that the call would read."""
import pytest
import torch

import nystr_coreset_approximate_b200 as wc

I32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("shape", [(2, 1), (2, 3), ()], ids=str)
def test_lengths_have_one_dimension(shape):
    """[B, k] lengths would be read as the first B entries of the first rows."""
    wide, lens, cu, table = torch.zeros(shape, **I32), torch.zeros(2, **I32), torch.zeros(3, **I32), torch.zeros(2, 3, **I32)
    q, pool = torch.zeros(5, 2, 64), torch.zeros(3, 2, 16, 64)
    for call in (
        lambda: wc.page_tables(wide, lens, table, lens, lens, 16, 4),
        lambda: wc.page_tables(lens, wide, table, lens, lens, 16, 4),
        lambda: wc.paged_attend(q, pool, pool, table, wide, cu, 0.1),
        lambda: wc.paged_attend(q, pool, pool, table, lens, torch.zeros(3, 1, **I32), 0.1),
        lambda: wc.paged_write(q, q, torch.zeros(5, 1, **I32), pool, pool),
    ):
        with pytest.raises(ValueError, match=r"one dimension|must be \["):
            call()


def test_the_message_names_the_lengths():
    wide, table = torch.zeros(2, 3, **I32), torch.zeros(2, 3, **I32)
    with pytest.raises(ValueError, match="ctx_lens must have one dimension"):
        wc.page_tables(wide, torch.zeros(2, **I32), table, wide, wide, 16, 4)
    with pytest.raises(ValueError, match="seq_lens must have one dimension"):
        wc.paged_attend(torch.zeros(5, 2, 64), *[torch.zeros(3, 2, 16, 64)] * 2, table, wide, torch.zeros(3, **I32), 0.1)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_the_workspace_does_not_depend_on_the_requests(d):
    """It holds two pieces of 256 rows for each of 148 SMs (148 where no GPU is there to ask) with a maximum and a sum for each
    row, a join for each, and the padding of three parts."""
    sizes = {int(wc.lib().wildcat_paged_attend_workspace_size(B, d)) for B in (0, 1, 1000, 65535)}
    pieces = 2 * 148 * 256 * (d + 2) * 4
    assert len(sizes) == 1 and (torch.cuda.is_available() or pieces <= sizes.pop() <= pieces + 148 * 16 + 1024)
