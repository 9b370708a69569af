"""Paged attention and what lies outside a row's mask: values of keys that a row does not see,
however large, leave its output as it is."""

import pytest

from exact_io_aware_69_b200 import fa

from paged_cases import make_batch, reference

pytestmark = pytest.mark.gpu

HUGE = {"bfloat16": 3.0e38, "float16": 65504.0}


def set_values(batch, b, keys, value):
    """Sets sequence b's cached values at `keys` in the pool and in the plain copy."""
    import torch
    pages = batch.v_pages if batch.layout == "bnhd" else batch.v_pages.transpose(1, 2)
    size = pages.shape[1]
    j = torch.tensor(list(keys))
    pages[batch.page_table[b, j // size].long(), j % size] = value
    batch.values[b][j] = value


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group,first,window", [
    (40, 1, 30, (-1, 0)),      # one query tile, a few of its later tokens
    (300, 4, 200, (-1, 0)),    # two query tiles
    (260, 2, 37, (-1, 0)),
    (90, 2, 64, (20, 3)),      # before the window of some rows, behind that of others
    (16, 1, 9, (-1, 0)),       # the step kernel
    (4, 4, 2, (-1, 0)),
])
def test_values_outside_a_rows_mask(n, group, first, window, d, dtype):
    """Sixteen neighbouring new tokens (fewer for short drafts) with the type's largest values:
    rows that see none of them are within the bounds of the definition. (Those that see
    them may pass the type's range.)"""
    import torch
    lengths = [(n, 700 + n), (n, n)]
    batch = make_batch(lengths, 2 * group, 2, d, 32, getattr(torch, dtype), seed=n + d)
    rows = torch.arange(n, device="cuda")
    left = n if window[0] < 0 else window[0]
    last = min(first + 16, n)
    blind = (rows + window[1] < first) | (rows - left >= last)
    assert blind.any() and not blind.all()
    for b, (_, k) in enumerate(lengths):
        set_values(batch, b, range(k - n + first, k - n + last), HUGE[dtype])
    o, L = fa.paged_attention(batch.q, *batch.cache, max_q=n, window=window)
    assert fa.device_status() == fa.FA_OK
    for b, (ro, rl, bo, bl) in enumerate(reference(batch, d ** -0.5, window)):
        go, gl = o[b * n:(b + 1) * n].double(), L[:, b * n:(b + 1) * n].double()
        assert ((go - ro).abs()[blind] <= bo[blind]).all()
        assert ((gl - rl).abs() <= bl).all()
