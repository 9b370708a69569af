"""Paged attention over keys that are not finite: a NaN or an infinite score shows in the O
and L of the rows that see it, at every place of a key tile, and in no other row."""

import pytest

from exact_io_aware_69_b200 import fa

from paged_cases import make_batch

pytestmark = pytest.mark.gpu

# (new tokens, query heads of a key head, keys): the step kernel, and the chunk kernel with
# one and with two query tiles an item
CASES = [(1, 4, 700), (3, 2, 300), (50, 1, 300), (20, 4, 3000), (200, 1, 500), (130, 4, 2000)]


def key_row(batch, b, key, head):
    """The pool's row of a key of sequence b (a view)."""
    pages = batch.k_pages if batch.layout == "bnhd" else batch.k_pages.transpose(1, 2)
    size = pages.shape[1]
    return pages[int(batch.page_table[b, key // size]), key % size, head]


def seen(n, keys, key):
    """Which of n new tokens see `key` under the causal mask."""
    import torch
    return torch.arange(n, device="cuda") + keys - n >= key


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group,keys", CASES)
def test_a_nan_key_at_every_place(n, group, keys, d):
    """One NaN key at a time: sixteen neighbouring places in each half of the last whole tile,
    and among the new tokens."""
    import torch
    batch = make_batch([(n, keys), (n, keys)], 2 * group, 2, d, 64, torch.bfloat16, seed=n)
    plain, plain_l = fa.paged_attention(batch.q, *batch.cache, max_q=n)
    tile = (keys // 128 - 1) * 128
    places = list(range(tile + 16, tile + 32)) + list(range(tile + 80, tile + 96))
    places += range(max(0, keys - n), min(keys, keys - n + 16))
    for key in places:
        row = key_row(batch, 1, key, 0)
        old = row.clone()
        row[5] = float("nan")
        o, L = fa.paged_attention(batch.q, *batch.cache, max_q=n)
        row.copy_(old)
        bad = torch.zeros(2 * n, 2 * group, dtype=torch.bool, device="cuda")
        bad[n:, :group] = seen(n, keys, key)[:, None]
        assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad), key
        assert torch.equal(L.isnan().T, bad), key
        assert torch.equal(o[~bad], plain[~bad]) and torch.equal(L.T[~bad], plain_l.T[~bad])
    assert fa.device_status() == fa.FA_OK


def without(batch, n, keys, key, d):
    """(O, its bound, L, its bound) of the one sequence's first key head, [n, group, ..], as
    if `key` were hidden: reference()'s bounds for bf16."""
    import torch
    group = batch.q.shape[1] // batch.keys[0].shape[1]
    q = batch.q[:, :group].double()
    k, v = (x[0][:, 0].double().cuda() for x in (batch.keys, batch.values))
    s = torch.einsum("igd,jd->igj", q, k) * d ** -0.5
    j = torch.arange(keys, device="cuda")
    hidden = (j > torch.arange(n, device="cuda")[:, None, None] + keys - n) | (j == key)
    s = s.masked_fill(hidden, -float("inf"))
    L = s.logsumexp(-1)
    w = (s - L[..., None]).exp()
    e = torch.einsum("igd,jd->igj", q.abs(), k.abs()).amax(-1) * d ** -0.5 * d * 2.0 ** -23
    u = 2.0 ** -8
    bound = (2 * u / (1 - u) + 4 * e[..., None]) * (w @ v.abs()) + u * (w @ v).abs() + 2.0 ** -25
    return w @ v, bound, L, e + 2e-6 * (1 + L.abs())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group,keys", CASES)
def test_an_infinite_key_at_every_place(n, group, keys, d):
    """A key of zeros with one infinite column: the score is +inf for queries with a positive
    value there, whose softmax is not a number, and -inf for those with a negative one,
    whose weight for it is 0."""
    import torch
    batch = make_batch([(n, keys)], 2 * group, 2, d, 32, torch.bfloat16, seed=n + 1)
    column = batch.q[:, :, 9]
    column[column == 0] = 0.5  # infinity times 0 is not a number
    tile = (keys // 128 - 1) * 128
    for key in list(range(tile + 16, tile + 32)) + list(range(tile + 80, tile + 96)):
        row = key_row(batch, 0, key, 0)
        old = row.clone()
        row.zero_()
        row[9] = float("inf")
        o, L = fa.paged_attention(batch.q, *batch.cache, max_q=n)
        row.copy_(old)
        sees = seen(n, keys, key)[:, None]
        bad = torch.zeros(n, 2 * group, dtype=torch.bool, device="cuda")
        bad[:, :group] = (column[:, :group] > 0) & sees
        assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad), key
        assert torch.equal(L.isnan().T, bad), key
        ro, bo, rl, bl = without(batch, n, keys, key, d)
        low = (column[:, :group] < 0) & sees
        assert ((o[:, :group].double() - ro).abs() <= bo)[low].all(), key
        assert ((L.T[:, :group].double() - rl).abs() <= bl)[low].all(), key
    assert fa.device_status() == fa.FA_OK
