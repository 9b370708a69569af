"""Paged attention calls that follow each other without a pause on one workspace: each
launch overlaps the one before, and must not read what an earlier call left there."""

import pytest

from exact_io_aware_69_b200 import fa

from paged_cases import make_batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shapes", [
    [([(1, 9000)], 64), ([(1, 7000), (1, 30)], 16), ([(1, 8500)], 64)],      # the step kernel
    [([(70, 4000)], 64), ([(1, 9000)], 16), ([(300, 900), (40, 5000)], 32)],  # both
])
def test_calls_in_a_row_share_a_workspace(shapes):
    import torch
    batches = [make_batch(lengths, 8, 2, 128, page, torch.bfloat16, seed=i, fill=0.0)
               for i, (lengths, page) in enumerate(shapes)]
    size = max(fa.paged_workspace_size(b.q.shape[0], b.max_q, 8, 2, 128) for b in batches)
    workspace = torch.full((size,), 255, device="cuda", dtype=torch.uint8)
    wants = []
    for b in batches:
        wants.append(fa.paged_attention(b.q, *b.cache, max_q=b.max_q))
        torch.cuda.synchronize()
    got = [(i, fa.paged_attention(batches[i].q, *batches[i].cache, max_q=batches[i].max_q,
                                  workspace=workspace))
           for i in [0, 1, 2, 2, 1, 0] * 50]
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    for i, (o, L) in got:
        assert torch.equal(o, wants[i][0]) and torch.equal(L, wants[i][1])


@pytest.mark.parametrize("n", [1, 50])
def test_a_decreasing_cu_q_leaves_the_batch_out(n):
    """Rows might belong to two sequences: none is written, and the status says so."""
    import torch
    batch = make_batch([(n, 300), (n, 200), (n, 700)], 4, 2, 128, 64, torch.bfloat16, seed=5)
    for cu in ([0, n, n - 1, 3 * n], [0, 3 * n, 0, 3 * n], [n, 0, 2 * n, 3 * n]):
        out = torch.full_like(batch.q, 7.0)
        lse = torch.full((4, 3 * n), 7.0, device="cuda")
        fa.paged_attention(batch.q, batch.k_pages, batch.v_pages, batch.page_table,
                           torch.tensor(cu, dtype=torch.int32, device="cuda"), batch.seq_k,
                           max_q=3 * n, out=out, lse=lse)
        assert fa.device_status() == fa.FA_ERR_INVALID
        assert (out == 7).all() and (lse == 7).all()
