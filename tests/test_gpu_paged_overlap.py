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
