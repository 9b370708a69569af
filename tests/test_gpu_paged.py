"""The paged cache: fa.paged_append and fa.paged_attention against plain forms in 64 bits.

Ragged batches from one token to long chunks, pages that end inside a tile, grouped heads,
windows, rows that see no key; NaN in every row of the pool that holds no key; packed rows
behind the last sequence; strided inputs, other streams, captured graphs, bad pages."""

import math

import pytest

from exact_io_aware_69_b200 import fa

from paged_cases import check, make_batch, reference
from test_gpu_rope import close, freqs_of, plain

pytestmark = pytest.mark.gpu

CAUSAL, FULL = (-1, 0), (-1, -1)


def attend(batch, window, d, scale=None, **kw):
    import torch
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    T, hq = batch.q.shape[:2]
    out = torch.full_like(batch.q, 7.0)
    lse = torch.full((hq, T), 7.0, device="cuda")
    kw.setdefault("max_q", batch.max_q)
    o, L = fa.paged_attention(batch.q, *batch.cache, window=window, scale=scale,
                              page_layout=batch.layout, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    used = sum(n for n, _ in batch.lengths)
    assert (o[used:] == 7).all() and (L[:, used:] == 7).all(), "rows behind the last sequence"
    check(batch, o, L, scale, window)
    return o, L


ATTEND = [  # (lengths, hq, hkv, d, page, window)
    ([(1, 1)], 1, 1, 64, 16, CAUSAL),
    ([(1, 129)], 8, 1, 128, 16, CAUSAL),
    ([(1, 1000)], 32, 8, 128, 16, CAUSAL),
    ([(1, 300), (1, 5), (1, 127), (1, 128), (1, 2049)], 8, 2, 128, 32, CAUSAL),
    ([(1, 900), (0, 40), (1, 1), (1, 0), (0, 0), (1, 640)], 6, 2, 64, 64, CAUSAL),
    ([(1, 5000)], 4, 4, 64, 128, CAUSAL),
    ([(1, 3000), (1, 411)], 14, 2, 128, 256, (200, 0)),
    ([(1, 700)], 16, 1, 128, 1024, FULL),
    ([(1, 1300)], 71, 1, 64, 16, CAUSAL),
    ([(1, 600)], 128, 1, 128, 16, CAUSAL),
    ([(4, 700), (2, 33), (3, 4096), (1, 17)], 8, 2, 128, 16, CAUSAL),
    ([(5, 700), (5, 5), (3, 2), (4, 0)], 15, 3, 64, 32, CAUSAL),
    ([(16, 2000), (7, 300)], 4, 4, 128, 64, (100, 3)),
    ([(9, 1000)], 20, 4, 64, 16, FULL),
    ([(100, 100)], 4, 2, 128, 16, CAUSAL),
    ([(257, 1000), (128, 128), (1, 64), (64, 1030)], 8, 2, 128, 64, CAUSAL),
    ([(300, 300), (33, 2111), (1, 1999)], 7, 1, 64, 128, CAUSAL),
    ([(513, 700)], 3, 3, 64, 32, (130, 0)),
    ([(140, 90), (200, 0), (50, 1)], 6, 2, 128, 16, CAUSAL),
    ([(200, 1500)], 12, 4, 128, 256, (64, 100)),
    ([(1024, 3333)], 16, 2, 128, 64, CAUSAL),
    ([(60, 60)] * 9 + [(1, 800)] * 7, 5, 5, 64, 16, CAUSAL),
    ([(150, 700)], 128, 1, 64, 512, CAUSAL),
    ([(3, 20000)], 48, 1, 64, 64, CAUSAL),
    ([(1, 1 + 37 * i % 700) for i in range(300)], 8, 2, 128, 16, CAUSAL),
    ([(1, 1 + i % 5) for i in range(2100)], 2, 1, 64, 16, CAUSAL),
    ([(1 + 29 * i % 211, 211 + 67 * i % 400) for i in range(70)], 4, 2, 64, 32, CAUSAL),
    ([(200, 500), (1, 300)], 8, 2, 128, 64, (0, 0)),
    ([(2, 500)], 8, 2, 128, 64, (0, 0)),
    ([(130, 900)], 4, 4, 128, 128, (5, -1)),
    ([(65, 400)], 2, 1, 64, 16, (-1, 40)),
    ([(32, 600), (7, 7)], 1, 1, 128, 16, CAUSAL),
    ([(17, 600), (1, 33)], 1, 1, 64, 16, CAUSAL),
    ([(24, 600), (7, 7)], 1, 1, 128, 16, CAUSAL),
    ([(5, 900), (6, 3000)], 8, 2, 128, 32, (700, 0)),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("index", range(len(ATTEND)))
def test_attention(index, dtype):
    import torch
    lengths, hq, hkv, d, page, window = ATTEND[index]
    layout = "bnhd" if (index + (dtype == "float16")) % 2 else "bhnd"
    batch = make_batch(lengths, hq, hkv, d, page, getattr(torch, dtype), layout, seed=index,
                       behind=index % 4, gain=1.0 + index % 3)
    attend(batch, window, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 40, 140])
def test_runs_of_sequences_without_keys(n, d):
    """Behind each sequence with keys come many items without any, more than a CTA holds in
    its ring: those must not wait for the products that the item before still owes."""
    import torch
    for lengths in ([(n, 300 + n)] + [(n, 0)] * 9) * 8, [(n, 900)] + [(n, 0)] * 60, \
                   ([(n, 0)] * 5 + [(n, n)] + [(0, 9)] * 3) * 10:
        batch = make_batch(lengths, 16, 8, d, 32, torch.bfloat16, seed=n)
        attend(batch, CAUSAL, d)
        # rows beyond the keys of a sequence see none either
        batch = make_batch([(n, k // 9) for n, k in lengths], 8, 8, d, 32, torch.float16, seed=d)
        attend(batch, (0, 0), d)


def test_attention_is_the_same_every_time():
    import torch
    batch = make_batch([(70, 5000), (1, 3000), (300, 300)], 8, 2, 128, 16, torch.bfloat16, seed=3)
    first = attend(batch, CAUSAL, 128)
    for _ in range(3):
        again = attend(batch, CAUSAL, 128)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_attention_agrees_with_the_contiguous_calls():
    """The same sequence through a cache, forward() and decode(): one length, all heads their
    own keys. Each is within the 16-bit bounds of the definition, so they are within twice
    those of each other."""
    import torch
    n, d, h = 384, 128, 3
    batch = make_batch([(n, n)], h, h, d, 64, torch.bfloat16, seed=9)
    o, L = attend(batch, CAUSAL, d)
    q, k, v = (x.cuda()[None] for x in (batch.q, batch.keys[0], batch.values[0]))
    ro, rL, _ = fa.forward(q.contiguous(), k.contiguous(), v.contiguous(), causal=True,
                           layout="bnhd", residual=False)
    assert (o.float() - ro[0].float()).abs().max() <= 4e-2
    assert (L - rL[0]).abs().max() <= 2e-3
    step = make_batch([(1, n)], h, h, d, 64, torch.bfloat16, seed=9)
    o, L = attend(step, CAUSAL, d)
    q, k, v = (x.cuda()[None] for x in (step.q, step.keys[0], step.values[0]))
    ro, rL = fa.decode(q.contiguous(), k.contiguous(), v.contiguous(), causal=True, layout="bnhd")
    assert (o.float() - ro[0].float()).abs().max() <= 4e-2
    assert (L - rL[0]).abs().max() <= 2e-3


def test_pages_that_share_a_prefix_and_max_q_bounds():
    """Two sequences over the same pages, and any bound above the longest chunk: the same."""
    import torch
    batch = make_batch([(4, 640), (4, 640)], 8, 2, 128, 64, torch.bfloat16, seed=4)
    batch.page_table[1] = batch.page_table[0]
    batch.keys[1], batch.values[1] = batch.keys[0], batch.values[0]
    for max_q in (4, 8, 100, None):
        attend(batch, CAUSAL, 128, max_q=max_q)


@pytest.mark.parametrize("n", [1, 90])
def test_attention_strided(n):
    """q as part of a projection's output, K and V views of one pool, O into another view."""
    import torch
    batch = make_batch([(n, 333), (n, 90)], 4, 2, 64, 32, torch.float16, seed=6, one_pool=True)
    assert not batch.k_pages.is_contiguous()
    T = batch.q.shape[0]
    wide = torch.randn(T, 9, 64, device="cuda").half()
    wide[:, 3:7] = batch.q
    batch.q = wide[:, 3:7]
    target = torch.zeros(4, T, 64, device="cuda").half()
    scale = 0.125
    o, L = fa.paged_attention(batch.q, *batch.cache, max_q=n, out=target.transpose(0, 1))
    torch.cuda.synchronize()
    check(batch, target.transpose(0, 1), L, scale, CAUSAL)


APPEND = [  # (lengths, hq, hkv, d, page, rot)
    ([(1, 1)], 0, 1, 64, 16, 64),
    ([(1, 300), (1, 17), (1, 16), (1, 1)], 8, 2, 128, 16, 128),
    ([(5, 21), (0, 7), (33, 33), (1, 640)], 6, 3, 64, 32, 16),
    ([(700, 1200), (64, 64), (129, 1000)], 4, 4, 128, 64, 64),
    ([(40, 90)] * 40, 2, 1, 128, 1024, 128),
    ([(19, 50)], 3, 2, 80, 16, 48),
    ([(3, 9)] * 1100, 1, 1, 64, 16, 32),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("index", range(len(APPEND)))
def test_append(index, interleaved):
    import torch
    lengths, hq, hkv, d, page, rot = APPEND[index]
    dtype = torch.bfloat16 if (index + interleaved) % 2 else torch.float16
    layout = "bnhd" if index % 2 else "bhnd"
    batch = make_batch(lengths, max(hq, 1), hkv, d, page, dtype, layout, seed=index,
                       behind=index % 3, fill=3.0)
    T = batch.q.shape[0]
    used = sum(n for n, _ in lengths)
    kv = torch.randn(T, 2 * hkv, d, device="cuda").to(dtype)
    k, v = kv[:, :hkv], kv[:, hkv:]
    freqs = freqs_of(rot)
    want_k, want_v = batch.k_pages.clone(), batch.v_pages.clone()
    q_out = torch.full_like(batch.q, 7.0)
    got = fa.paged_append(k, v, *batch.cache, q=batch.q if hq else None, freqs=freqs,
                          magnitude=1.25, interleaved=interleaved, page_layout=layout,
                          q_out=q_out if hq else None)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    pos = torch.cat([torch.arange(k_ - n, k_) for n, k_ in lengths]).cuda()
    rk, bk = plain(k[:used], pos[:, None], freqs, 1.25, interleaved)
    owner = torch.repeat_interleave(torch.arange(len(lengths)),
                                    torch.tensor([n for n, _ in lengths])).cuda()
    pages = batch.page_table[owner, pos // page].long()

    def rows(pool):
        return (pool if layout == "bnhd" else pool.transpose(1, 2))[pages, pos % page]
    close(rows(batch.k_pages), (rk, bk))
    assert torch.equal(rows(batch.v_pages), v[:used])
    for pool, want in ((batch.k_pages, want_k), (batch.v_pages, want_v)):  # nothing else moved
        view, old = (p if layout == "bnhd" else p.transpose(1, 2) for p in (pool, want))
        view[pages, pos % page] = old[pages, pos % page]
        assert torch.equal(pool, want)
    if hq:
        close(got[:used], plain(batch.q[:used], pos[:, None], freqs, 1.25, interleaved))
        assert (got[used:] == 7).all()
    else:
        assert got is None


def test_append_without_rotation_and_with_other_positions():
    import torch
    batch = make_batch([(6, 20), (3, 3)], 2, 2, 64, 16, torch.bfloat16, fill=0.0)
    k, v = (torch.randn(9, 2, 64, device="cuda").bfloat16() for _ in range(2))
    assert fa.paged_append(k, v, *batch.cache) is None
    pages = batch.page_table[[0] * 6 + [1] * 3, [0, 0, 1, 1, 1, 1, 0, 0, 0]].long()
    slots = [14, 15, 0, 1, 2, 3, 0, 1, 2]
    assert torch.equal(batch.k_pages[pages, slots], k)
    assert torch.equal(batch.v_pages[pages, slots], v)
    freqs = freqs_of(64)
    pos = torch.randint(0, 100000, (9,), dtype=torch.int32, device="cuda")
    q = batch.q.clone()
    got = fa.paged_append(k, v, *batch.cache, q=q, freqs=freqs, positions=pos, q_out=q)
    assert got is q
    close(q, plain(batch.q, pos[:, None], freqs, 1.0, False))
    close(batch.k_pages[pages, slots], plain(k, pos[:, None], freqs, 1.0, False))


def test_bad_pages_and_lengths():
    """A page index outside the pool reads as zeros and is not written, a sequence with
    inconsistent lengths is left out; the others are served, and the status says so."""
    import torch
    for n, page in ((1, 16), (1, 256), (80, 16), (80, 256)):
        batch = make_batch([(n, 600), (n, 300), (n, 200)], 4, 2, 128, page, torch.bfloat16,
                           seed=2, fill=0.0)
        for bad in (-1, -2**31, 2**31 - 1, batch.k_pages.shape[0]):
            table = batch.page_table.clone()
            table[1, 0] = bad
            out = torch.full_like(batch.q, 7.0)
            o, L = fa.paged_attention(batch.q, batch.k_pages, batch.v_pages, table, batch.cu_q,
                                      batch.seq_k, max_q=n, out=out)
            assert fa.device_status() == fa.FA_ERR_INVALID
            assert fa.device_status() == fa.FA_OK
            k1, v1 = batch.keys[1].clone(), batch.values[1].clone()
            batch.keys[1][:page], batch.values[1][:page] = 0, 0
            check(batch, o, L, 128 ** -0.5, CAUSAL)
            batch.keys[1], batch.values[1] = k1, v1
        seq_k = batch.seq_k.clone()
        seq_k[1] = 2**31 - 1
        out = torch.full_like(batch.q, 7.0)
        o, L = fa.paged_attention(batch.q, batch.k_pages, batch.v_pages, batch.page_table,
                                  batch.cu_q, seq_k, max_q=n, out=out)
        assert fa.device_status() == fa.FA_ERR_INVALID
        assert (o[n:2 * n] == 7).all()
        # the split of the others' keys depends on the whole batch, and so do their roundings:
        # held to the definition, with the left-out rows from a call that serves them
        want, wantL = fa.paged_attention(batch.q, *batch.cache, max_q=n)
        o[n:2 * n], L[:, n:2 * n] = want[n:2 * n], wantL[:, n:2 * n]
        check(batch, o, L, 128 ** -0.5, CAUSAL)
        k, v = (torch.ones(3 * n, 2, 128, device="cuda").bfloat16() for _ in range(2))
        before = batch.k_pages.clone()
        table = batch.page_table.clone()
        table[0, (600 - 1) // page] = batch.k_pages.shape[0]
        seq_k = torch.tensor([600, -5, n - 1], dtype=torch.int32, device="cuda")
        fa.paged_append(k, v, batch.k_pages, batch.v_pages, table, batch.cu_q, seq_k)
        assert fa.device_status() == fa.FA_ERR_INVALID
        if n == 1:
            assert torch.equal(batch.k_pages, before)


def test_chunks_then_steps_equal_the_whole():
    """A prompt appended and attended in chunks, then token by token, gives what rotating the
    whole and forward() gives -- through one captured step whose lengths and inputs move on."""
    import torch
    torch.manual_seed(8)
    total, chunks, hq, hkv, d, page = 200, [70, 1, 64, 60], 6, 3, 64, 16
    q, k, v = (torch.randn(total, h, d, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    freqs = fa.rope_frequencies(32, method="linear", factor=2.0)
    kp, vp = (torch.full((20, page, hkv, d), float("nan"), device="cuda").bfloat16()
              for _ in range(2))
    table = torch.randperm(20, device="cuda").int()[None, :13].contiguous()
    got_o, got_l, at = [], [], 0
    for n in chunks:
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        sk = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        rows = slice(at, at + n)
        qr = fa.paged_append(k[rows], v[rows], kp, vp, table, cu, sk, q=q[rows], freqs=freqs)
        o, L = fa.paged_attention(qr, kp, vp, table, cu, sk, max_q=n)
        got_o.append(o), got_l.append(L)
        at += n
    # the last tokens through a graph
    tok = [x[:1].clone() for x in (q, k, v)]
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    sk = torch.tensor([at + 1], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr = fa.paged_append(tok[1], tok[2], kp, vp, table, cu, sk, q=tok[0], freqs=freqs)
        o, L = fa.paged_attention(qr, kp, vp, table, cu, sk, max_q=1)
    while at < total:
        for x, y in zip(tok, (q, k, v)):
            x.copy_(y[at:at + 1])
        sk.fill_(at + 1)
        graph.replay()
        got_o.append(o.clone()), got_l.append(L.clone())
        at += 1
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    qr, kr = fa.rope(q[None], k[None], freqs, layout="bnhd")
    rep = [x.repeat_interleave(hq // hkv, 2).contiguous() for x in (kr, v[None])]
    ro, rl, _ = fa.forward(qr, *rep, causal=True, layout="bnhd", residual=False)
    assert (torch.cat(got_o).float() - ro[0].float()).abs().max() <= 4e-2
    assert (torch.cat(got_l, 1) - rl[0]).abs().max() <= 2e-3


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("n", [1, 5, 300])
def test_pages_before_the_window_may_be_gone(n, page):
    """Pages whose keys all lie before every new token's window are not looked up: their
    table entries may point nowhere, and the pages may hold other sequences' keys."""
    import torch
    left = 333
    batch = make_batch([(n, 3000), (n, 1111), (n, n + 1)], 8, 2, 128, page, torch.bfloat16,
                       seed=n)
    want = attend(batch, (left, 0), 128)
    for b, (_, k) in enumerate(batch.lengths):
        gone = max(0, k - n - left) // page
        batch.page_table[b, :gone] = -1
    got = attend(batch, (left, 0), 128)  # its status is FA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n", [1, 40])
def test_lengths_that_do_not_fit(n):
    """A sequence with more new tokens than max_q, and rows that cu_q gives to nobody."""
    import torch
    d = 128
    batch = make_batch([(n, 300), (n + 2, 200), (n, 100)], 4, 2, d, 64, torch.bfloat16, seed=5)
    want, wantL = fa.paged_attention(batch.q, *batch.cache, max_q=n + 2)
    out = torch.full_like(batch.q, 7.0)
    o, L = fa.paged_attention(batch.q, *batch.cache, max_q=n, out=out)
    assert fa.device_status() == fa.FA_ERR_INVALID
    rows = slice(n, 2 * n + 2)
    assert (o[rows] == 7).all()
    o[rows], L[:, rows] = want[rows], wantL[:, rows]
    check(batch, o, L, d ** -0.5, CAUSAL)
    for cu in ([0, n, n - 1, 3 * n + 2], [0, n, 2 * n + 2, 3 * n + 3], [-1, n, 2 * n + 2, 3 * n + 2]):
        cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        fa.paged_attention(batch.q, batch.k_pages, batch.v_pages, batch.page_table, cu_q,
                           batch.seq_k)
        assert fa.device_status() == fa.FA_ERR_INVALID
        k = torch.zeros(3 * n + 2, 2, d, device="cuda").bfloat16()
        pools = [p.clone() for p in (batch.k_pages, batch.v_pages)]
        fa.paged_append(k, k, *pools, batch.page_table, cu_q, batch.seq_k)
        assert fa.device_status() == fa.FA_ERR_INVALID
    # rows before the first sequence and between none: only the named ones are written
    cu_q = torch.tensor([n, n, 2 * n + 2, 2 * n + 2], dtype=torch.int32, device="cuda")
    out = torch.full_like(batch.q, 7.0)
    o, L = fa.paged_attention(batch.q, batch.k_pages, batch.v_pages, batch.page_table, cu_q,
                              batch.seq_k, out=out)
    assert fa.device_status() == fa.FA_OK
    assert (o[:n] == 7).all() and (o[2 * n + 2:] == 7).all()
    ref = reference(batch, d ** -0.5, CAUSAL)[1]
    assert ((o[rows].double() - ref[0]).abs() <= ref[2]).all()


@pytest.mark.parametrize("n", [1, 50])
def test_nan_reaches_its_rows_only(n):
    """A NaN query, and a NaN in a key that only later tokens see: NaN where the definition
    has it, the other rows as they are."""
    import torch
    d = 64
    batch = make_batch([(n, 3000), (n, 700)], 4, 2, d, 64, torch.bfloat16, seed=7)
    batch.q[n, 1, 3] = float("nan")
    o, L = fa.paged_attention(batch.q, *batch.cache, max_q=n)
    assert fa.device_status() == fa.FA_OK
    bad = torch.zeros(2 * n, 4, dtype=torch.bool, device="cuda")
    bad[n, 1] = True
    assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(L.isnan().T, bad)
    batch.q[n, 1, 3] = 0.5
    if n > 1:
        at = 3000 - n + 20  # the key of new token 20
        page = batch.page_table[0, at // 64].long()
        old = batch.k_pages[page, at % 64, 0].clone()
        batch.k_pages[page, at % 64, 0] = float("nan")
        o, L = fa.paged_attention(batch.q, *batch.cache, max_q=n)
        bad[:] = False
        bad[20:n, :2] = True
        assert torch.equal(o.isnan().any(-1), bad) and torch.equal(L.isnan().T, bad)
        batch.k_pages[page, at % 64, 0] = old


@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_rows_of_one_key_tile(d):
    """Rows of a single query tile, whose key tiles are dealt out in turn, that see keys of
    one tile only, the second of three: a NaN query there is NaN, its neighbours are not."""
    import torch
    batch = make_batch([(100, 400)], 1, 1, d, 64, torch.bfloat16, seed=8)
    for row in (10, 50, 90):  # keys 260 .. 310, 300 .. 350 (one tile), 340 .. 390 (two)
        q = batch.q.clone()
        q[row, 0, 5] = float("nan")
        o, L = fa.paged_attention(q, *batch.cache, max_q=100, window=(50, 0))
        assert fa.device_status() == fa.FA_OK
        bad = torch.zeros(100, 1, dtype=torch.bool, device="cuda")
        bad[row] = True
        assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
        assert torch.equal(L.isnan().T, bad)


def test_a_pool_past_32_bit_offsets():
    """Pages whose elements lie beyond 2^32: written and read in place."""
    import torch
    if torch.cuda.mem_get_info()[0] < 30 * 2**30:
        pytest.skip("needs 20 GB of device memory")
    page, hkv, d = 256, 16, 128
    count = 2 * 2**32 // (2 * page * hkv * d) + 3
    pool = torch.empty((count, 2, page, hkv, d), device="cuda", dtype=torch.bfloat16)
    assert pool[-1, 1].storage_offset() > 2**32
    kp, vp = pool[:, 0], pool[:, 1]
    table = torch.tensor([[count - 1, 0, count - 2]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(600, hkv, d, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(600, 2 * hkv, d, device="cuda").bfloat16()
    cu = torch.tensor([0, 600], dtype=torch.int32, device="cuda")
    sk = torch.tensor([600], dtype=torch.int32, device="cuda")
    fa.paged_append(k, v, kp, vp, table, cu, sk)
    assert torch.equal(kp[count - 1], k[:256]) and torch.equal(vp[count - 2, :88], v[512:])
    for rows in (600, 1):
        q_ = q[600 - rows:]
        cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        o, L = fa.paged_attention(q_, kp, vp, table, cu, sk, max_q=rows)
        assert fa.device_status() == fa.FA_OK
        whole = make_batch([(rows, 600)], 2 * hkv, hkv, d, 256, torch.bfloat16)
        whole.q, whole.keys, whole.values = q_, [k.cpu()], [v.cpu()]
        check(whole, o, L, d ** -0.5, CAUSAL)


def test_two_graphs_share_a_workspace():
    """Replayed in turn, each gives what an eager call gives: a call leaves nothing in the
    workspace that the next one reads."""
    import torch
    batches = [make_batch([(1, 5000), (1, 40)], 8, 2, 128, 16, torch.bfloat16, seed=1),
               make_batch([(90, 3000)], 8, 2, 128, 64, torch.bfloat16, seed=2)]
    wants = [fa.paged_attention(b.q, *b.cache, max_q=b.max_q) for b in batches]
    size = max(fa.paged_workspace_size(b.q.shape[0], b.max_q, 8, 2, 128) for b in batches)
    workspace = torch.full((size,), 255, device="cuda", dtype=torch.uint8)
    graphs, outs = [], []
    for b in batches:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fa.paged_attention(b.q, *b.cache, max_q=b.max_q, workspace=workspace))
        graphs.append(graph)
    for _ in range(4):
        for graph, out, want in zip(graphs, outs, wants):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_long_chain_of_dependent_calls():
    """Rotated appends and attention back to back, each reading what the one before wrote
    (launches overlap; reads must not), against the same calls one by one."""
    import torch
    torch.manual_seed(2)
    freqs = freqs_of(64)

    def chain(wait):
        gen = torch.Generator("cuda").manual_seed(5)
        kp, vp = (torch.zeros(70, 16, 2, 64, device="cuda").bfloat16() for _ in range(2))
        table = torch.arange(70, device="cuda", dtype=torch.int32).view(2, 35)
        x = torch.randn(2, 8, 64, device="cuda", generator=gen).bfloat16()
        cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        seen = []
        for i in range(1, 300):
            sk = torch.full((2,), i, dtype=torch.int32, device="cuda")
            q = fa.paged_append(x[:, :2], x[:, 2:4], kp, vp, table, cu, sk, q=x, freqs=freqs)
            if wait:
                torch.cuda.synchronize()
            o, _ = fa.paged_attention(q, kp, vp, table, cu, sk, max_q=1)
            if wait:
                torch.cuda.synchronize()
            x, _ = fa.rope(o[None], None, freqs, layout="bnhd")
            x = x[0]
            seen.append(x)
        return torch.stack(seen), kp, vp
    assert all(torch.equal(a, b) for a, b in zip(chain(False), chain(True)))


def test_attention_on_other_streams_at_once():
    """Two calls that may overlap, each with its own workspace, on streams of their own."""
    import torch
    batches = [make_batch([(1, 4000), (1, 900)], 8, 2, 128, 16, torch.bfloat16, seed=1),
               make_batch([(200, 2000)], 8, 2, 128, 64, torch.bfloat16, seed=2)]
    wants = [attend(b, CAUSAL, 128) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [fa.paged_attention(b.q, *b.cache, max_q=b.max_q, page_layout=b.layout, stream=s)
               for b, s in zip(batches, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, wants):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_refusals():
    import torch
    batch = make_batch([(1, 40), (1, 20)], 4, 2, 64, 16, torch.bfloat16, fill=0.0)
    k = v = torch.zeros(2, 2, 64, device="cuda").bfloat16()

    def cache(**kw):
        c = dict(k_pages=batch.k_pages, v_pages=batch.v_pages, page_table=batch.page_table,
                 cu_q=batch.cu_q, seq_k=batch.seq_k)
        c.update(kw)
        return c
    for kw in (dict(k_pages=batch.k_pages.half()), dict(v_pages=batch.v_pages[1:]),
               dict(page_table=batch.page_table.long()), dict(page_table=batch.page_table[:1]),
               dict(cu_q=batch.cu_q[:2]), dict(seq_k=batch.seq_k.cpu()),
               dict(k_pages=batch.k_pages[..., :32], v_pages=batch.v_pages[..., :32]),
               dict(k_pages=batch.k_pages[:, :12], v_pages=batch.v_pages[:, :12])):
        with pytest.raises(fa.FaError):
            fa.paged_attention(batch.q, **cache(**kw), max_q=1)
        with pytest.raises(fa.FaError):
            fa.paged_append(k, v, **cache(**kw))
    for kw in (dict(q=batch.q[:, :3]), dict(q=batch.q.float()), dict(scale=0.0),
               dict(scale=float("inf")), dict(page_layout="x"), dict(max_q=-1),
               dict(lse=torch.zeros(4, 3, device="cuda")), dict(out=batch.q[:1])):
        with pytest.raises(fa.FaError):
            fa.paged_attention(**{**cache(), "q": batch.q, "max_q": 1, **kw})
    for kw in (dict(v=v[:1]), dict(v=v.half()), dict(q=batch.q), dict(k=k[:, :1], v=v[:, :1]),
               dict(freqs=freqs_of(128)), dict(positions=batch.cu_q)):
        with pytest.raises(fa.FaError):
            fa.paged_append(**{**cache(), "k": k, "v": v, **kw})
    none = batch.q[:0]
    o, L = fa.paged_attention(none, **cache(), max_q=1)
    assert o.shape == none.shape and L.shape == (4, 0)
