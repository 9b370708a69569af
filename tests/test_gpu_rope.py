"""fa.rope and fa.rope_backward against the rotation in 64 bits: both pair layouts, part of
the head, far positions, strided and in-place tensors, one token and long inputs; the
gradient against the formula and against differences."""

import math

import pytest

from exact_io_aware_69_b200 import fa

from paged_cases import half_step

pytestmark = pytest.mark.gpu


def plain(x, positions, freqs, magnitude, interleaved, inverse=False):
    """(rotated x in 64 bits, its error bound); positions broadcast against x[..., 0]."""
    import torch
    r = 2 * freqs.shape[0]
    a = positions.double()[..., None] * freqs
    c, s = a.cos() * magnitude, a.sin() * magnitude * (-1 if inverse else 1)
    y = x.double().clone()
    x0, x1 = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    x0, x1 = x0.clone(), x1.clone()
    span = (x0.abs() + x1.abs()) * magnitude * 1e-6
    bound = torch.zeros_like(y)
    for part, value in ((0, x0 * c - x1 * s), (1, x1 * c + x0 * s)):
        index = slice(part, r, 2) if interleaved else slice(part * r // 2, (part + 1) * r // 2)
        y[..., index] = value
        bound[..., index] = half_step(x.dtype) * value.abs() + span + 2.0 ** -25
    return y, bound


def close(got, want):
    ref, bound = want
    diff = (got.double() - ref).abs()
    assert (diff <= bound).all(), f"off by {(diff / bound.clamp(min=1e-30)).max().item():.2f}"


def freqs_of(rot, method="none"):
    return fa.rope_frequencies(rot, method=method, factor=4.0, train_len=2048)


@pytest.mark.parametrize("B,N,hq,hk,d,rot", [
    (1, 1, 1, 1, 64, 64), (2, 1, 32, 8, 128, 128), (1, 5, 3, 1, 128, 32), (3, 333, 7, 7, 64, 16),
    (1, 4099, 8, 2, 128, 128), (2, 700, 5, 1, 80, 80), (1, 37, 2, 2, 256, 64),
    (1, 9, 3, 2, 1024, 1024), (1, 1300, 40, 8, 128, 96),
])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_rope_matches_the_plain_rotation(B, N, hq, hk, d, rot, interleaved, layout):
    import torch
    torch.manual_seed(rot + N)
    dtype = torch.float16 if (N + d + interleaved) % 2 else torch.bfloat16
    shapes = [(B, h, N, d) if layout == "bhnd" else (B, N, h, d) for h in (hq, hk)]
    q, k = (torch.randn(s, device="cuda").to(dtype) for s in shapes)
    freqs = freqs_of(rot, "ramp")
    pos = torch.randint(0, 2_000_000, (B, N), device="cuda", dtype=torch.int32)
    at = pos[:, None] if layout == "bhnd" else pos[:, :, None]
    for call, inverse in ((fa.rope, False), (fa.rope_backward, True)):
        yq, yk = call(q, k, freqs, positions=pos, magnitude=1.25, interleaved=interleaved,
                      layout=layout)
        close(yq, plain(q, at, freqs, 1.25, interleaved, inverse))
        close(yk, plain(k, at, freqs, 1.25, interleaved, inverse))
    assert fa.device_status() == fa.FA_OK


def test_rope_positions_forms_and_only_q():
    import torch
    q = torch.randn(2, 3, 50, 64, device="cuda").bfloat16()
    freqs = freqs_of(64)
    row = torch.arange(50, device="cuda", dtype=torch.int32)
    want = plain(q, row, freqs, 1.0, False)
    for positions in (None, row, row.expand(2, 50), torch.stack((row, row))):
        y, none = fa.rope(q, None, freqs, positions=positions)
        assert none is None
        close(y, want)
    back = torch.arange(0, -50, -1, device="cuda", dtype=torch.int32)  # negative: turned back
    close(fa.rope(q, None, freqs, positions=back)[0], plain(q, back, freqs, 1.0, False))
    far = torch.full((50,), 2**31 - 1, device="cuda", dtype=torch.int32)
    # at 2^31 the 64-bit angle itself is rounded to 2^-22 rad, here and in the reference
    y, bound = plain(q, far, freqs, 1.0, False)
    close(fa.rope(q, None, freqs, positions=far)[0], (y, bound + 2.0**-21 * 8))


@pytest.mark.parametrize("method", ["none", "linear", "base", "ramp"])
def test_frequencies(method):
    import torch
    f = fa.rope_frequencies(64, base=500000.0, method=method, factor=8.0, train_len=8192).cpu()
    g = fa.rope_frequencies(64, base=500000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    i = torch.arange(32, dtype=torch.float64)
    assert torch.allclose(g, 500000.0 ** (-i / 32), rtol=1e-14)
    ratio = g / f
    if method == "none":
        assert torch.equal(f, g)
    elif method == "linear":
        assert torch.allclose(ratio, torch.full_like(ratio, 8.0), rtol=1e-14)
    elif method == "base":
        assert ratio[0] == 1 and math.isclose(ratio[-1], 8.0, rel_tol=1e-12)
    else:
        turns = 8192 * g / (2 * math.pi)
        assert (ratio[turns >= 4] == 1).all() and torch.allclose(
            ratio[turns <= 1], torch.full_like(ratio[turns <= 1], 8.0), rtol=1e-14)
        assert (ratio.diff() >= 0).all()


def test_rope_in_place_and_strided():
    """q and k as views of one projection's output, rotated in place: V keeps its values."""
    import torch
    torch.manual_seed(1)
    B, N, hq, hk, d = 2, 77, 6, 2, 64
    qkv = torch.randn(B, N, hq + 2 * hk, d, device="cuda").half()
    before = qkv.clone()
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    freqs = freqs_of(32)
    row = torch.arange(N, device="cuda", dtype=torch.int32)
    wants = [plain(x, row[:, None], freqs, 0.5, True) for x in (q, k)]
    yq, yk = fa.rope(q, k, freqs, magnitude=0.5, interleaved=True, layout="bnhd", q_out=q,
                     k_out=k)
    assert yq.data_ptr() == q.data_ptr()
    for got, want in zip((yq, yk), wants):
        close(got, want)
    assert torch.equal(qkv[:, :, hq + hk:], before[:, :, hq + hk:])
    assert torch.equal(qkv[:, :, :hq, 32:], before[:, :, :hq, 32:])


def test_gradient_against_differences():
    """sum(w * rope(x)) differs by e * (rope_backward(w))_i when x_i moves by e. The rotation
    is linear, so the difference of two 64-bit sums is off only by the roundings of the two
    outputs that x_i reaches, and the gradient by its own."""
    import torch
    torch.manual_seed(3)
    x = torch.randn(1, 2, 5, 64, device="cuda").half()
    w = torch.randn_like(x)
    freqs = freqs_of(32)
    kw = dict(magnitude=1.5, positions=torch.tensor([0, 1, 7, 900, 65537], dtype=torch.int32,
                                                    device="cuda"))
    grad = fa.rope_backward(w, None, freqs, **kw)[0].double()
    u = half_step(torch.float16)
    base = fa.rope(x, None, freqs, **kw)[0].double()
    for index in ((0, 0, 0, 0), (0, 1, 2, 17), (0, 0, 3, 31), (0, 1, 4, 5), (0, 0, 4, 60)):
        moved = x.clone()
        moved[index] += 4.0
        step = (moved[index] - x[index]).double()
        y = fa.rope(moved, None, freqs, **kw)[0].double()
        got = ((y - base) * w.double()).sum() / step
        head = (0, index[1], index[2])
        slack = (u * (y[head].abs() + base[head].abs()) * w[head].double().abs()).sum() / step \
            + u * grad[index].abs() + 1e-5
        assert abs(got - grad[index]) <= slack


def test_rope_on_another_stream_and_captured():
    import torch
    torch.manual_seed(5)
    q = torch.randn(1, 64, 8, 128, device="cuda").bfloat16()
    k = torch.randn(1, 64, 2, 128, device="cuda").bfloat16()
    freqs = freqs_of(128)
    row = torch.arange(64, device="cuda", dtype=torch.int32)
    want = fa.rope(q, k, freqs, positions=row, layout="bnhd")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.rope(q, k, freqs, positions=row, layout="bnhd", stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.rope(q, k, freqs, positions=row, layout="bnhd")
    row += 1000
    graph.replay()
    torch.cuda.synchronize()
    want = fa.rope(q, k, freqs, positions=row, layout="bnhd")
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_rope_refuses():
    import torch
    q = torch.randn(1, 2, 8, 64, device="cuda").bfloat16()
    freqs = freqs_of(64)
    bad = [dict(q=q.float()), dict(q=q[0]), dict(k=q.half()), dict(k=q[:, :, :4]),
           dict(freqs=freqs.float()), dict(freqs=freqs[::2]), dict(freqs=freqs.cpu()),
           dict(freqs=freqs_of(128)), dict(freqs=freqs[:4].contiguous()),
           dict(positions=torch.arange(8, device="cuda")),
           dict(positions=torch.zeros(9, dtype=torch.int32, device="cuda")),
           dict(layout="nbhd"), dict(q_out=q[:, :, :, ::2]), dict(q_out=q.half()),
           dict(q=torch.randn(1, 2, 8, 72, device="cuda").bfloat16()[..., 4:68]),
           dict(q=q.transpose(2, 3)), dict(magnitude=float("nan"))]
    for kw in bad:
        args = dict(q=q, k=None, freqs=freqs)
        args.update(kw)
        with pytest.raises(fa.FaError):
            fa.rope(**args)
    empty = torch.empty(0, 2, 8, 64, device="cuda", dtype=torch.bfloat16)
    assert fa.rope(empty, None, freqs)[0].shape == empty.shape
