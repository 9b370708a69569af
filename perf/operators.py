"""Rotary positions, the paged key/value cache and attention over it: the cases that are measured.

Three operators that go together. `rope` turns pairs of columns of Q and K by an angle
proportional to the token's position (and `rope_grad` turns a gradient back), `append`
writes the rotated keys and the values of new tokens into the pages of a cache, and
`attend` is exact attention of those tokens over everything their sequence has cached.

Tokens of a ragged batch are packed: q is [T, Hq, d], sequence b owns the rows
cu_q[b] .. cu_q[b + 1] - 1, has seq_k[b] cached keys (its new tokens included) and finds
key j in row j % page of page page_table[b, j // page]. Query i of a sequence with n new
tokens sees key j iff i + off - left <= j <= i + off + right with off = seq_k - n
(negative edge: unbounded); Hq = group * Hkv and query head h reads key head h // group.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # Training at the repository's headline shape (2 x 8192 tokens, 32 heads, d 128)
        # with grouped keys: Q and K rotated before the forward.
        dict(name="rope_train", op="rope", batch=2, n=8192, hq=32, hkv=8, d=128, rot=128,
             dtype="bf16", interleaved=False, layout="bnhd", first=0, method="none", factor=1.0),
        # The gradients of the same rotation after the backward: part of the head, pairs
        # side by side, an odd length, far positions of a context stretched eight times.
        dict(name="rope_grad", op="rope_grad", batch=4, n=2047, hq=16, hkv=16, d=64, rot=32,
             dtype="fp16", interleaved=True, layout="bhnd", first=100000, method="ramp",
             factor=8.0),
        # One new token for each of four sequences: nothing but latency.
        dict(name="rope_token", op="rope", batch=4, n=1, hq=32, hkv=8, d=128, rot=128,
             dtype="bf16", interleaved=False, layout="bnhd", first=4097, method="base",
             factor=4.0),
        # A serving step: 64 sequences add one token each, small pages.
        dict(name="append_step", op="append", batch=64, singles=64, q_lo=1, q_hi=1, c_lo=100,
             c_hi=900, hq=32, hkv=8, d=128, rot=128, dtype="bf16", interleaved=False, page=16,
             layout="bnhd", method="linear", factor=2.0, mix=1),
        # Prompts written into the cache in ragged chunks, all heads their own keys.
        dict(name="append_chunk", op="append", batch=6, singles=1, q_lo=700, q_hi=3001, c_lo=1,
             c_hi=2000, hq=16, hkv=16, d=64, rot=64, dtype="fp16", interleaved=True, page=64,
             layout="bhnd", method="ramp", factor=8.0, mix=2),
        # One user, one token, a thousand keys: the latency of a step.
        dict(name="attend_token", op="attend", batch=1, singles=1, q_lo=1, q_hi=1, c_lo=1000,
             c_hi=1000, hq=32, hkv=8, d=128, dtype="bf16", page=16, layout="bnhd", left=-1,
             right=0, mix=3),
        # A full serving batch: one token each over contexts of very different lengths.
        dict(name="attend_step", op="attend", batch=64, singles=64, q_lo=1, q_hi=1, c_lo=300,
             c_hi=16384, hq=32, hkv=8, d=128, dtype="bf16", page=16, layout="bnhd", left=-1,
             right=0, mix=4),
        # Two long contexts (the repository's decode length), few sequences to share out.
        dict(name="attend_step_long", op="attend", batch=2, singles=2, q_lo=1, q_hi=1,
             c_lo=65000, c_hi=65536, hq=16, hkv=4, d=64, dtype="fp16", page=64, layout="bhnd",
             left=-1, right=0, mix=5),
        # Five drafted tokens per sequence checked at once.
        dict(name="attend_draft", op="attend", batch=24, singles=0, q_lo=2, q_hi=5, c_lo=500,
             c_hi=8000, hq=32, hkv=8, d=128, dtype="fp16", page=32, layout="bnhd", left=-1,
             right=0, mix=6),
        # A prompt's next 2048 tokens over what was cached before.
        dict(name="attend_chunk", op="attend", batch=1, singles=0, q_lo=2048, q_hi=2048,
             c_lo=14000, c_hi=14336, hq=32, hkv=8, d=128, dtype="bf16", page=128, layout="bnhd",
             left=-1, right=0, mix=7),
        # Prompts and single tokens in one batch, odd sizes, a sliding window, d 64.
        dict(name="attend_mixed", op="attend", batch=20, singles=13, q_lo=100, q_hi=1999,
             c_lo=1, c_hi=7000, hq=16, hkv=16, d=64, dtype="bf16", page=64, layout="bhnd",
             left=2500, right=0, mix=8),
        # The largest: 4096 tokens over 65536 keys.
        dict(name="attend_long", op="attend", batch=1, singles=0, q_lo=4096, q_hi=4096,
             c_lo=61440, c_hi=61440, hq=32, hkv=8, d=128, dtype="bf16", page=64, layout="bnhd",
             left=-1, right=0, mix=9),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    most = _cost(listed()[-1])
    while True:
        op = rng.choice(["rope", "rope_grad", "append", "attend", "attend", "attend"])
        d = rng.choice([64, 128])
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        case = dict(op=op, hq=group * hkv, hkv=hkv, d=d, dtype=rng.choice(["bf16", "fp16"]),
                    layout=rng.choice(["bnhd", "bhnd"]))
        if op != "attend":
            case.update(rot=rng.choice([d, d, d // 2, d // 4]),
                        interleaved=rng.random() < 0.5,
                        method=rng.choice(["none", "linear", "base", "ramp"]),
                        factor=rng.choice([2.0, 3.5, 8.0]))
        if op in ("rope", "rope_grad"):
            case.update(batch=_spread(rng, 1, 16), n=_spread(rng, 1, 16384),
                        first=rng.choice([0, _spread(rng, 1, 1000000)]))
        else:
            batch = _spread(rng, 1, 96)
            singles = rng.choice([0, batch, rng.randint(0, batch)])
            q_hi = rng.choice([_spread(rng, 2, 16), _spread(rng, 17, 4096)])
            c_hi = _spread(rng, 2, 65536)
            case.update(batch=batch, singles=singles, q_lo=_spread(rng, 1, q_hi), q_hi=q_hi,
                        c_lo=_spread(rng, 1, c_hi), c_hi=c_hi,
                        page=rng.choice([16, 32, 64, 128, 256]), mix=rng.randint(0, 10**6))
        if op == "attend":
            case.update(left=rng.choice([-1, -1, -1, _spread(rng, 1, 20000)]),
                        right=rng.choice([0, 0, 0, -1]))
        if _cost(case) <= most and _rows(case) <= 2**21 // hkv:
            return case


def _lengths(case):
    """(new tokens, cached keys after them) of every sequence."""
    rng = random.Random(case["mix"])
    out = []
    for b in range(case["batch"]):
        n = 1 if b < case["singles"] else _spread(rng, case["q_lo"], case["q_hi"])
        out.append((n, n + _spread(rng, case["c_lo"], case["c_hi"]) - 1))
    rng.shuffle(out)
    return out


def _rows(case):
    """Key rows that the case keeps in memory, per head."""
    if case["op"] in ("rope", "rope_grad"):
        return case["batch"] * case["n"]
    return sum(-(-k // case["page"]) * case["page"] for _, k in _lengths(case))


def _pairs(case):
    """(query, key) pairs inside the mask, per head, and keys that some query sees."""
    pairs = seen = 0
    for n, k in _lengths(case):
        off = k - n
        left = k if case["left"] < 0 else case["left"]
        right = k if case["right"] < 0 else case["right"]
        first = max(0, off - left)
        seen += max(0, min(k - 1, n - 1 + off + right) - first + 1)
        # sum over i of min(k - 1, i + off + right) - max(0, i + off - left) + 1
        hi = [min(k - 1, i + off + right) for i in (0, n - 1)]
        if hi[0] == hi[1] == k - 1:
            top = n * (k - 1)
        elif off + right + n - 1 <= k - 1:
            top = n * (hi[0] + hi[1]) // 2
        else:
            cut = k - 1 - off - right
            top = (cut + 1) * (off + right) + cut * (cut + 1) // 2 + (n - cut - 1) * (k - 1)
        low = max(0, min(n, left - off + 1))  # rows whose left edge is key 0
        bottom = sum((off - left + low, off - left + n - 1)) * (n - low) // 2
        pairs += top - bottom + n
    return pairs, seen


def work(case):
    e = 2  # bytes of a 16-bit value
    if case["op"] in ("rope", "rope_grad"):
        values = case["batch"] * case["n"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 2 * e * values + 4 * case["rot"], "flops": 3 * values}
    tokens = sum(n for n, _ in _lengths(case))
    if case["op"] == "append":
        values = tokens * (case["hq"] + 2 * case["hkv"]) * case["d"]
        return {"bytes": 2 * e * values, "flops": 3 * values}
    pairs, seen = _pairs(case)
    moved = seen * case["hkv"] * 2 + tokens * case["hq"] * 2
    return {"bytes": moved * case["d"] * e + 4 * tokens * case["hq"],
            "flops": 4 * pairs * case["hq"] * case["d"]}


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1e15


def _frequencies(case):
    """Angle per position of each pair, in 64 bits."""
    r = case["rot"]
    base, s = 10000.0, case["factor"]
    if case["method"] == "base":
        base *= s ** (r / (r - 2))
    freq = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["method"] == "linear":
        freq = freq / s
    if case["method"] == "ramp":  # fast pairs as they are, slow ones stretched
        turns = 4096 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / s)
    return freq.cuda()


def _random(gen, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * gain).to(dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    state = dict(case=case)
    if case["op"] != "attend":
        state["freqs"] = _frequencies(case)
        state["magnitude"] = 1.0 if case["method"] != "ramp" else 0.1 * math.log(case["factor"]) + 1
    if case["op"] in ("rope", "rope_grad"):
        b, n = case["batch"], case["n"]
        for name, h in (("q", hq), ("k", hkv)):
            shape = (b, n, h, d) if case["layout"] == "bnhd" else (b, h, n, d)
            state[name] = _random(gen, shape, dtype)
        # every sequence of the batch at its own place
        start = case["first"] + 17 * torch.arange(b, device="cuda")
        state["positions"] = (start[:, None] + torch.arange(n, device="cuda")).int()
        return state

    lengths = _lengths(case)
    state["lengths"] = lengths
    tokens, page = sum(n for n, _ in lengths), case["page"]
    needed = [-(-k // page) for _, k in lengths]
    total, width = sum(needed), max(needed)
    # pages are handed out in any order; entries behind a sequence's last page are not valid
    order = torch.randperm(total, generator=gen, device="cuda").int()
    column = torch.arange(width, device="cuda")
    counts = torch.tensor(needed, device="cuda")
    starts = counts.cumsum(0) - counts
    index = (starts[:, None] + column).clamp(max=total - 1)
    state["page_table"] = torch.where(column < counts[:, None], order[index], -1).int()
    n_new = torch.tensor([n for n, _ in lengths], dtype=torch.int32, device="cuda")
    state["cu_q"] = torch.nn.functional.pad(n_new.cumsum(0), (1, 0)).int()
    state["seq_k"] = torch.tensor([k for _, k in lengths], dtype=torch.int32, device="cuda")
    state["max_q"] = max(n for n, _ in lengths)
    shape = (total, page, hkv, d) if case["layout"] == "bnhd" else (total, hkv, page, d)
    state["k_pages"] = _random(gen, shape, dtype)
    state["v_pages"] = _random(gen, shape, dtype)
    # heads differ in how sharply they look
    gain = 0.5 + 1.5 * torch.rand((1, hq, 1), generator=gen, device="cuda")
    state["q"] = _random(gen, (tokens, hq, d), dtype, gain)
    if case["op"] == "append":
        state["k"] = _random(gen, (tokens, hkv, d), dtype)
        state["v"] = _random(gen, (tokens, hkv, d), dtype)
    return state


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from exact_io_aware_69_b200 import fa
        if op in ("rope", "rope_grad"):
            call = fa.rope if op == "rope" else fa.rope_backward
            return call(state["q"], state["k"], state["freqs"], positions=state["positions"],
                        magnitude=state["magnitude"], interleaved=case["interleaved"],
                        layout=case["layout"])
        cache = (state["k_pages"], state["v_pages"], state["page_table"], state["cu_q"],
                 state["seq_k"])
        if op == "append":
            q = fa.paged_append(state["k"], state["v"], *cache, q=state["q"],
                                freqs=state["freqs"], magnitude=state["magnitude"],
                                interleaved=case["interleaved"], page_layout=case["layout"])
            return q, state["k_pages"], state["v_pages"]
        return fa.paged_attention(state["q"], *cache, max_q=state["max_q"],
                                  window=(case["left"], case["right"]),
                                  page_layout=case["layout"])
    if op in ("rope", "rope_grad"):
        positions = state["positions"][:, :, None] if case["layout"] == "bnhd" \
            else state["positions"][:, None, :]
        sign = 1.0 if op == "rope" else -1.0
        return (_rotate(state["q"], positions, state, sign),
                _rotate(state["k"], positions, state, sign))
    if op == "append":
        return _append(state)
    rows = len(state["lengths"]) * state["max_q"]
    return _attend_padded(state) if rows <= 2 * state["q"].shape[0] and state["max_q"] <= 16 \
        else _attend_each(state)


def _rotate(x, positions, state, sign=1.0):
    """The plain rotation; the angles of far positions are formed in 64 bits."""
    case = state["case"]
    r = case["rot"]
    angle = positions.double()[..., None] * state["freqs"]
    cos = (angle.cos() * state["magnitude"]).float()
    sin = (angle.sin() * (sign * state["magnitude"])).float()
    y = x.float()
    if case["interleaved"]:
        x0, x1 = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1).flatten(-2)
    else:
        x0, x1 = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _owners(state):
    """The sequence and the position of every packed token."""
    n_new = state["cu_q"].diff()
    tokens = state["q"].shape[0]
    owner = torch.repeat_interleave(torch.arange(len(n_new), device="cuda"), n_new,
                                    output_size=tokens)
    place = torch.arange(tokens, device="cuda") - state["cu_q"][owner]
    return owner, place, place + (state["seq_k"] - n_new)[owner]


def _append(state):
    page = state["case"]["page"]
    owner, _, position = _owners(state)
    pages = state["page_table"][owner, position // page].long()
    k = _rotate(state["k"], position[:, None], state)
    where = (pages, position % page) if state["case"]["layout"] == "bnhd" \
        else (pages, slice(None), position % page)
    state["k_pages"][where] = k
    state["v_pages"][where] = state["v"]
    return _rotate(state["q"], position[:, None], state), state["k_pages"], state["v_pages"]


def _visible(i, j, n, k, case):
    """Whether query i of n sees key j of k."""
    seen = j < k
    if case["left"] >= 0:
        seen = seen & (j >= i + (k - n) - case["left"])
    if case["right"] >= 0:
        seen = seen & (j <= i + (k - n) + case["right"])
    return seen


def _softmax_product(scores, v):
    """(O, L) of masked scores [..., rows, keys]; rows that see nothing get 0 and -inf."""
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, 1.0, total), (top + total.log())[..., 0]


def _rows_of(pages, table, layout):
    """The cached rows of the pages in `table`, in order: [..., keys, Hkv, d]."""
    x = pages[table.long()]
    return (x if layout == "bnhd" else x.transpose(-3, -2)).flatten(-4, -3)


def _attend_padded(state):
    """All sequences at once, for batches of few new tokens each."""
    case, q = state["case"], state["q"]
    hq, hkv, d, top = case["hq"], case["hkv"], case["d"], state["max_q"]
    owner, place, _ = _owners(state)
    n, k = state["cu_q"].diff()[:, None, None], state["seq_k"][:, None, None]
    batch = n.shape[0]
    padded = q.new_zeros((batch, top, hq, d), dtype=torch.float32)
    padded[owner, place] = q.float()
    grouped = padded.view(batch, top, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    keys, values = (_rows_of(state[name], state["page_table"].clamp(min=0), case["layout"])
                    .transpose(1, 2).float() for name in ("k_pages", "v_pages"))
    j = torch.arange(keys.shape[2], device="cuda")
    i = torch.arange(top, device="cuda")[:, None]
    seen = _visible(i, j, n, k, case)[:, None].repeat(1, 1, hq // hkv, 1)
    scores = (grouped @ keys.mT).mul_(d ** -0.5).masked_fill_(~seen, -math.inf)
    o, lse = _softmax_product(scores, values)
    o = o.view(batch, hkv, hq // hkv, top, d).permute(0, 3, 1, 2, 4).reshape(batch, top, hq, d)
    lse = lse.view(batch, hq, top).transpose(1, 2)
    return o[owner, place].to(q.dtype), lse[owner, place].T.contiguous()


def _attend_each(state):
    """One sequence after the other, as many key heads at once as 4 GB of scores hold: padding
    long chunks to one length would waste most of the work."""
    case, q = state["case"], state["q"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.empty_like(q)
    lse = torch.empty((hq, q.shape[0]), device="cuda")
    begin, g = 0, hq // hkv
    for b, (n, k) in enumerate(state["lengths"]):
        table = state["page_table"][b, :-(-k // case["page"])]
        keys, values = (_rows_of(state[name], table, case["layout"])[:k].transpose(0, 1)
                        for name in ("k_pages", "v_pages"))
        unseen = ~_visible(torch.arange(n, device="cuda")[:, None],
                           torch.arange(k, device="cuda"), n, k, case)
        rows = q[begin:begin + n].transpose(0, 1).unflatten(0, (hkv, g))
        step = min(hkv, max(1, 2**30 // (n * k * g)))
        for h in range(0, hkv, step):
            grouped = rows[h:h + step].float().flatten(1, 2)
            scores = (grouped @ keys[h:h + step].float().mT).mul_(d ** -0.5)
            scores.unflatten(1, (g, n)).masked_fill_(unseen, -math.inf)
            o, l = _softmax_product(scores, values[h:h + step].float())
            heads = slice(h * g, (h + step) * g)
            out[begin:begin + n, heads] = o.view(-1, n, d).transpose(0, 1).to(q.dtype)
            lse[heads, begin:begin + n] = l.view(-1, n)
        begin += n
    return out, lse


def exact(case, seed):
    """The definition in 64 bits: rotations as complex products, attention from logits row block
    by row block."""
    state = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attention(state)

    def turn(x, position, conjugate=False):
        r = case["rot"]
        unit = torch.polar(torch.full_like(state["freqs"], state["magnitude"]).expand(
            *position.shape, r // 2), position.double()[..., None] * state["freqs"])
        unit = unit.conj() if conjugate else unit
        x = x.double()
        head = x[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
        head = head if case["interleaved"] else head.mT
        turned = torch.view_as_real(torch.view_as_complex(head.contiguous()) * unit)
        turned = turned if case["interleaved"] else turned.mT
        return torch.cat((turned.flatten(-2), x[..., r:]), -1)

    if case["op"] != "append":
        at = state["positions"].unsqueeze(2 if case["layout"] == "bnhd" else 1)
        return tuple(turn(state[name], at, case["op"] == "rope_grad") for name in ("q", "k"))
    at = torch.cat([torch.arange(k - n, k) for n, k in state["lengths"]]).cuda()
    k_new, page = turn(state["k"], at[:, None]), case["page"]
    pools = [state["k_pages"].double(), state["v_pages"].double()]
    views = [p if case["layout"] == "bnhd" else p.transpose(1, 2) for p in pools]
    token = 0
    for b, (n, k) in enumerate(state["lengths"]):
        positions = torch.arange(k - n, k, device="cuda")
        slot = state["page_table"][b].long()[positions // page] * page + positions % page
        for view, new in zip(views, (k_new, state["v"].double())):
            view[slot // page, slot % page] = new[token:token + n]
        token += n
    return turn(state["q"], at[:, None]), pools[0], pools[1]


def _exact_attention(state):
    case = state["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    q = state["q"].double()
    o, lse = torch.zeros_like(q), torch.zeros((hq, q.shape[0]), dtype=torch.float64, device="cuda")
    token = 0
    for b, (n, k) in enumerate(state["lengths"]):
        left = k if case["left"] < 0 else case["left"]
        right = k if case["right"] < 0 else case["right"]
        j = torch.arange(k, device="cuda")
        slots = (state["page_table"][b].long()[j // page], j % page)
        step = max(1, 2**27 // (k * (hq // hkv)))
        for h in range(hkv):
            pick = [state[name][slots[0], slots[1], h] if case["layout"] == "bnhd"
                    else state[name][slots[0], h, slots[1]] for name in ("k_pages", "v_pages")]
            keys, values = pick[0].double(), pick[1].double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for lo in range(0, n, step):
                rows = slice(token + lo, token + min(n, lo + step))
                middle = torch.arange(lo, min(n, lo + step), device="cuda")[:, None, None] + k - n
                logits = torch.einsum("ihd,jd->ihj", q[rows, heads], keys) / math.sqrt(d)
                logits.masked_fill_((j < middle - left) | (j > middle + right), -math.inf)
                sums = torch.logsumexp(logits, -1)
                weights = torch.exp(logits - sums.nan_to_num(neginf=0.0)[..., None])
                o[rows, heads] = torch.einsum("ihj,jd->ihd", weights, values)
                lse[heads, rows] = sums.T
        token += n
    return o, lse
