"""What a serving loop runs around the paged cache, as measured workloads: projections of few rows with
4-bit weights, verification of drafted tokens, and the management of a cache's pages.

``op`` "linear": ``rows`` rows of a projection from ``k`` to ``n`` features, the weights in 4 bits with
a scale (and a zero point) per ``group`` of inputs; "gated": the weights are a gate's and an up
projection's, the result silu(gate) * up; "add": a residual is added.

"verify": ``sequences`` sequences with 0 .. ``drafts`` drafted tokens each (every sequence ``drafts`` where not
``ragged``), verified against the target's logits over ``vocab`` entries. ``draft`` says what is known of the
draft: its "logits", or the tokens alone.

"branch": ``sequences`` prompts of ``shortest`` .. ``longest`` cached positions, each continued ``ways`` ways:
the branches of the step before are dropped, new ones are forked, all sequences grow by ``new`` positions,
and pages that are written to while shared are copied.

"compact": a pool of ``2 * sequences`` such sequences, every other of which ends; the pages of the others move to
the front, and as many sequences come anew.
"""
import math

import torch

own = False


def _linear(name, rows, k, n, group, out="bf16", zero=False, gated=False, add=False):
    c = dict(op="linear", rows=rows, k=k, n=n, group=group, out=out, zero=zero, gated=gated, add=add)
    return dict(c, name=name) if name else c


def _verify(name, sequences, drafts, vocab, dtype, draft="logits", ragged=True, temperature=0.9, sharp=3.0):
    c = dict(op="verify", sequences=sequences, drafts=drafts, vocab=vocab, dtype=dtype, draft=draft, ragged=ragged,
             temperature=temperature, sharp=sharp)
    return dict(c, name=name) if name else c


def _pages(name, op, sequences, shortest, longest, dtype="bf16", kv_heads=8, head_dim=128, page=64, ways=1, new=1):
    c = dict(op=op, sequences=sequences, shortest=shortest, longest=longest, dtype=dtype, kv_heads=kv_heads, head_dim=head_dim,
             page=page, ways=ways, new=new)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one caller's qkv projection, one token: nothing but latency
        _linear("linear 1 row, 2048 to 4096", 1, 2048, 4096, 128),
        # a head over an odd vocabulary, logits in 32 bits for the sampler
        _linear("linear 3 rows, head of 50001", 3, 2048, 50001, 128, out="fp32"),
        # a gate and up projection, one caller's step with four drafted tokens, weights with zero points
        _linear("linear 5 rows, gated 2x6144", 5, 2048, 12288, 64, zero=True, gated=True),
        # a wide down projection of a full batch, onto the residual
        _linear("linear 64 rows, 16384 to 8192", 64, 16384, 8192, 128, add=True),
        # the gate and up projection of a full batch with four drafted tokens each
        _linear("linear 320 rows, gated 2x6144", 320, 2048, 12288, 32, gated=True),
        # one caller, four drafted codes
        _verify("verify 1x4 of 2048", 1, 4, 2048, "fp32", ragged=False),
        # a full batch, drafts of a lookup whose probabilities are not known
        _verify("verify 64x0-4 of 32000, tokens", 64, 4, 32000, "bf16", draft="tokens"),
        # a full batch over a large, odd vocabulary, drafts of a small model
        _verify("verify 48x7 of 131075", 48, 7, 131075, "fp32", ragged=False),
        # four continuations of each of eight prompts
        _pages("branch 8x4", "branch", 8, 700, 3001, ways=4, new=5),
        # a full pool, two ways each, cache in 8 bits, small pages
        _pages("branch 200x2 e4m3", "branch", 200, 311, 6000, dtype="e4m3", page=32, ways=2, new=3),
        # a few sequences of a small cache
        _pages("compact 6 of 12", "compact", 6, 200, 1500, kv_heads=2, head_dim=64, page=16),
        # a large pool gives its end back
        _pages("compact 40 of 80", "compact", 40, 311, 6000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "verify", "verify", "branch", "compact"])
    if op == "linear":
        group = rng.choice([32, 64, 128])
        rows, k, n = _log(rng, 1, 400), max(1, _log(rng, 128, 16384) // group) * group, _log(rng, 40, 32768)
        while rows * k * n > 64 * 16384 * 8192 or k * n > 16384 * 8192:
            rows, n = max(1, rows // 2), max(40, n // 2 + 1)
        gated = rng.random() < 0.4
        return _linear("", rows, k, n // 2 * 2 if gated else n, group, rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.4,
                       gated, rng.random() < 0.4)
    if op == "verify":
        vocab, drafts = _log(rng, 256, 140000), rng.randint(0, 7)
        return _verify("", max(1, min(_log(rng, 1, 128), 48 * 7 * 131075 // (vocab * (drafts + 1)))), drafts, vocab,
                       rng.choice(["fp32", "bf16"]), rng.choice(["logits", "tokens"]), rng.random() < 0.5,
                       rng.choice([0.0, 0.7, 1.0, round(rng.uniform(0.3, 1.5), 3)]), round(rng.uniform(2.0, 5.0), 2))
    heads = dict(zip(("kv_heads", "head_dim"), rng.choice([(8, 128), (16, 128), (4, 128), (2, 64)])))
    dtype, page = rng.choice(["bf16", "e4m3"]), rng.choice([16, 32, 64, 128])
    longest = _log(rng, 20, 6000)
    shortest = max(1, longest // rng.randint(1, 12))
    if op == "branch":
        return _pages("", op, _log(rng, 1, 64), shortest, longest, dtype, page=page, ways=rng.randint(1, 5), new=rng.randint(1, 9), **heads)
    return _pages("", op, _log(rng, 1, 30), shortest, longest, dtype, page=page, **heads)


def _starts(c):
    """First row of each sequence, and the row past the last: a row for each drafted token and one more."""
    start = [0]
    for i in range(c["sequences"]):
        n = (i * 7 + 3) % (c["drafts"] + 1) if c["ragged"] else c["drafts"]
        start.append(start[-1] + n + 1)
    return start


def _lengths(c):
    """Cached positions of each of the prompts (branch) or of all sequences (compact)."""
    n = c["sequences"] * (1 if c["op"] == "branch" else 2)
    return [c["longest"] - (c["longest"] - c["shortest"]) * ((i * 5) % n) // max(1, n - 1) for i in range(n)]


def _page_bytes(c):
    return 2 * c["kv_heads"] * c["page"] * (c["head_dim"] * 2 if c["dtype"] == "bf16" else c["head_dim"] + 1)


def work(case):
    c = case
    if c["op"] == "linear":
        outs = c["n"] // 2 if c["gated"] else c["n"]
        held = c["k"] * c["n"] // 2 + c["k"] // c["group"] * c["n"] * (3 if c["zero"] else 2)
        out = c["rows"] * outs * (2 if c["out"] == "bf16" else 4)
        return {"bytes": held + c["rows"] * c["k"] * 2 + out * (2 if c["add"] else 1), "flops": 2 * c["rows"] * c["k"] * c["n"]}
    if c["op"] == "verify":
        rows, n = _starts(c)[-1], c["sequences"]
        read = rows + (rows - n if c["draft"] == "logits" and c["temperature"] > 0 else 0)
        return {"bytes": read * c["vocab"] * (2 if c["dtype"] == "bf16" else 4) + rows * 12 + n * 16, "flops": read * c["vocab"] * 4}
    held = [-(-L // c["page"]) for L in _lengths(c)]
    if c["op"] == "branch":
        shared = sum(L % c["page"] > 0 for L in _lengths(c))
        return {"bytes": 2 * shared * c["ways"] * _page_bytes(c) + sum(held) * 4 * 2 * c["ways"], "flops": 0}
    ends, stays = sum(held[0::2]), sum(held[1::2])
    # from the second pass on those that stay lie behind those that end: as many pages move as the fewer of the two hold
    return {"bytes": 2 * min(ends, stays) * _page_bytes(c) + (ends + stays) * 4 * 2, "flops": 0}


def prepare(case, seed):
    c = case
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def whole(lo, hi, shape, dtype=torch.int32):
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=dtype)

    def normal(shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    def uniform(n):
        return torch.rand(n, generator=g, device=dev, dtype=torch.float32)

    s = dict(case=c)
    if c["op"] == "linear":
        out = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        outs = c["n"] // 2 if c["gated"] else c["n"]
        groups = (c["n"], c["k"] // c["group"])
        s["q"] = whole(0, 256, (c["n"], c["k"] // 2), torch.uint8)          # two weights a byte, the even one in its low half
        s["scale"] = (torch.exp(0.3 * torch.randn(groups, generator=g, device=dev)) * 0.2 / math.sqrt(c["k"])).to(torch.bfloat16)
        s["zero"] = whole(5, 11, groups, torch.uint8) if c["zero"] else None
        s["x"] = normal((c["rows"], c["k"]))
        s["add"] = normal((c["rows"], outs), 1.0, out) if c["add"] else None
        s["out"] = torch.zeros((c["rows"], outs), dtype=out, device=dev)
        if own:
            from persistent_megakernel_streaming_gb300 import cp
            s["linear"] = cp.Linear(s["q"], s["scale"], s["zero"], gated=c["gated"])
        return s
    if c["op"] == "verify":
        start = _starts(c)
        rows, n, v = start[-1], c["sequences"], c["vocab"]
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        near = normal((rows, v), c["sharp"], torch.float32)
        s["logits"] = near.to(dtype)
        guess = (near + normal((rows, v), 0.5, torch.float32)).to(dtype)     # a draft that mostly agrees
        del near
        t = max(c["temperature"], 0.1)
        top = guess.float() / t - torch.log(-torch.log(torch.rand((rows, v), generator=g, device=dev).clamp(1e-7, 1 - 1e-7)))
        s["draft"] = top.argmax(-1).to(torch.int32)                          # a token drawn from the draft
        del top
        s["draft_logits"] = guess if c["draft"] == "logits" else None
        s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
        s["u_accept"], s["u_token"] = uniform(rows), uniform(n)
        s["temperature"] = torch.full((n,), c["temperature"], dtype=torch.float32, device=dev)
        s["accepted"], s["token"] = (torch.zeros(n, dtype=torch.int32, device=dev) for _ in range(2))
        s["prob"] = torch.zeros(rows, dtype=torch.float32, device=dev)
        return s
    length = _lengths(c)
    page, ways = c["page"], c["ways"] if c["op"] == "branch" else 0
    held = [-(-L // page) for L in length]
    n = len(length)
    spare = n * (ways + 1) * (c["new"] // page + 2) if ways else 3           # what the branches take
    pages, wide = sum(held) + spare, max(held) + c["new"] // page + 2
    total = n * (ways + 1)                                                   # prompts first, then the branches' places
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    if not ways:
        order = torch.randperm(pages - spare, generator=g, device=dev).to(torch.int32)
    count = torch.tensor(held, device=dev)
    first, at = (count.cumsum(0) - count)[:, None], torch.arange(wide, device=dev)[None, :]
    mine = at < count[:, None]
    table = torch.full((total, wide), -1, dtype=torch.int32, device=dev)
    table[:n] = torch.where(mine, order[(first + at).clamp(max=len(order) - 1)], -1)
    s["table"] = table
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
    s["refs"][order[: sum(held)].long()] = 1
    s["length"] = torch.zeros(total, dtype=torch.int32, device=dev)
    s["length"][:n] = torch.tensor(length, dtype=torch.int32, device=dev)
    shape = (pages, c["kv_heads"], page, c["head_dim"])
    for name in ("k", "v"):
        if c["dtype"] == "bf16":
            s[name], s[name + "_scale"] = normal(shape), None
        else:
            s[name] = normal(shape, 100.0).to(torch.float8_e4m3fn)
            s[name + "_scale"] = whole(110, 130, shape[:3], torch.uint8)
    s["moves"] = torch.zeros((max(total, pages // 2 + 1), 2), dtype=torch.int32, device=dev)
    s["count"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if ways:
        s["keep"] = s["length"].clone()
        s["src"] = torch.arange(n, dtype=torch.int32, device=dev).repeat_interleave(ways)
        s["dst"] = torch.arange(n, total, dtype=torch.int32, device=dev)
        s["new"] = torch.full((total,), c["new"], dtype=torch.int32, device=dev)
    else:
        even = torch.arange(n, device=dev) % 2 == 0                          # the sequences that end in turn
        s["keep"] = [torch.where(even == (k == 0), 0, s["length"]) for k in range(2)]
        s["new"] = [s["length"] - keep for keep in s["keep"]]
        s["turn"] = 0
    if own:
        from persistent_megakernel_streaming_gb300 import cp
        s["pool"] = cp.Pages(s["refs"], s["table"], s["length"], page)
        s["cache"] = cp.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------------ plain forms
def _weights(s):
    """The weights as the bf16 numbers they stand for, [n][k]."""
    c = s["case"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], -1).view(c["n"], c["k"] // c["group"], c["group"])
    z = 8 if s["zero"] is None else s["zero"][..., None].float()
    w = (q.float() - z) * s["scale"].float()[..., None]
    return w.to(torch.bfloat16).float().view(c["n"], c["k"])


def _plain_linear(s):
    y = s["x"].float() @ _weights(s).T
    if s["case"]["gated"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1 + torch.exp(-gate)) * up
    if s["add"] is not None:
        y = y + s["add"].float()
    s["out"].copy_(y)
    return s["out"]


def _softmax(x, temperature):
    """Probabilities over the last axis, each step in 32 bits, the sum in 64."""
    x = x.float() * (1 / temperature)[:, None]
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e * (1 / e.sum(-1, dtype=torch.float64, keepdim=True)).float()


def _plain_verify(s):
    c = s["case"]
    start, v = s["start"].long(), c["vocab"]
    n, rows = len(start) - 1, len(s["logits"])
    row = torch.arange(rows, device=start.device)
    seq = torch.searchsorted(start[1:].contiguous(), row, right=True)
    last = row == start[1:][seq] - 1
    d = torch.where(last, 0, s["draft"]).long()
    heat = s["temperature"][seq]
    greedy = heat <= 0
    heat = torch.where(greedy, 1.0, heat)
    p = _softmax(s["logits"], heat)
    p_d = p.gather(1, d[:, None])[:, 0]
    if s["draft_logits"] is None:
        q, q_d = None, torch.ones_like(p_d)
    else:
        q = _softmax(s["draft_logits"], heat)
        q_d = q.gather(1, d[:, None])[:, 0]
    best = s["logits"].float().argmax(-1)
    yes = torch.where(greedy, d == best, s["u_accept"].double() * q_d.double() < p_d.double()) & ~last
    place = row - start[:-1][seq]
    first = torch.full((n,), rows, device=start.device).scatter_reduce(0, seq, torch.where(yes, rows, place), "amin")
    at = start[:-1] + first                                                  # the refused row, or the last
    w = p[at]
    del p
    refused = ~last[at]
    if q is None:
        w = torch.where(refused[:, None] & (torch.arange(v, device=w.device)[None] == d[at][:, None]), 0, w)
    else:
        w = torch.where(refused[:, None], (w - q[at]).clamp(min=0), w)
        del q
    total = w.double().cumsum(-1)
    token = (total <= s["u_token"].double()[:, None] * total[:, -1:]).sum(-1).clamp(max=v - 1)
    s["accepted"].copy_(first)
    s["token"].copy_(torch.where(greedy[at], best[at], token))
    s["prob"].copy_(torch.where(last, s["prob"], p_d))
    return s["accepted"], s["token"], s["prob"]


def _pages_of(length, page):
    return (length + page - 1) // page


def _held(s):
    """Which table entries stand for pages."""
    return torch.arange(s["table"].shape[1], device=s["table"].device)[None] < _pages_of(s["length"], s["case"]["page"])[:, None]


def _count(s, entries, mask, by):
    s["refs"].scatter_add_(0, torch.where(mask, entries, 0).reshape(-1).long(), (mask * by).to(torch.int32).reshape(-1))


def _plain_trim(s, keep):
    had = _held(s)
    s["length"].copy_(torch.minimum(s["length"], keep))
    drop = had & ~_held(s)
    _count(s, s["table"], drop, -1)
    s["table"].masked_fill_(drop, -1)


def _plain_fork(s, src, dst):
    src, dst = src.long(), dst.long()
    held = _held(s)[src]
    rows = s["table"][src]
    s["table"][dst] = torch.where(held, rows, s["table"][dst])
    s["length"][dst] = s["length"][src]
    _count(s, rows, held, 1)


def _plain_grow(s, new):
    page, table, refs, length = s["case"]["page"], s["table"], s["refs"], s["length"]
    n, wide = table.shape
    i = torch.arange(n, device=table.device)
    tail = (length // page).long().clamp(max=wide - 1)
    last = torch.where(length % page != 0, table[i, tail], -1)
    shared = (new > 0) & (last >= 0) & (refs[last.clamp(min=0).long()] > 1)
    before = ((last[None] == last[:, None]) & shared[None] & (i[None] < i[:, None])).sum(-1)
    copied = shared & (before < refs[last.clamp(min=0).long()] - 1)          # the last sharer keeps the page
    had, want = _pages_of(length, page), _pages_of(length + new, page)
    fresh = want - had + copied
    end = fresh.cumsum(0)
    free = refs == 0
    rank = free.cumsum(0) - 1
    at = torch.full((len(refs) + 1,), -1, dtype=torch.int32, device=table.device)
    at[torch.where(free, rank, len(refs))] = torch.arange(len(refs), dtype=torch.int32, device=table.device)
    begin = end - fresh
    own_page = at[torch.where(copied, begin, 0)]
    k = copied.cumsum(0) - 1                                                 # the pool holds enough in these cases
    slot = torch.where(copied, k, len(s["moves"]) - 1)
    kept = s["moves"][-1].clone()
    s["moves"][slot] = torch.where(copied[:, None], torch.stack([last, own_page], -1), kept)
    s["count"].copy_(copied.sum())
    _count(s, last, copied, -1)
    table[i, tail] = torch.where(copied, own_page, table[i, tail])
    col = torch.arange(wide, device=table.device)[None]
    more = (col >= had[:, None]) & (col < want[:, None])
    pick = begin[:, None] + copied[:, None] + col - had[:, None]
    table.copy_(torch.where(more, at[torch.where(more, pick, 0)], table))
    _count(s, table, more, 1)
    _count(s, own_page, copied, 1)
    length.add_(new)


def _plain_compact(s):
    refs = s["refs"]
    pages = len(refs)
    at = torch.arange(pages, device=refs.device)
    live = refs > 0
    n = live.sum()
    move, hole = live & (at >= n), ~live & (at < n)
    place = torch.full((pages + 1,), -1, device=refs.device)
    place[torch.where(hole, hole.cumsum(0) - 1, pages)] = at
    rank = move.cumsum(0) - 1
    to = torch.where(move, place[rank.clamp(min=0)], at)
    kept = s["moves"][-1].clone()
    slot = torch.where(move, rank, len(s["moves"]) - 1)
    s["moves"][slot] = torch.where(move[:, None], torch.stack([at, to], -1).to(torch.int32), kept)
    s["count"].copy_(move.sum())
    old = refs.clone()
    refs.masked_fill_(move, 0)
    refs.scatter_add_(0, to, torch.where(move, old, 0))
    s["table"].copy_(torch.where(_held(s), to[s["table"].clamp(min=0).long()].to(torch.int32), s["table"]))


def _plain_copy(s):
    moves = s["moves"][: int(s["count"])].long()
    for name in ("k", "v", "k_scale", "v_scale"):
        if s[name] is not None:
            x = s[name].view(torch.uint8) if s[name].element_size() == 1 else s[name]
            x[moves[:, 1]] = x[moves[:, 0]]


def _outputs(s):
    """The pages' state and contents; e4m3 as the values and scales they are held as."""
    return [s["table"], s["refs"], s["length"], s["count"], s["k"], s["v"], s["k_scale"], s["v_scale"]]


def run(state):
    s = state
    c = s["case"]
    if c["op"] == "linear":
        if not own:
            return _plain_linear(s)
        s["linear"].apply(s["x"], s["out"], add=s["add"])
        return s["out"]
    if c["op"] == "verify":
        if not own:
            return _plain_verify(s)
        from persistent_megakernel_streaming_gb300 import cp
        cp.verify(s["logits"], s["draft"], s["start"], s["u_accept"], s["u_token"], s["temperature"], s["accepted"], s["token"],
                  prob=s["prob"], draft_logits=s["draft_logits"])
        return s["accepted"], s["token"], s["prob"]
    if c["op"] == "branch":
        if own:
            s["pool"].trim(s["keep"])
            s["pool"].fork(s["src"], s["dst"])
            s["pool"].grow(s["new"], s["moves"], s["count"])
            s["cache"].copy(s["moves"], s["count"])
        else:
            _plain_trim(s, s["keep"])
            _plain_fork(s, s["src"], s["dst"])
            _plain_grow(s, s["new"])
            _plain_copy(s)
        return _outputs(s)
    keep, new = s["keep"][s["turn"]], s["new"][s["turn"]]
    s["turn"] ^= 1                                                           # the next pass ends the other half
    if own:
        s["pool"].trim(keep)
        s["pool"].compact(s["moves"], s["count"])
        s["cache"].copy(s["moves"], s["count"])
        s["pool"].grow(new, s["moves"], s["count"])
    else:
        _plain_trim(s, keep)
        _plain_compact(s)
        _plain_copy(s)
        _plain_grow(s, new)
    return _outputs(s)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The computed numbers in 64 bits from the definitions: a projection's results, and the target's probabilities of
    the drafted tokens. Pages hold no computed numbers."""
    c = case
    if c["op"] in ("branch", "compact"):
        return None
    s = prepare(case, seed)
    if c["op"] == "verify":
        start = _starts(c)
        prob = torch.zeros(start[-1], dtype=torch.float64, device=s["prob"].device)
        heat = c["temperature"] if c["temperature"] > 0 else 1.0
        for i in range(c["sequences"]):
            for r in range(start[i], start[i + 1] - 1):
                x = s["logits"][r].double() / heat
                prob[r] = torch.exp(x[s["draft"][r].long()] - torch.logsumexp(x, 0))
        return None, None, prob
    x = s["x"].double()
    y = torch.empty((c["rows"], c["n"]), dtype=torch.float64, device=x.device)
    for a in range(0, c["n"], 2048):
        q = s["q"][a:a + 2048]
        w = torch.empty((len(q), c["k"]), dtype=torch.float64, device=x.device)
        w[:, 0::2], w[:, 1::2] = (q % 16).double(), torch.div(q, 16, rounding_mode="floor").double()
        by = torch.arange(c["k"], device=x.device) // c["group"]
        w -= 8.0 if s["zero"] is None else s["zero"][a:a + 2048].double()[:, by]
        w = (w * s["scale"][a:a + 2048].double()[:, by]).to(torch.bfloat16).double()    # a weight is a bf16 number
        y[:, a:a + 2048] = x @ w.T
    if c["gated"]:
        half = c["n"] // 2
        y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
    return y if s["add"] is None else y + s["add"].double()
