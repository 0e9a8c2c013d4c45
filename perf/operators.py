"""The paged-cache operators as measured workloads: writing the rows of a qkv projection to a paged
K/V cache (QK-norm, RoPE, quantisation), reading cached rows back, and attention of each sequence's
new rows over its cached positions.

A case is a ragged batch: ``sequences`` sequences whose cached lengths are spread over
``shortest`` .. ``longest`` (new rows included). ``mix`` "all": every sequence has ``new`` new rows;
"every 4th": one in four has ``new`` of them and the others one, as when prompts are read in pieces
between other sequences' steps. ``pad`` rows behind the last sequence belong to nobody and stay as
they are.
"""
import math

import torch

own = False

FP8_MAX = 448.0
MIN_EXP = -110          # smallest exponent of a stored scale
EPS, ROPE_BASE = 1e-6, 10000.0


def _case(name, op, dtype, sequences, new, shortest, longest, q_heads=16, kv_heads=8, head_dim=128, page=64,
          mix="all", causal=True, window=0, pad=0):
    c = dict(op=op, dtype=dtype, sequences=sequences, new=new, shortest=shortest, longest=longest, q_heads=q_heads,
             kv_heads=kv_heads, head_dim=head_dim, page=page, mix=mix, causal=causal, window=window, pad=pad)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one caller, one token a step: nothing but latency
        _case("attend 1x1 over 777", "attend", "bf16", 1, 1, 777, 777, page=16),
        # a full serving batch, one token each, contexts of many ages
        _case("attend 64x1 bf16 ragged", "attend", "bf16", 64, 1, 311, 6000),
        # the same with the cache in 8 bits and longer contexts
        _case("attend 64x1 e4m3 ragged", "attend", "e4m3", 64, 1, 500, 12001, page=32),
        # a prompt piece behind a long context
        _case("attend 1x512 over 32768", "attend", "bf16", 1, 512, 32768, 32768, page=128),
        # prompt pieces between other sequences' steps, in a batch padded for a graph
        _case("attend mixed e4m3", "attend", "e4m3", 16, 301, 700, 9000, page=16, mix="every 4th", pad=27),
        # two prompts read at once from nothing, one query head per kv head
        _case("attend 2x4096 prompts", "attend", "bf16", 2, 4096, 4096, 4096, kv_heads=16),
        # a small decoder's sliding window, heads of 64, four query heads per kv head
        _case("attend 8x1000 window", "attend", "bf16", 8, 1000, 1000, 5003, q_heads=8, kv_heads=2, head_dim=64,
              page=32, window=1024),
        # one step's rows of a full batch, written and read back
        _case("write 64x1 e4m3", "write", "e4m3", 64, 1, 311, 6000, page=32),
        # a long prompt's rows
        _case("write 1x8191 bf16", "write", "bf16", 1, 8191, 8191, 8191),
        # ragged prompt pieces, one query head per kv head
        _case("write mixed e4m3", "write", "e4m3", 24, 1500, 2000, 4000, kv_heads=16, page=16, mix="every 4th", pad=5),
        # a short shared prefix read back
        _case("read 1x1000 e4m3", "read", "e4m3", 1, 1000, 1000, 1000, q_heads=4, kv_heads=2, head_dim=64, page=16),
        # whole contexts read back to be handed on
        _case("read 12x8000 e4m3", "read", "e4m3", 12, 8000, 8000, 8001),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "read"])
    dtype = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    q_heads, kv_heads, head_dim = rng.choice([(16, 8, 128), (16, 8, 128), (16, 16, 128), (16, 4, 128), (8, 2, 64), (4, 2, 64)])
    heads = dict(q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page)
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    if op == "attend" and rng.random() < 0.5:       # steps: one to a few new rows each
        n, new = _log(rng, 1, 64), rng.choice([1, 1, 2, 5])
        longest = _log(rng, 40, 8000)
        return _case("", op, dtype, n, new, max(new, longest // rng.randint(1, 20)), longest, pad=pad,
                     window=rng.choice([0, 0, 0, 257]), **heads)
    n, new = _log(rng, 1, 8), _log(rng, 9, 1500)
    longest = new + (_log(rng, 1, 8000) if rng.random() < 0.7 else 0)
    if op == "attend":
        return _case("", op, dtype, n, new, max(new, longest // rng.randint(1, 4)), longest, pad=pad,
                     mix=rng.choice(["all", "every 4th"]), causal=rng.random() < 0.8,
                     window=rng.choice([0, 0, _log(rng, 30, 3000)]), **heads)
    if op == "write":
        n, new = (_log(rng, 1, 128), 1) if rng.random() < 0.4 else (n, new)
        return _case("", op, dtype, n, new, max(new, longest // rng.randint(1, 3)), max(new, longest), pad=pad,
                     mix=rng.choice(["all", "every 4th"]), **heads)
    return _case("", op, dtype, n, new, new, longest, pad=pad, **heads)


def _lengths(c):
    """Cached length and new rows of every sequence; the longest stands first, the shortest last."""
    n = c["sequences"]
    length = [c["longest"] - (c["longest"] - c["shortest"]) * i // max(1, n - 1) for i in range(n)]
    new = [c["new"] if c["mix"] == "all" or i % 4 == 0 else 1 for i in range(n)]
    return length, new


def _visible(c):
    """Over all new rows, the positions they see; and the positions that some row of the sequence sees."""
    pairs, read = 0, 0
    for L, n in zip(*_lengths(c)):
        w = c["window"] or L
        lo = max(0, L - n - w + 1)
        read += L - lo
        if c["causal"]:
            first, last = L - n + 1, L                  # what the first and the last row would see without a window
            short = max(0, min(last, w) - first + 1)    # rows whose window is not full
            pairs += short * (first + min(last, w)) // 2 + (n - short) * w
        else:
            pairs += sum(L - max(0, L - n + i - w + 1) for i in range(n))
    return pairs, read


def work(case):
    c = case
    rows = sum(_lengths(c)[1])
    d, hq, hkv = c["head_dim"], c["q_heads"], c["kv_heads"]
    held = 2 * hkv * (d * 2 if c["dtype"] == "bf16" else d + 1)         # K and V of one position as the cache holds them
    if c["op"] == "attend":
        pairs, read = _visible(c)
        return {"bytes": rows * hq * d * 4 + read * held, "flops": 4 * d * hq * pairs}
    if c["op"] == "write":
        back = 0 if c["dtype"] == "bf16" else held + 2 * hkv * d * 2    # read back where it is held in 8 bits
        return {"bytes": rows * ((hq + 2 * hkv) * d * 2 + hq * d * 2 + held + back), "flops": rows * (hq + hkv) * d * 10}
    return {"bytes": rows * (held + 2 * hkv * d * 2), "flops": rows * 2 * hkv * d}


def _quantise(x):
    """e4m3 values and scale exponents of rows x[..., head_dim], with the least power of two that holds the row."""
    m, e = torch.frexp(x.abs().amax(-1))                # amax = m 2^e, m in [0.5, 1): 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, MIN_EXP), e).clamp(min=MIN_EXP)
    return torch.ldexp(x, -e[..., None]).float().to(torch.float8_e4m3fn), e


def prepare(case, seed):
    c = case
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    length, new = _lengths(c)
    n, d, hq, hkv, page = c["sequences"], c["head_dim"], c["q_heads"], c["kv_heads"], c["page"]
    need = [-(-L // page) for L in length]
    pages = sum(need) + 3
    wide = max(need) + 1
    start = [0]
    for k in new:
        start.append(start[-1] + k)
    rows = start[-1] + c["pad"]
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([sum(need[:i]) for i in range(n)], device=dev)[:, None]
    at = torch.arange(wide, device=dev)[None, :]
    held = at < torch.tensor(need, device=dev)[:, None]
    table = torch.where(held, order[(first + at).clamp(max=pages - 1)], torch.full_like(order[:1], -1))
    s = dict(case=c, rows=rows, max_new=max(new), max_len=max(length), pages=table.contiguous(),
             start=torch.tensor(start, dtype=torch.int32, device=dev), length=torch.tensor(length, dtype=torch.int32, device=dev))
    shape = (pages, hkv, page, d)

    def normal(shp, std=1.0):
        return (torch.randn(shp, generator=g, device=dev, dtype=torch.float32) * std).to(torch.bfloat16)

    for name in ("k", "v"):
        if c["op"] == "write":                          # an empty cache
            s[name] = torch.zeros(shape, dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.uint8, device=dev)
            s[name + "_scale"] = None if c["dtype"] == "bf16" else torch.zeros(shape[:3], dtype=torch.uint8, device=dev)
        elif c["dtype"] == "bf16":
            s[name], s[name + "_scale"] = normal(shape), None
        else:
            size = torch.exp(0.5 * torch.randn(shape[:3], generator=g, device=dev))     # tokens differ in size
            x, e = _quantise(torch.randn(shape, generator=g, device=dev) * size[..., None])
            s[name], s[name + "_scale"] = x.view(torch.uint8), (e + 127).to(torch.uint8)
            del x, e
    if c["op"] == "attend":
        s["q"] = normal((rows, hq, d), 1.5)
        s["out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=dev)
    else:
        s["k_back"] = torch.zeros((rows, hkv, d), dtype=torch.bfloat16, device=dev)
        s["v_back"] = torch.zeros_like(s["k_back"])
    if c["op"] == "write":
        s["qkv"] = normal((rows, (hq + 2 * hkv) * d))
        s["q_out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=dev)
        s["q_norm"], s["k_norm"] = ((1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2))
    if own:
        from persistent_megakernel_streaming_gb300 import cp
        s["cache"] = cp.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = cp.Batch(s["start"], s["length"], s["pages"], rows, max_new=s["max_new"], max_len=s["max_len"])
    return s


def _rows(s):
    """Sequence and position of each row that belongs to a sequence."""
    row = torch.arange(s["rows"], device=s["start"].device)
    n = s["start"].numel() - 1
    seq = torch.searchsorted(s["start"][1:].contiguous(), row.to(torch.int32), right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    pos = s["length"][seq] - s["start"][seq + 1] + row
    return row, seq, pos, real


def _slots(s, seq, pos):
    """Page and place in the page of position pos of sequence seq."""
    page = s["case"]["page"]
    return s["pages"][seq, pos // page].long(), pos % page


def _values(s, name, page, place):
    """Cached rows [..., kv_heads, head_dim] as the values they stand for, in 32 bits."""
    x = s[name][page, :, place]
    if s["case"]["dtype"] == "bf16":
        return x.float()
    return torch.ldexp(x.view(torch.float8_e4m3fn).float(), (s[name + "_scale"][page, :, place].int() - 127)[..., None])


def _plain_attend(s):
    c = s["case"]
    n, hq, hkv, d = c["sequences"], c["q_heads"], c["kv_heads"], c["head_dim"]
    dev = s["q"].device
    row, seq, pos, real = _rows(s)
    t = torch.arange(s["max_len"], device=dev)
    i = torch.arange(n, device=dev)
    there = t[None] < s["length"][:, None]                                          # [n, T]
    page, place = _slots(s, i[:, None], torch.where(there, t[None], 0))
    k, v = (_values(s, name, page, place) for name in ("k", "v"))                   # [n, T, hkv, d]
    v = torch.where(there[..., None, None], v, 0)
    local = torch.arange(s["max_new"], device=dev)
    mine = local[None] < (s["start"][1:] - s["start"][:-1])[:, None]                # [n, max_new]
    at = (s["start"][:-1, None] + local[None]).clamp(max=s["rows"] - 1).long()
    q = s["q"][at].float().view(n, -1, hkv, hq // hkv, d)
    score = torch.einsum("nmhgd,nthd->nhgmt", q, k) / math.sqrt(d)
    p = pos[at]                                                                     # [n, max_new]
    see = there[:, None] & mine[..., None]
    if c["causal"]:
        see = see & (t[None, None] <= p[..., None])
    if c["window"]:
        see = see & (t[None, None] > p[..., None] - c["window"])
    see = see[:, None, None]
    score = torch.where(see, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(score - top)
    del score
    o = torch.einsum("nhgmt,nthd->nmhgd", w, v) / w.sum(-1).clamp(min=1e-30).permute(0, 3, 1, 2)[..., None]
    s["out"][at[mine]] = o.reshape(n, -1, hq, d)[mine].to(torch.bfloat16)
    return s["out"]


def _angles(pos, d):
    """cos and sin of the rotary angles in 64 bits: far positions turn many times."""
    j = torch.arange(d // 2, device=pos.device, dtype=torch.float64)
    a = pos.double()[:, None] * torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device=pos.device), -2 * j / d)
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def _plain_write(s):
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    row, seq, pos, real = _rows(s)
    row, seq, pos = row[real], seq[real], pos[real]
    x = s["qkv"][row].double().view(len(row), hq + 2 * hkv, d)
    q, k, v = x.split([hq, hkv, hkv], 1)
    cos, sin = _angles(pos, d)

    def turned(y, gain):
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * gain.double()
        a, b = y.split(d // 2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k = turned(q, s["q_norm"]), turned(k, s["k_norm"])
    s["q_out"][row] = q.to(torch.bfloat16)
    page, place = _slots(s, seq, pos)
    if c["dtype"] == "bf16":
        s["k"][page, :, place], s["v"][page, :, place] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        return s["q_out"], s["k"], s["v"]
    k8, ke = _quantise(k)
    v8, ve = _quantise(v)
    s["k"][page, :, place], s["v"][page, :, place] = k8.view(torch.uint8), v8.view(torch.uint8)
    s["k_scale"][page, :, place], s["v_scale"][page, :, place] = (ke + 127).to(torch.uint8), (ve + 127).to(torch.uint8)
    return (s["q_out"], *_plain_read(s))


def _plain_read(s):
    row, seq, pos, real = _rows(s)
    page, place = _slots(s, seq[real], pos[real])
    for name in ("k", "v"):
        s[name + "_back"][row[real]] = _values(s, name, page, place).to(torch.bfloat16)
    return s["k_back"], s["v_back"]


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read}[c["op"]](s)
    if c["op"] == "attend":
        s["cache"].attend(s["batch"], s["q"], s["out"], causal=c["causal"], window=c["window"])
        return s["out"]
    if c["op"] == "write":
        s["cache"].append(s["batch"], s["qkv"], s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], rms_eps=EPS,
                          rope_base=ROPE_BASE)
        if c["dtype"] == "bf16":
            return s["q_out"], s["k"], s["v"]
        s["cache"].read(s["batch"], s["k_back"], s["v_back"])
        return s["q_out"], s["k_back"], s["v_back"]
    s["cache"].read(s["batch"], s["k_back"], s["v_back"])
    return s["k_back"], s["v_back"]


def exact(case, seed):
    """The same outputs in 64 bits, sequence by sequence from the definition."""
    c = case
    s = prepare(case, seed)
    length, new = _lengths(c)
    hq, hkv, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    dev = s["start"].device
    if c["op"] == "attend":
        out = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device=dev)
    else:
        back = [torch.zeros((s["rows"], hkv, d), dtype=torch.float64, device=dev) for _ in range(2)]
    if c["op"] == "write":
        q_out = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device=dev)
        pools = [torch.zeros(s["k"].shape, dtype=torch.float64, device=dev) for _ in range(2)]

    def decoded(byte, e):
        b = byte.long()
        ex, man = (b >> 3) & 15, (b & 7).double()
        size = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(ex.double() - 7))
        return torch.where(b > 127, -size, size) * torch.exp2(e.double() - 127)[..., None]

    def nearest(y):
        """The e4m3 value times its row's power of two nearest to y, ties to an even last bit."""
        top = y.abs().amax(-1, keepdim=True).clamp(min=1e-300)
        e = torch.ceil(torch.log2(top / FP8_MAX)).clamp(min=MIN_EXP)
        e = torch.where(top > FP8_MAX * torch.exp2(e), e + 1, e)
        z = y / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(z / step) * step * torch.exp2(e)

    r = 0
    for i, (L, m) in enumerate(zip(length, new)):
        t = torch.arange(L, device=dev)
        pg, place = s["pages"][i, t // page].long(), t % page
        rows = slice(r, r + m)
        if c["op"] == "write":
            x = s["qkv"][rows].double()
            pos = torch.arange(L - m, L, device=dev, dtype=torch.float64)
            j = torch.arange(d // 2, device=dev, dtype=torch.float64)
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev), pos[:, None] * ROPE_BASE ** (-2 * j / d))

            def head(y, gain):
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + EPS) * gain.double()
                z = torch.complex(y[..., : d // 2], y[..., d // 2:]) * turn[:, None]
                return torch.cat([z.real, z.imag], -1)

            q_out[rows] = head(x[:, : hq * d].reshape(m, hq, d), s["q_norm"])
            k = head(x[:, hq * d:(hq + hkv) * d].reshape(m, hkv, d), s["k_norm"])
            v = x[:, (hq + hkv) * d:].reshape(m, hkv, d)
            for pool, y, into in zip(pools, (k, v), back):
                pool[pg[L - m:], :, place[L - m:]] = y
                into[rows] = nearest(y) if c["dtype"] == "e4m3" else y
            r += m
            continue
        got = []
        for name in ("k", "v"):
            x = s[name][pg, :, place]
            got.append(x.double() if c["dtype"] == "bf16" else decoded(x, s[name + "_scale"][pg, :, place]))
        if c["op"] == "read":
            for into, y in zip(back, got):
                into[rows] = y[L - m:]
            r += m
            continue
        k, v = got
        pos = torch.arange(L - m, L, device=dev)[:, None]
        for h in range(hq):
            a = s["q"][rows, h].double() @ k[:, h // (hq // hkv)].T * d ** -0.5
            hide = torch.zeros_like(a, dtype=torch.bool)
            if c["causal"]:
                hide |= t[None] > pos
            if c["window"]:
                hide |= t[None] <= pos - c["window"]
            out[rows, h] = torch.softmax(a.masked_fill(hide, -math.inf), -1) @ v[:, h // (hq // hkv)]
        r += m
    if c["op"] == "attend":
        return out
    if c["op"] == "read":
        return tuple(back)
    return (q_out, *(pools if c["dtype"] == "bf16" else back))
