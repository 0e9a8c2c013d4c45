"""Probabilities of drafted tokens where logits are large against their differences: small temperatures, common offsets, the
largest numbers, ties. The formula from the fp32 products l * (1 / T) on is computed in 64 bits; what the kernels may be off
does not depend on how large those products are."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from oracle import verify as ref
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24              # half of fp32's, relative
MOST_U = 1 - 2.0 ** -24


def bound(vocab, below):
    """Relative error of a probability exp(x - m) / sum, in half steps: `below` = m - x of its own token.

    Numerator: the difference rounds (`below`), the exponential is off by 2 steps (4). A term of the sum: difference,
    product with log2(e) and that number's own rounding (2.3 (m - x)), the exponential 2^-22 (4), and on the way up to three
    factors between partial maxima, whose differences round too (3 (m - x) + 15); the mean of m - x, weighted by the terms,
    is at most ln(vocab). Additions: up to 64 in a thread, 5 in a warp, 5 and 5 over warps and pieces, a few more over the 32nd
    piece. The division 1."""
    return STEP * (below + 4 + 5.3 * np.log(vocab) + 19 + 90 + 1)


def run(logits, draft, start, u_accept, u_token, temperature, draft_logits=None):
    n, rows = len(start) - 1, len(logits)
    accepted, token = (torch.full((n,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    prob = torch.full((rows,), -7.0, device="cuda")
    f = lambda a: torch.tensor(np.asarray(a, np.float32)).cuda()
    i = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    cp.verify(logits.cuda(), i(draft), i(start), f(u_accept), f(u_token), f(temperature), accepted, token, prob=prob,
              draft_logits=None if draft_logits is None else draft_logits.cuda())
    return accepted.cpu().numpy(), token.cpu().numpy(), prob.cpu().numpy().astype(np.float64)


def wide(t):
    return t.float().numpy()


def check(logits, draft, start, u_accept, u_token, temperature, draft_logits=None):
    accepted, token, prob = run(logits, draft, start, u_accept, u_token, temperature, draft_logits)
    vocab = logits.shape[1]
    for i in range(len(start) - 1):
        taken, refused, near = 0, False, False
        for r in range(start[i], start[i + 1] - 1):
            d = int(draft[r])
            p, x = ref.probabilities(wide(logits[r]), temperature[i])
            ep = bound(vocab, x.max() - x[d])
            assert abs(prob[r] - p[d]) <= ep * p[d] + 2.0 ** -125, (r, prob[r], p[d])
            assert prob[r] <= 1
            q, eq = 1.0, 0.0
            if draft_logits is not None:
                qs, y = ref.probabilities(wide(draft_logits[r]), temperature[i])
                q, eq = qs[d], bound(vocab, y.max() - y[d])
            a, b = float(np.float32(u_accept[r])) * q, p[d]
            if not refused:
                if abs(a - b) <= (ep + eq) * max(a, b) + 2.0 ** -125:
                    near = True                                  # either way
                    break
                refused = not a < b
                taken += not refused
        if near:
            continue
        assert accepted[i] == taken, i
        r = start[i] + taken
        p, x = ref.probabilities(wide(logits[r]), temperature[i])
        w, size = p.copy(), 1.0
        if refused and draft_logits is None:
            w[draft[r]] = 0
        elif refused:
            w, size = np.maximum(p - ref.probabilities(wide(draft_logits[r]), temperature[i])[0], 0), 2.0
        if w.sum() <= bound(vocab, np.log(vocab)) * size:
            continue                                             # what is left is within what p and q are off
        c = np.cumsum(w)
        target, off, t = float(np.float32(u_token[i])) * c[-1], 4 * bound(vocab, np.log(vocab)) * size, int(token[i])
        assert 0 <= t < vocab and c[t] >= target - off and (c[t - 1] if t else 0.0) <= target + off, i
    return accepted, token, prob


def batch(vocab, dtype, seed, sequences=6, drafts=3, sharp=3.0, offset=0.0, factor=1.0):
    """Rows of which each sequence's first has two equal largest logits, its second one far above the others."""
    g = np.random.default_rng(seed)
    rows = sequences * (drafts + 1)
    x = (17 + sharp * g.standard_normal((rows, vocab))) * factor + offset
    y = x + 0.5 * sharp * factor * g.standard_normal((rows, vocab))
    start = np.arange(sequences + 1) * (drafts + 1)
    draft = g.integers(0, vocab, rows)
    for r in range(rows):
        top = np.argsort(x[r])[-3:]
        kind = r % (drafts + 1)
        if kind == 0 and vocab > 1:
            x[r, top[0]] = x[r, top[2]]
            draft[r] = top[0]
        elif kind == 1:
            x[r, top[2]] += 20 * sharp * factor
            draft[r] = top[2]
        elif g.random() < 0.7:
            draft[r] = top[g.integers(0, 3)]
    logits, near = torch.tensor(x, dtype=torch.float32).to(dtype), torch.tensor(y, dtype=torch.float32).to(dtype)
    return logits, draft, start, g.random(rows) * 0.999, g.random(sequences), near


# one launch, two launches, several pieces, more pieces than a warp has lanes
VOCABS = [517, 4096, 4097, 9001, 140001]


@pytest.mark.parametrize("temperature", [0.9, 1e-2, 1e-3, 1e-4, 1e-6, 1e-8, 1e-30])
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_temperatures(temperature, vocab, dtype):
    x, draft, start, ua, ut, y = batch(vocab, dtype, vocab)
    heat = [temperature] * (len(start) - 1)
    check(x, draft, start, ua, ut, heat, y)
    check(x, draft, start, ua, ut, heat)


@pytest.mark.parametrize("offset", [1e4, -1e4, 1e6, -1e6, 3e7])
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_common_offsets(offset, vocab, dtype):
    x, draft, start, ua, ut, y = batch(vocab, dtype, vocab + 1, offset=offset)
    heat = [1.0, 0.7, 1.3, 1.0, 0.25, 2.0]
    check(x, draft, start, ua, ut, heat, y)
    check(x, draft, start, ua, ut, heat)


@pytest.mark.parametrize("factor", [1e10, 1e30, 3e36])
@pytest.mark.parametrize("vocab", VOCABS)
def test_large_logits(factor, vocab):
    x, draft, start, ua, ut, y = batch(vocab, torch.float32, vocab + 2, factor=factor)
    x.clamp_(-3.3e38, 3.3e38)
    check(x, draft, start, ua, ut, [1.0] * 6, y)
    check(-x, draft, start, ua, ut, [1.0] * 6)


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_certain_and_tied_tokens(vocab, dtype):
    """All of the probability, and half of it, exactly: 1 is taken whatever the draw, 1/2 below 1/2."""
    for temperature in (1e-2, 1e-4, 1e-6, 1e-8):
        for top in (5.0, 23.0, 30.0, -30.0):
            x = torch.full((8, vocab), top - 4.0)
            x[:, 7] = top
            x[4:, vocab - 2] = top                              # two sequences of a certain token, two of tied ones
            draft = [7, 7, 7, 0, 7, 0, vocab - 2, 0]
            ua = [MOST_U, MOST_U, MOST_U, 0, 0.5, 0, 0.4999999, 0]
            accepted, token, prob = run(x.to(dtype), draft, [0, 4, 6, 8], ua, [0.3, 0.3, 0.6], [temperature] * 3)
            assert prob[[0, 1, 2]].tolist() == [1.0] * 3 and prob[[4, 6]].tolist() == [0.5] * 2
            assert accepted.tolist() == [3, 0, 1]
            assert token.tolist() == [7, vocab - 2, vocab - 2]   # the last: of the row behind, 0.6 of two halves


@pytest.mark.parametrize("vocab", [64, 8192])
def test_rows_of_the_lowest_number(vocab):
    """fp32's lowest has no probability, whatever else there is; bf16's is a number like another."""
    for dtype, temperature, weighs in ((torch.float32, 1.0, False), (torch.float32, 0.5, False), (torch.float32, 2.0, True),
                                       (torch.bfloat16, 1.0, True), (torch.bfloat16, 0.5, False)):
        x = torch.full((3, vocab), torch.finfo(dtype).min, dtype=dtype)
        accepted, token, prob = run(x, [3, 0, 0], [0, 2, 3], [0.0, 0, 0], [0.5, 0.5], [temperature] * 2)
        assert accepted.tolist() == [int(weighs), 0]
        assert token.tolist() == ([vocab // 2] * 2 if weighs else [-1] * 2)
        assert prob[0] == (1 / vocab if weighs else 0)
