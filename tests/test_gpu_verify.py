"""Verification of drafted tokens against float64: which tokens are taken, the token behind them, masks, ends and repeats."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from oracle import verify as ref
from persistent_megakernel_streaming_gb300 import cp

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def make(drafted, vocab, dtype=torch.float32, seed=0, temperature=0.9, sharp=3.0, with_draft=True, pad=0):
    """A batch of len(drafted) sequences; a draft that is near the target."""
    g = torch.Generator().manual_seed(seed)
    n, rows = len(drafted), sum(drafted) + len(drafted) + pad
    b = dict(start=np.concatenate([[0], np.cumsum([d + 1 for d in drafted])]).astype(np.int32))
    near = torch.randn(rows, vocab, generator=g) * sharp
    b["logits"] = near.to(dtype)
    b["draft_logits"] = (near + 0.5 * torch.randn(rows, vocab, generator=g)).to(dtype) if with_draft else None
    b["draft"] = torch.argmax(near + 1.5 * torch.randn(rows, vocab, generator=g), -1).to(torch.int32)
    b["u_accept"], b["u_token"] = torch.rand(rows, generator=g), torch.rand(n, generator=g)
    b["temperature"] = torch.full((n,), float(temperature)) if np.isscalar(temperature) else torch.tensor(temperature)
    return b


def run(b, workspace=None, stream=None, move=lambda t: t.cuda()):
    n, rows = len(b["start"]) - 1, len(b["logits"])
    accepted, token = (torch.full((n,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    prob = torch.full((rows,), -7.0, device="cuda")
    cp.verify(move(b["logits"]), b["draft"].cuda(), torch.from_numpy(b["start"]).cuda(), b["u_accept"].cuda(), b["u_token"].cuda(),
              b["temperature"].cuda().float(), accepted, token, prob=prob,
              draft_logits=None if b["draft_logits"] is None else move(b["draft_logits"]), workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return accepted.cpu().numpy(), token.cpu().numpy(), prob.cpu().numpy()


def wide(t):
    return None if t is None else t.float().double().numpy()


def check(b, got=None):
    """A probability's relative error: an exponential whose argument is off by some half steps of the largest scaled
    logits, and some steps of its own. A decision nearer than that may fall either way, and so may a draw whose target is
    within the weights' errors of a token's edge."""
    accepted, token, prob = run(b) if got is None else got
    vocab = b["logits"].shape[1]
    want, p = ref.verify(b["start"], wide(b["logits"]), b["draft"].numpy(), b["u_accept"].numpy(), b["u_token"].numpy(),
                         b["temperature"].numpy(), wide(b["draft_logits"]))
    top = np.abs(np.where(np.isfinite(wide(b["logits"])), wide(b["logits"]), 0)).max()
    heat = b["temperature"].float().numpy()
    most = top / min([t for t in heat if t > 0] + [1.0])
    eps = (4 * most + 64) * 2.0 ** -24
    drafted = ~np.isnan(p)
    assert (np.abs(prob[drafted] - p[drafted]) <= eps * p[drafted] + 1e-37).all()
    assert (prob[~drafted] == -7).all()
    close = 0
    for i, w in enumerate(want):
        if w["near"] < 2 * eps and accepted[i] != w["accepted"]:
            close += 1
            continue
        assert accepted[i] == w["accepted"], i
        if "cum" not in w:
            assert token[i] == w["token"], i
            continue
        t = int(token[i])
        off = 4 * eps * w["size"]
        assert 0 <= t < vocab and w["cum"][t] >= w["target"] - off, i
        assert (w["cum"][t - 1] if t else 0.0) <= w["target"] + off, i
        if w["weights"][t] <= 0:
            assert off > 0 and (abs(w["cum"] - w["target"]) <= off).any()
    assert close <= 1
    return accepted, token, prob


@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 31, 33, 255, 1000, 2048, 8191, 8192, 8193, 8200, 16385, 32000, 50257])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabularies(vocab, dtype):
    check(make([0, 1, 4, 2, 3], vocab, dtype, seed=vocab))
    check(make([5, 0, 1], vocab, dtype, seed=vocab + 1, with_draft=False, temperature=1.3))


@pytest.mark.parametrize("temperature", [0.05, 0.3, 1.0, 2.5, 1e30, 0.0, -1.0, NAN])
@pytest.mark.parametrize("with_draft", [False, True])
def test_temperatures(temperature, with_draft):
    check(make([3, 0, 7, 1], 1003, seed=3, temperature=temperature, with_draft=with_draft, sharp=1.0))


def test_mixed_temperatures_and_many_sequences():
    g = np.random.default_rng(0)
    b = make([int(x) for x in g.integers(0, 6, 300)], 517, seed=5, sharp=2.0, pad=11)
    b["temperature"] = torch.from_numpy(np.where(g.random(300) < 0.3, 0.0, g.uniform(0.2, 1.5, 300)).astype(np.float32))
    accepted, token, _ = check(b)
    assert accepted.max() >= 4 and (accepted == 0).any()


@pytest.mark.parametrize("vocab", [4601, 4605, 4606, 5113, 5114, 8185, 8187, 8189, 8701, 8702, 8704, 9212, 9213, 9214, 9216, 9217, 10232, 10233, 10234, 10240, 10241, 16381, 17405, 17406])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_that_end_about_where_a_piece_does(vocab, dtype):
    check(make([3, 0, 2], vocab, dtype, seed=vocab))
    check(make([2, 1], vocab, dtype, seed=vocab, pad=3))


def test_as_many_sequences_as_a_call_takes():
    """Every sequence's rows are found among 65535, ragged, with empty ones among them."""
    g = np.random.default_rng(3)
    for vocab in (3, 4100):
        n = 65535 if vocab == 3 else 5000
        drafted = g.integers(0, 3, n)
        b = make([0], vocab, seed=24, temperature=0.0)
        start = np.concatenate([[0], np.cumsum(drafted)]).astype(np.int32)            # 0, 1 or 2 rows
        rows = int(start[-1])
        best = g.integers(0, vocab, rows)
        x = torch.zeros(rows, vocab, device="cuda")
        x[torch.arange(rows), torch.from_numpy(best).cuda()] = 1.0
        b.update(start=start, logits=x, draft_logits=None, draft=torch.from_numpy(best.astype(np.int32)), u_accept=torch.zeros(rows),
                 u_token=torch.zeros(n), temperature=torch.zeros(n))
        accepted, token, _ = run(b)
        np.testing.assert_array_equal(accepted, np.maximum(drafted - 1, 0))
        np.testing.assert_array_equal(token, np.where(drafted > 0, best[np.minimum(start[1:] - 1, rows - 1)], -1))


def test_long_drafts_and_large_vocabularies():
    check(make([40, 100, 0], 400, seed=6, sharp=1.0))
    check(make([2, 1], 151000, seed=7))
    check(make([1], 300001, seed=8, with_draft=False))
    for dtype in (torch.float32, torch.bfloat16):                   # more than the blocks' shared memory keeps
        check(make([1, 0, 2], 400003, dtype, seed=22))
        check(make([1, 2], 900001, dtype, seed=23, with_draft=False, temperature=2.0))


def test_the_same_draw_wherever_it_is_computed():
    """Weights in 32 bits, their sums exact beyond 32: the token that 64-bit sums of the same weights give."""
    b = make([2] * 40 + [0] * 40, 5000, seed=9, sharp=1.0)          # flat: many edges to fall on either side of
    accepted, token, _ = check(b)
    start, t = torch.from_numpy(b["start"]).long(), b["temperature"].cuda()

    def soft(x):
        x = x * (1 / t)[:, None]
        e = torch.exp(x - x.amax(-1, keepdim=True))
        return e * (1 / e.sum(-1, dtype=torch.float64, keepdim=True)).float()

    at = start[:-1] + torch.from_numpy(accepted).long()
    refused = (at < start[1:] - 1).cuda()
    p, q = soft(b["logits"].cuda()[at]), soft(b["draft_logits"].cuda()[at])
    w = torch.where(refused[:, None], (p - q).clamp(min=0), p)
    c = w.double().cumsum(-1)
    want = (c <= b["u_token"].cuda().double()[:, None] * c[:, -1:]).sum(-1)
    np.testing.assert_array_equal(token, want.cpu().numpy())
    assert refused.any() and not refused.all()


@pytest.mark.parametrize("sequences", [3, 152, 153, 310])
@pytest.mark.parametrize("vocab", [517, 4095, 4096, 4097])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_vocabularies_of_few_and_many_sequences(sequences, vocab, dtype):
    """On both sides of where the rows' sums are made elsewhere, and of where blocks are smaller; rows that start anywhere."""
    g = np.random.default_rng(sequences + vocab)
    drafted = [int(x) for x in g.integers(0, 5, sequences)]
    b = make(drafted, vocab, dtype, seed=vocab, sharp=2.0)
    b["temperature"] = torch.from_numpy(np.where(g.random(sequences) < 0.2, 0.0, g.uniform(0.3, 1.4, sequences)).astype(np.float32))

    def odd(t):
        t = t.cuda()
        w = torch.full((t.shape[0], t.shape[1] + 5), 9e3, dtype=t.dtype, device="cuda")
        w[:, 3:-2] = t
        return w[:, 3:-2]

    usual = run(b)
    check(b, usual)
    # where a row starts within 16 bytes decides which logits a thread sums, and a sum of other fp32 partial sums is another
    # rounding of the same number: 4097 logits, 0.0952981561 for 0.0952981487, one step of 2^-27
    check(b, run(b, move=odd))
    few = dict(b, start=b["start"][: 3], temperature=b["temperature"][: 2], u_token=b["u_token"][: 2])
    for got, want in zip(run(few)[:2], usual):
        np.testing.assert_array_equal(got, want[:2])                        # however many sequences there are


def test_a_draft_equal_to_the_target_is_always_taken():
    for vocab in (50, 3001, 20000):
        b = make([6] * 20, vocab, seed=10)
        b["draft_logits"] = b["logits"].clone()
        b["u_accept"][:] = 1 - 2.0 ** -24
        assert (run(b)[0] == 6).all()


def test_ends_of_the_uniforms():
    b = make([0] * 6, 700, seed=11)
    b["u_token"] = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 7.0, -3.0, NAN])
    _, token, _ = run(b)
    assert token[0] == token[4] == token[5] == 0
    # 1 and above count as 1 - 2^-24, which the last token's probability need not reach: float64's own draw at that number
    for i in (1, 2, 3):
        p, _ = ref.softmax(wide(b["logits"])[i], 0.9)
        c = np.cumsum(p)
        assert token[i] == np.flatnonzero(c > (1 - 2.0 ** -24) * c[-1])[0] >= 697
    b = make([3] * 4, 700, seed=12, with_draft=False)
    b["u_accept"][:] = 0.0
    assert (run(b)[0] == 3).all()
    b["u_accept"][:] = 1.0                                          # nothing certain: nothing taken
    accepted, token, _ = run(b)
    assert (accepted == 0).all() and (token != b["draft"].numpy()[b["start"][:-1]]).all()


def test_masked_logits():
    """NaN, infinities and the type's lowest value: no probability, or all of it."""
    for dtype in (torch.float32, torch.bfloat16):
        low = torch.finfo(dtype).min
        b = make([2, 2, 2, 2, 0, 0, 0, 1], 900, dtype, seed=13, sharp=1.0)
        x, y = b["logits"], b["draft_logits"]
        keep = torch.zeros(900, dtype=torch.bool)
        keep[[5, 17, 800]] = True
        for r, v in ((0, low), (3, -INF), (6, NAN)):
            x[r, ~keep] = v
            b["draft"][r] = 17
        y[0, ~keep] = low
        y[3, ~keep] = -INF
        x[9, [100, 200]] = INF                                      # sequence 3: two tokens share it all
        b["draft"][9] = 100
        x[12] = -INF                                                # sequences without any distribution
        x[13] = low
        x[14] = NAN
        x[15] = -INF
        accepted, token, prob = run(b)
        want, p = ref.verify(b["start"], wide(x), b["draft"].numpy(), b["u_accept"].numpy(), b["u_token"].numpy(),
                             b["temperature"].numpy(), wide(y))
        for i in range(4):
            assert accepted[i] == want[i]["accepted"], i
        assert token[4] == token[5] == token[6] == -1
        assert accepted[7] == 0 and token[7] == -1 and prob[15] == 0
        assert abs(prob[9] - 0.5) < 1e-6
        for r in (0, 3, 6):
            assert abs(prob[r] - p[r]) < 1e-5 and p[r] > 0.05
        for i, r in ((0, 0), (1, 3), (2, 6)):
            if accepted[i] == 0:
                assert token[i] in (5, 17, 800)


def test_greedy_ties_go_to_the_lowest_index():
    for vocab in (40, 9000, 20000):
        x = torch.zeros(4, vocab)
        x[0, [vocab - 1, 30, 7]] = 2.0
        x[1, [31, 39]] = 5.0
        x[2] = -3.0
        x[3, vocab - 2] = INF
        b = make([2, 0], vocab, seed=14, temperature=0.0)
        b["logits"], b["draft"] = x, torch.tensor([7, 31, 0, 0], dtype=torch.int32)
        accepted, token, _ = run(b)
        assert accepted.tolist() == [2, 0] and token.tolist() == [0, vocab - 2]
        b["draft"][1] = 39
        accepted, token, _ = run(b)
        assert accepted.tolist() == [1, 0] and token[0] == 31


def test_tokens_outside_the_vocabulary_are_not_taken():
    for temperature in (0.0, 0.8):
        for with_draft in (False, True):
            for d in (-1, 300, 2 ** 31 - 1, -2 ** 31):
                b = make([2, 1], 300, seed=15, temperature=temperature, with_draft=with_draft)
                b["draft"][0] = d
                b["u_accept"][0] = 0.0
                accepted, token, prob = run(b)
                assert accepted[0] == 0 and 0 <= token[0] < 300 and prob[0] == 0


def test_starts_out_of_order_and_empty_sequences():
    b = make([2, 1, 0], 100, seed=16, pad=2)
    assert b["start"].tolist() == [0, 3, 5, 6]
    for start in ([0, 3, 2, 6], [0, 3, 5, 9], [-1, 3, 5, 6], [0, 2 ** 31 - 1, 5, 6], [0, -5, 5, 6]):
        c = dict(b, start=np.array(start, np.int32))
        accepted, token, _ = run(c)
        assert (accepted == -1).all() and (token == -1).all()
    c = dict(b, start=np.array([0, 3, 3, 6], np.int32))
    accepted, token, prob = run(c)
    assert accepted[1] == 0 and token[1] == -1
    check(c, (accepted, token, prob))
    check(dict(b, start=np.array([1, 3, 5, 6], np.int32)))          # a first row that belongs to nobody


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(dtype):
    b = make([3, 1, 2], 1001, dtype, seed=17)
    want = run(b)
    for pad, lead in ((0, 1), (7, 3), (3, 0), (1, 5)):
        def move(t):
            pool = torch.full((t.shape[0], t.shape[1] + pad + lead), NAN, dtype=t.dtype, device="cuda")
            pool[:, lead:lead + t.shape[1]] = t.cuda()
            return pool[:, lead:lead + t.shape[1]]
        got = run(b, move=move)
        check(b, got)
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])


def test_streams_graphs_workspaces_and_repeats():
    b = make([4, 0, 2, 7], 9001, seed=18)
    n, rows = 4, len(b["logits"])
    need = cp.verify_workspace_bytes(n, rows, 9001)
    assert need > 0
    want = run(b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(b, stream=side, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    for x, y in zip(want, got):
        np.testing.assert_array_equal(x, y)
    d = {k: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v).cuda() for k, v in b.items()}
    outs = [[torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2)] for _ in range(2)]
    graphs = []
    for accepted, token in outs:
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cp.verify(d["logits"], d["draft"], d["start"], d["u_accept"], d["u_token"], d["temperature"], accepted, token,
                      draft_logits=d["draft_logits"], workspace=ws)
        graphs.append((graph, ws))
    for seed in (19, 20):
        c = make([4, 0, 2, 7], 9001, seed=seed)
        for k in ("logits", "draft_logits", "draft", "u_accept", "u_token"):
            d[k].copy_(c[k])
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = check(c)
        for accepted, token in outs:
            np.testing.assert_array_equal(accepted.cpu().numpy(), want[0])
            np.testing.assert_array_equal(token.cpu().numpy(), want[1])


def test_the_distribution_of_what_comes_out():
    """The first token behind the accepted ones follows the target, whatever the draft: chi-square over 4000 sequences."""
    g = torch.Generator().manual_seed(21)
    n, vocab = 4000, 6
    x, y = torch.randn(vocab, generator=g), torch.randn(vocab, generator=g)
    p, q = torch.softmax(x / 0.9, 0), torch.softmax(y / 0.9, 0)
    b = dict(start=np.arange(0, 2 * n + 1, 2).astype(np.int32), logits=x.expand(2 * n, vocab).contiguous(),
             draft_logits=y.expand(2 * n, vocab).contiguous(),
             draft=torch.multinomial(q, 2 * n, True, generator=g).to(torch.int32),
             u_accept=torch.rand(2 * n, generator=g), u_token=torch.rand(n, generator=g), temperature=torch.full((n,), 0.9))
    accepted, token, _ = run(b)
    first = np.where(accepted == 1, b["draft"].numpy()[::2], token)
    seen = np.bincount(first, minlength=vocab)
    chi = ((seen - n * p.numpy()) ** 2 / (n * p.numpy())).sum()
    assert chi < 27.9                                                # the inputs are fixed; 1 in 25000 of random ones would pass it


def test_refusals():
    b = make([1], 5000)
    args = [b["logits"].cuda(), b["draft"].cuda(), torch.from_numpy(b["start"]).cuda(), b["u_accept"].cuda(), b["u_token"].cuda(),
            b["temperature"].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")]
    cp.verify(*args)
    for k, wrong in ((0, args[0].half()), (0, args[0].cpu()), (1, args[1].long()), (1, args[1][:1]), (2, args[2][:1]), (3, args[3].double()),
                     (4, args[4].cpu()), (5, args[5].half()), (7, torch.zeros(2, dtype=torch.int32, device="cuda"))):
        bad = list(args)
        bad[k] = wrong
        with pytest.raises(ValueError):
            cp.verify(*bad)
    with pytest.raises(ValueError):
        cp.verify(*args, draft_logits=args[0].bfloat16())
    with pytest.raises(ValueError):
        cp.verify(*args, draft_logits=args[0][:1].expand(2, 5000))
    with pytest.raises(cp.CPError):
        cp.verify(*args, workspace=torch.zeros(15, dtype=torch.uint8, device="cuda"))
    with pytest.raises(cp.CPError):
        cp.verify(*args, workspace=torch.zeros(1000, dtype=torch.uint8, device="cuda")[1:])
