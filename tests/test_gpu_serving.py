"""The operators of a serving loop together: prompts are forked, grown and written, steps with drafted tokens run through
4-bit projections, the paged cache and verification, refused positions are trimmed and the pool is compacted. Each stage is
compared with float64 on the inputs that it got; what the cache holds at the end, with every row that was written."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from oracle import cache as cref
from oracle import linear as lref
from oracle.pages import Pool
from persistent_megakernel_streaming_gb300 import cp
from test_gpu_linear import check as check_linear
from test_gpu_verify import check as check_verify

pytestmark = pytest.mark.gpu

HIDDEN, HQ, HKV, D, FFN, VOCAB, PAGE, EPS = 256, 4, 2, 64, 384, 500, 16, 1e-6


def wide(t):
    return t.float().double().cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Projection:
    def __init__(self, g, n, k, group, zero, gated=False):
        q = g.integers(0, 256, (n, k // 2)).astype(np.uint8)
        scale = torch.from_numpy((np.exp(0.2 * g.standard_normal((n, k // group))) * 0.25 / np.sqrt(k)).astype(np.float32)).to(torch.bfloat16)
        z = g.integers(5, 11, (n, k // group)).astype(np.uint8) if zero else None
        self.w, self.gated = lref.weights(q, wide(scale), z), gated
        self.lin = cp.Linear(torch.from_numpy(q).cuda(), scale.cuda(), None if z is None else torch.from_numpy(z).cuda(), gated=gated)

    def __call__(self, x, dtype, add=None):
        out = torch.empty((x.shape[0], self.lin.outs), dtype=dtype, device="cuda")
        self.lin.apply(x, out, add=add)
        check_linear(out, *lref.apply(wide(x), self.w, self.gated, None if add is None else wide(add)), dtype)
        return out


def norm(x, gain):
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()).to(torch.bfloat16)


class Talker:
    """One layer over a pool of pages, and everything that it is told, kept beside it."""

    def __init__(self, dtype, sequences, pages, width, seed):
        g = np.random.default_rng(seed)
        self.embed = torch.from_numpy(g.standard_normal((VOCAB, HIDDEN)).astype(np.float32)).cuda()
        self.qkv, self.o = Projection(g, (HQ + 2 * HKV) * D, HIDDEN, 64, True), Projection(g, HIDDEN, HQ * D, 128, False)
        self.gate_up, self.down = Projection(g, 2 * FFN, HIDDEN, 32, False, gated=True), Projection(g, HIDDEN, FFN, 64, True)
        self.head = Projection(g, VOCAB, HIDDEN, 128, False)
        self.gains = [(1 + 0.1 * torch.randn(n, device="cuda")).to(torch.bfloat16) for n in (HIDDEN, HIDDEN, HIDDEN, D)]
        shape = (pages, HKV, PAGE, D)
        self.table, self.length, self.refs = i32(np.full((sequences, width), -1)), i32(np.zeros(sequences)), i32(np.zeros(pages))
        if dtype == "bf16":
            self.cache = cp.Cache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        else:
            self.cache = cp.Cache(*(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)),
                                  *(torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)))
        self.pool, self.plain = cp.Pages(self.refs, self.table, self.length, PAGE), Pool(np.zeros(pages), self.table.cpu().numpy(), np.zeros(sequences), PAGE)
        self.moves, self.count = i32(np.zeros((max(sequences, pages // 2), 2))), i32([0])
        self.rows = [[] for _ in range(sequences)]       # what was written: (k, v) of each position
        self.n = sequences

    def same(self, moves=None):
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.plain.table)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.plain.refs)
        np.testing.assert_array_equal(self.length.cpu().numpy(), self.plain.length)
        assert self.pool.status() == 0 and self.cache.status() == 0 and not self.plain.bad
        if moves is not None:
            assert int(self.count) == len(moves) and self.moves[: len(moves)].cpu().numpy().tolist() == [list(m) for m in moves]

    def fork(self, src, dst):
        self.pool.fork(i32(src), i32(dst))
        self.plain.fork(src, dst)
        for s, d in zip(src, dst):
            self.rows[d] = list(self.rows[s])
        self.same()

    def trim(self, keep):
        self.pool.trim(i32(keep))
        self.plain.trim(keep)
        self.rows = [r[:k] for r, k in zip(self.rows, keep)]
        self.same()

    def compact(self):
        self.pool.compact(self.moves, self.count)
        self.cache.copy(self.moves, self.count)
        moves, _ = self.plain.compact()
        self.same(moves)
        return moves

    def read(self):
        """Every sequence's cached rows."""
        length = self.length.cpu().numpy()
        start = np.concatenate([[0], np.cumsum(length)]).astype(np.int32)
        k, v = (torch.zeros((int(start[-1]), HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.cache.read(cp.Batch(i32(start), self.length, self.table, int(start[-1])), k, v)
        return [(k[a:b], v[a:b]) for a, b in zip(start[:-1], start[1:])]

    def run(self, tokens):
        """Logits of the new tokens [sequence][...], in fp32."""
        new = [len(t) for t in tokens]
        self.pool.grow(i32(new), self.moves, self.count)
        self.cache.copy(self.moves, self.count)
        moves, count = self.plain.grow(new)
        assert count >= 0
        self.same(moves)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = int(start[-1])
        batch = cp.Batch(i32(start), self.length, self.table, rows, max_new=max(new))
        x = self.embed[torch.from_numpy(np.concatenate([np.asarray(t, np.int64) for t in tokens])).cuda()]
        qkv = self.qkv(norm(x, self.gains[0]), torch.bfloat16)
        q, out = (torch.empty((rows, HQ, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.cache.append(batch, qkv, q, q_norm=self.gains[3], k_norm=self.gains[3], rope_base=1e4)
        self.cache.attend(batch, q, out)
        held = self.read()
        for i, (k, v) in enumerate(held):
            self.rows[i] += [(k[len(k) - new[i] + j].clone(), v[len(v) - new[i] + j].clone()) for j in range(new[i])]
            if not new[i]:
                continue
            r, length = slice(start[i], start[i + 1]), len(k)
            y, size, reach = cref.attend(wide(q[r]), wide(k), wide(v), length - new[i], D ** -0.5, True, 0)
            rel = 2 * (D + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + 2.0 ** -8 + length * 2.0 ** -24
            tol = np.abs(y) * 2.0 ** -8 + size * rel * 1.01 + 2.0 ** -25 * length * float(v.abs().max())
            assert (np.abs(wide(out[r]) - y) <= tol).all()
        x = self.o(out.view(rows, HQ * D), torch.float32, add=x)
        x = self.down(self.gate_up(norm(x, self.gains[1]), torch.bfloat16), torch.float32, add=x)
        return self.head(norm(x, self.gains[2]), torch.float32), start


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_drafted_steps_of_forked_prompts(dtype):
    g = np.random.default_rng(7)
    t = Talker(dtype, 6, 40, 12, 1)
    prompts = [list(g.integers(0, VOCAB, n)) for n in (37, 16)]
    logits, start = t.run(prompts + [[]] * 4)
    t.fork([0, 0, 1], [2, 3, 4])                          # sequence 5 stays empty
    live = [0, 1, 2, 3, 4]
    last = {i: int(g.integers(0, VOCAB)) for i in live}   # a first token each: the branches part
    taken = 0                                             # by verification, whatever of it had been run
    for step in range(6):
        drafts = {i: list(g.integers(0, VOCAB, int(g.integers(0, 5)))) for i in live}
        before = t.length.cpu().numpy().copy()
        logits, start = t.run([[last[i]] + drafts[i] if i in drafts else [] for i in range(t.n)])
        # a draft that often agrees: the target's best token in place of some guesses
        best = logits.argmax(-1).cpu().numpy()
        draft = np.zeros(len(logits), np.int32)
        for i in live:
            for j in range(len(drafts[i])):
                draft[start[i] + j] = drafts[i][j]
        b = dict(start=start, logits=logits.cpu(), draft_logits=None, draft=torch.from_numpy(draft),
                 u_accept=torch.from_numpy(g.random(len(logits), np.float32) * (0.02 if step % 2 else 1)),
                 u_token=torch.from_numpy(g.random(t.n, np.float32)),
                 temperature=torch.tensor([0.0 if i == 1 else 0.8 for i in range(t.n)]))
        if step == 2:                                     # the greedy sequence's own continuation, all of it taken
            for j in range(len(drafts[1])):
                b["draft"][start[1] + j] = int(best[start[1] + j])
        accepted, token, _ = check_verify(b)
        assert accepted[5] == 0 and token[5] == -1
        keep = []
        for i in range(t.n):
            if i not in live:
                keep.append(2 ** 31 - 1)
                continue
            # positions behind the last accepted token are given up (its drafts were run as they stood)
            ran = drafts[i]
            agree = 0
            while agree < accepted[i] and int(b["draft"][start[i] + agree]) == ran[agree]:
                agree += 1
            keep.append(int(before[i]) + 1 + agree)
            last[i] = int(token[i])
            taken += int(accepted[i])
        t.trim(keep)
        if step == 3:                                     # two sequences end, a branch of another comes
            t.trim([0 if i in (1, 3) else 2 ** 31 - 1 for i in range(t.n)])
            t.fork([2], [1])
            live = [0, 1, 2, 4]
            last[1] = int(g.integers(0, VOCAB))
            assert t.compact()
    assert taken > 0
    t.compact()
    assert (t.refs[int((t.refs != 0).sum()):] == 0).all()
    for (k, v), rows in zip(t.read(), t.rows):
        assert len(k) == len(rows)
        for j, (a, b) in enumerate(rows):
            assert torch.equal(k[j], a) and torch.equal(v[j], b)


def test_a_captured_step_follows_lengths_and_tables():
    """Growing, projecting, writing and attending captured once and replayed: page tables and lengths change from replay to
    replay, and the results are those of the calls made one by one."""
    a, b = Talker("bf16", 3, 30, 8, 3), Talker("bf16", 3, 30, 8, 3)
    b.gains = a.gains
    g = np.random.default_rng(8)
    for t in (a, b):
        t.run([[1, 2, 3, 4, 5], [6] * 17, []])
        t.fork([1], [2])
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    add, start = i32([1, 1, 1]), i32([0, 1, 2, 3])
    outs = [torch.zeros((3, HQ, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(t, out, workspace):
        t.pool.grow(add, t.moves, t.count)
        t.cache.copy(t.moves, t.count)
        batch = cp.Batch(start, t.length, t.table, 3, max_new=1, max_len=8 * PAGE)
        qkv = torch.empty((3, (HQ + 2 * HKV) * D), dtype=torch.bfloat16, device="cuda")
        t.qkv.lin.apply(norm(t.embed[ids], t.gains[0]), qkv)
        q = torch.empty((3, HQ, D), dtype=torch.bfloat16, device="cuda")
        t.cache.append(batch, qkv, q, q_norm=t.gains[3], k_norm=t.gains[3], rope_base=1e4)
        t.cache.attend(batch, q, out, workspace=workspace)

    spaces = [torch.zeros(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    step(b, outs[1], spaces[1])                           # everything loaded before the capture
    b.pool.trim(i32([5, 17, 17]))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(a, outs[0], spaces[0])
    step(a, outs[0], spaces[0])
    a.pool.trim(i32([5, 17, 17]))
    for k in range(40):
        ids.copy_(torch.from_numpy(g.integers(0, VOCAB, 3)))
        graph.replay()
        step(b, outs[1], spaces[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]), k
        assert torch.equal(a.length, b.length) and int(a.length[0]) == 6 + k
    assert a.pool.status() == b.pool.status() == a.cache.status() == b.cache.status() == 0
