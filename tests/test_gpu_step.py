"""The operators that close a decode step on the GPU against the fp64 oracle: verification of drafted tokens, page tables,
copying and compacting pages, microscaled 4-bit floating point, and a step that runs them together."""
import numpy as np
import pytest

import synth
import tenant_rank_serving_amd as trs
from gpu_util import dev_i32, note, torch
from oracle import step

pytestmark = pytest.mark.gpu

# One rounding to bf16 is off by at most 2^-8 of the value (half a step of eps 2^-7).
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    trs.lib()


def bits(a):
    return synth.to_bf16_bits(np.asarray(a, np.float32))


def vals(b):
    return synth.bf16_bits_to_f32(np.asarray(b, np.uint16)).astype(np.float64)


def dev_bits(b):
    t = torch()
    return t.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(t.bfloat16)


def host_bits(x):
    t = torch()
    return x.contiguous().view(t.int16).cpu().numpy().view(np.uint16)


def dev_f32(a):
    return torch().from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


# ----------------------------------------------------------- verification
class Verify:
    """Logits of sequences of nq rows; `extra` rows in front and behind belong to none."""

    def __init__(self, seed, nq, vocab, dtype, draft, temperature="mixed", extra=(0, 0), pad=0, hot=4.0):
        t = torch()
        rng = np.random.default_rng(seed)
        self.vocab, self.b = vocab, len(nq)
        self.q_start = extra[0] + np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        n = self.n = int(self.q_start[-1]) + extra[1]
        x = rng.normal(size=(n, vocab)) * 2
        x[np.arange(n), rng.integers(0, vocab, n)] += hot
        y = x + rng.normal(size=(n, vocab)) * 0.8
        if dtype == "bf16":
            self.x, self.y = vals(bits(x)), vals(bits(y))
        else:
            self.x, self.y = (a.astype(np.float32).astype(np.float64) for a in (x, y))
        self.dtype, self.draft, self.pad = dtype, draft, pad
        self.temp = {"mixed": np.where(np.arange(self.b) % 3 == 1, 0.0, rng.uniform(0.4, 1.5, self.b)), "none": None,
                     "hot": rng.uniform(0.4, 1.5, self.b)}[temperature]
        if self.temp is not None:
            self.temp = self.temp.astype(np.float32).astype(np.float64)
        self.accept = rng.random(n).astype(np.float32)
        self.pick = rng.random(self.b).astype(np.float32)
        drawn = (self.y + rng.gumbel(size=self.y.shape)).argmax(1)
        self.tokens = np.roll(drawn, 1).astype(np.int32)
        for b in range(0, self.b, 2):    # so that whole rows of drafts stand too
            r = np.arange(self.q_start[b], self.q_start[b + 1] - 1)
            self.tokens[r + 1] = self.x[r].argmax(1)
            self.accept[r] *= 0.02

    def logits(self, a):
        """On the device, rows `pad` elements apart from each other; the room between holds NaN."""
        t = torch()
        wide = np.full((self.n, self.vocab + self.pad), np.nan)
        wide[:, :self.vocab] = a
        d = dev_bits(bits(wide)) if self.dtype == "bf16" else dev_f32(wide)
        return d[:, :self.vocab]

    def upload(self):
        t = torch()
        self.batch = trs.VerifyBatch(dev_i32(self.q_start), dev_i32(self.tokens), dev_f32(self.accept), dev_f32(self.pick),
                                     None if self.temp is None else dev_f32(self.temp))
        self.target = self.logits(self.x)
        self.dr = None
        if self.draft:
            y = self.y.copy()
            last = self.q_start[1:][self.q_start[1:] > self.q_start[:-1]] - 1
            y[last] = np.nan                                     # not read
            self.dr = self.logits(y)
        self.out = t.full((self.n,), -7, dtype=t.int32, device="cuda")
        self.prob = t.full((self.n,), -7.0, device="cuda")
        self.count = t.full((self.b,), -7, dtype=t.int32, device="cuda")
        self.ws = t.full((trs.dc_verify_workspace_bytes(self.vocab, self.n, self.b),), 0xA5, dtype=t.uint8, device="cuda")
        return self

    def run(self):
        trs.dc_verify_drafts(self.batch, self.target, self.dr, self.out, self.count, self.ws, self.prob)

    def reference(self):
        return step.verify(self.x, self.y if self.draft else None, self.q_start, self.tokens, self.accept, self.pick, self.temp)

    def compare(self):
        out, prob, count, margin = self.reference()
        # both sides are good to about 1e-13 of the sums: nothing may lie nearer to a border
        assert margin > 1e-11, margin
        got, gp = self.out.cpu().numpy(), self.prob.cpu().numpy().astype(np.float64)
        assert self.count.cpu().numpy().tolist() == count
        assert got.tolist() == [-7 if o is None else o for o in out]
        want = np.array([-7.0 if p is None else p for p in prob])
        assert (np.abs(gp - want) <= 2.0 ** -24 * np.abs(want) * (1 + 1e-6) + 2.0 ** -149).all()   # one rounding to fp32

    def check(self):
        self.upload()
        self.run()
        torch().cuda.synchronize()
        self.compare()
        return self


VERIFY = [
    # nq, vocab, dtype, draft, temperature, extra, pad
    ([1], 1, "bf16", False, "none", (0, 0), 0),
    ([1], 7, "f32", False, "hot", (0, 0), 0),
    ([3], 2, "bf16", True, "hot", (0, 0), 0),
    ([1], 32000, "bf16", False, "none", (0, 0), 0),
    ([5, 0, 1, 3, 9], 1000, "bf16", True, "mixed", (2, 3), 24),
    ([5, 0, 1, 3, 9], 1003, "bf16", True, "mixed", (2, 3), 0),
    ([5, 0, 1, 3, 9], 1003, "f32", False, "mixed", (1, 0), 2),
    ([2, 2, 2, 2], 2049, "f32", True, "hot", (0, 1), 1),
    ([17, 33, 16], 300, "bf16", True, "hot", (0, 0), 3),
    ([20] * 3, 8193, "bf16", False, "mixed", (0, 0), 8),
    ([6] * 40, 50257, "bf16", True, "mixed", (0, 0), 0),
    ([4] * 70, 33333, "f32", True, "hot", (0, 0), 0),
]


@pytest.mark.parametrize("nq,vocab,dtype,draft,temperature,extra,pad", VERIFY)
def test_verify(nq, vocab, dtype, draft, temperature, extra, pad):
    note("verify", len(nq), vocab, dtype, draft, temperature, extra, pad)
    Verify(vocab + len(nq), nq, vocab, dtype, draft, temperature, extra, pad).check()


def test_verify_masks_and_rows_without_a_distribution():
    note("verify, masks")
    v = Verify(3, [4] * 12, 4099, "bf16", True, "hot")
    rng = np.random.default_rng(5)
    v.x[rng.random(v.x.shape) < 0.7] = -np.inf               # most of the vocabulary is not allowed
    v.x[:, 4000:] = -np.inf
    s = v.q_start
    v.tokens[s[0] + 1] = -1                                  # tokens outside the vocabulary
    v.tokens[s[1] + 1] = 4099
    v.tokens[s[2] + 1] = 4050                                # one that is not allowed
    v.x[s[3]] = -np.inf                                      # nothing is
    v.x[s[4] + 1, 77] = np.nan
    v.x[s[5], 4098] = np.inf
    v.y[s[6]] = -np.inf                                      # rows of the draft without a distribution
    v.y[s[7], 5] = np.nan
    v.y[s[8]] = v.x[s[8]]                                    # equal rows: whatever is drawn stands
    v.tokens[s[8] + 1] = v.x[s[8]].argmax()
    v.x[s[9]:s[10]] = -np.inf                                # one token is left
    v.x[s[9]:s[10], 4098] = 3.0
    v.temp[10], v.temp[11] = np.inf, 1e-30
    v.check()


@pytest.mark.parametrize("nq,vocab,dtype,draft", [
    ([1], 150001, "bf16", False), ([2, 1], 150001, "f32", True), ([3] * 5, 300001, "bf16", True), ([1, 2, 2, 3], 600007, "f32", False)])
def test_verify_many_pieces(nq, vocab, dtype, draft):
    """More pieces of a row than lanes of a wave, of each of the sizes."""
    note("verify, many pieces", nq, vocab, dtype, draft)
    for seed in (1, 2, 3):
        Verify(seed, nq, vocab, dtype, draft, "hot", hot=0.0).check()


@pytest.mark.parametrize("b,vocab,dtype", [(6, 5003, "bf16"), (6, 5003, "f32"), (64, 70001, "bf16"), (64, 70001, "f32")])
def test_verify_looked_up_drafts_of_likely_tokens(b, vocab, dtype):
    """Drafts without logits that have nearly all or all of the probability and fall: the rest of the row, or the draft."""
    note("verify, likely", b, vocab, dtype)
    v = Verify(b, [2] * b, vocab, dtype, False, "hot")
    rng = np.random.default_rng(b)
    v.accept[:] = np.nan                                     # no draft stands
    rows = np.arange(0, 2 * b, 2)
    at = rng.integers(0, vocab, b)
    at[:4] = [0, vocab - 1, 2047, 4096]
    v.tokens[rows + 1] = at
    lift = np.resize([0.0, 12.0, 24.0, 40.0], b)             # 40 T: the rest has 1e-13 of it
    v.x[rows, at] = 12.0 + lift
    alone = rows[4::5]
    v.x[alone] = -np.inf                                     # nothing is left
    v.x[alone, at[4::5]] = 1.0
    if dtype == "bf16":
        v.x = vals(bits(v.x))
    v.check()
    out = v.out.cpu().numpy()
    assert (out[alone] == at[4::5]).all() and (np.delete(out[rows], np.s_[4::5]) != np.delete(at, np.s_[4::5])).all()


@pytest.mark.parametrize("vocab,dtype,pad,shift", [(5003, "f32", 3, 0.0), (5003, "bf16", 1, 0.0), (40, "f32", 1, 4.0), (12001, "f32", 0, 4.0),
                                                   (70001, "bf16", 8, 0.0), (70001, "f32", 5, 4.0)])
def test_verify_draft_distribution_equal_to_the_target(vocab, dtype, pad, shift):
    """Equal distributions whose sums round differently (rows that lie differently, logits a constant apart): nothing is
    left of p - q, and where a draft falls all the same p is drawn from."""
    t = torch()
    note("verify, p = q", vocab, dtype, pad, shift)
    b = 32
    v = Verify(vocab, [2] * b, vocab, dtype, True, "hot")
    v.x = np.round(v.x * 16) / 16                            # so that the constant is added exactly
    v.x[:, 5] = -np.inf
    if dtype == "bf16":
        v.x = vals(bits(v.x))
    v.y = v.x + shift
    rows = v.q_start[:-1]
    v.tokens[rows + 1] = np.resize([-1, 5, vocab], b)        # outside the vocabulary, and one that neither allows
    v.upload()
    y = v.y.copy()
    wide = np.full((v.n, vocab + pad), np.nan)
    wide[:, :vocab] = y
    v.dr = (dev_bits(bits(wide)) if dtype == "bf16" else dev_f32(wide))[:, :vocab]
    v.run()
    t.cuda.synchronize()
    v.compare()


@pytest.mark.parametrize("eps", [1e-1, 1e-3, 1e-5])
def test_verify_draft_distribution_close_to_the_target(eps):
    """Draft logits that differ from the target's by little: what is left of p - q is small beside p, whose rounding
    (1e-13 of its sum) moves the borders by more of it."""
    note("verify, close", eps)
    b, vocab = 48, 701
    v = Verify(14, [2] * b, vocab, "f32", True, "hot")
    v.y = (v.x + np.random.default_rng(3).normal(size=v.x.shape) * eps).astype(np.float32).astype(np.float64)
    v.accept[:] = np.nan                                     # no draft stands
    v.upload()
    v.run()
    torch().cuda.synchronize()
    out = v.out.cpu().numpy().reshape(b, 2)
    for i in range(b):
        p, q = (step.distribution(a[2 * i], v.temp[i]) for a in (v.x, v.y))
        left = np.maximum(p - q, 0.0)
        token, margin = step.pick(left, v.pick[i])
        assert margin * left.sum() > 1e-12                   # ten times the rounding
        assert out[i].tolist() == [token, -1], i


def test_verify_greedy_ties_and_masks():
    note("verify, greedy")
    v = Verify(4, [3] * 6, 9001, "f32", True, "hot")
    v.temp[:] = [0.0, -1.0, np.nan, 0.0, 0.0, 0.0]
    s = v.q_start
    for b in range(6):
        top = v.x[s[b]:s[b + 1]].max() + 1
        v.x[s[b]:s[b + 1], [8999, 4000 + b, 9000]] = top     # the lowest of three
        v.tokens[s[b] + 1] = 4000 + b
        v.tokens[s[b] + 2] = 8999 if b % 2 else 4000 + b
    v.x[s[3] + 1] = -np.inf
    v.x[s[4], 3] = np.nan
    v.accept[:] = 1.0
    v.check()
    assert v.out.cpu().tolist()[:3] == [4000, 4000, 4000] and v.count.cpu().tolist() == [3, 2, 3, 1, 0, 2]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verify_random_numbers_at_their_ends(dtype):
    note("verify, ends", dtype)
    v = Verify(6, [2] * 6, 5000, dtype, True, "hot")
    v.x[:, :3], v.x[:, 4990:] = -np.inf, -np.inf
    v.pick[:] = [0.0, 1.0, 1.5, -1.0, np.nan, 1 - 2.0 ** -24]
    v.accept[:] = 1.0
    v.accept[::2] = [np.nan] * 6                             # compares false: no draft stands
    v.upload()
    v.run()
    torch().cuda.synchronize()
    out = v.out.cpu().numpy().reshape(6, 2)
    assert (out[:, 1] == -1).all() and (v.count.cpu().numpy() == 1).all()
    p = np.stack([step.distribution(v.x[2 * b], v.temp[b]) for b in range(6)])
    q = np.stack([step.distribution(v.y[2 * b], v.temp[b]) for b in range(6)])
    some = [np.nonzero(np.maximum(p[b] - q[b], 0) > 1e-12)[0] for b in range(6)]
    for b, want in ((0, 0), (3, 0), (1, -1), (2, -1), (4, -1)):   # the first or the last that has weight
        assert out[b, 0] == some[b][want], b


@pytest.mark.parametrize("scale", [1e-38, 60.0, 1e5, 3e38])
def test_verify_logits_of_every_size(scale):
    note("verify, size", scale)
    v = Verify(8, [3] * 8, 3001, "f32", True, "hot", hot=0.0)
    f = scale / np.abs(np.concatenate([v.x, v.y])).max()
    v.x, v.y = ((a * f).astype(np.float32).astype(np.float64) for a in (v.x, v.y))
    v.check()


def test_verify_is_the_same_with_every_workspace_and_on_every_call():
    t = torch()
    note("verify, again")
    v = Verify(9, [5] * 20, 32000, "bf16", True).check()
    first = [x.clone() for x in (v.out, v.count, v.prob)]
    for fill in (0, 255, 1):
        v.ws.fill_(fill)
        v.out.fill_(-9)
        v.run()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(first, (v.out, v.count, v.prob)))
    out, count = t.zeros_like(v.out), t.zeros_like(v.count)
    trs.dc_verify_drafts(v.batch, v.target, v.dr, out, count, v.ws)   # no probabilities
    assert t.equal(out, first[0]) and t.equal(count, first[1])


def test_verify_captured_two_sizes_share_a_workspace():
    """Two captured calls, of one piece and of many pieces a row, one after the other in one workspace on another
    stream; replays follow the random numbers and logits that changed since."""
    t = torch()
    note("verify, captured")
    a, b = Verify(10, [3] * 4, 900, "bf16", True).upload(), Verify(11, [2] * 30, 30000, "f32", False).upload()
    a.ws = b.ws = t.empty(max(a.ws.numel(), b.ws.numel()), dtype=t.uint8, device="cuda")
    side, g = t.cuda.Stream(), t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(g, stream=side):
        a.run()
        b.run()
    for k in range(4):
        for v in (a, b):
            rng = np.random.default_rng(k)
            v.accept, v.pick = rng.random(v.n).astype(np.float32), rng.random(v.b).astype(np.float32)
            v.batch._keep[2].copy_(dev_f32(v.accept))
            v.batch._keep[3].copy_(dev_f32(v.pick))
            v.x = np.roll(v.x, 1, 1)
            v.target.copy_(v.logits(v.x))
            v.out.fill_(-7)
            v.prob.fill_(-7)
        t.cuda.synchronize()
        with t.cuda.stream(side):
            g.replay()
        t.cuda.synchronize()
        a.compare()
        b.compare()


@pytest.mark.parametrize("b", [255, 256, 257, 511, 513, 5000, 65535, 65537])
def test_verify_many_sequences(b):
    """Sequences in numbers around those whose starts a block looks at at once, empty ones among them."""
    t = torch()
    note("verify, many sequences", b)
    rng = np.random.default_rng(b)
    nq = rng.integers(0, 3, b)
    nq[:2], nq[-2:] = 0, rng.integers(0, 2, 2)
    vocab, q_start = 3, 4 + np.concatenate([[0], np.cumsum(nq)])
    n = int(q_start[-1]) + 5
    x = vals(bits(rng.normal(size=(n, vocab)) * 3))
    picks, accept = rng.random(b).astype(np.float32), rng.random(n).astype(np.float32)
    tokens, temp = rng.integers(0, vocab, n), np.resize([0.5, 1.0, 0.0, 2.0], b)
    batch = trs.VerifyBatch(dev_i32(q_start), dev_i32(tokens), dev_f32(accept), dev_f32(picks), dev_f32(temp))
    out, count = t.full((n,), -7, dtype=t.int32, device="cuda"), t.full((b,), -7, dtype=t.int32, device="cuda")
    ws = t.full((trs.dc_verify_workspace_bytes(vocab, n, b),), 0xA5, dtype=t.uint8, device="cuda")
    trs.dc_verify_drafts(batch, dev_bits(bits(x)), None, out, count, ws)
    want, _, wcount, margin = step.verify(x, None, q_start, tokens, accept, picks, temp)
    assert margin > 1e-11
    assert count.tolist() == wcount and out.tolist() == [-7 if o is None else o for o in want]


def shortest(call, before=lambda: None, times=5):
    """The shortest of some calls, us."""
    t = torch()
    best = float("inf")
    for _ in range(times):
        before()
        a, b = (t.cuda.Event(enable_timing=True) for _ in range(2))
        t.cuda.synchronize()
        a.record()
        call()
        b.record()
        t.cuda.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


def test_verify_work_grows_with_the_batch_not_with_its_square():
    """Four times as many sequences take about four times as long (10 times, where every row looks through all starts)."""
    t = torch()
    vocab, us = 8, []
    for n in (1 << 17, 1 << 19):
        note("verify, large batch", n, vocab)
        x = t.randn(n, vocab, device="cuda").bfloat16()
        batch = trs.VerifyBatch(t.arange(n + 1, dtype=t.int32, device="cuda"), t.zeros(n, dtype=t.int32, device="cuda"),
                                t.rand(n, device="cuda"), t.rand(n, device="cuda"))
        out, count = t.zeros(n, dtype=t.int32, device="cuda"), t.zeros(n, dtype=t.int32, device="cuda")
        ws = t.empty(trs.dc_verify_workspace_bytes(vocab, n, n), dtype=t.uint8, device="cuda")
        us.append(shortest(lambda: trs.dc_verify_drafts(batch, x, None, out, count, ws)))
        assert (count == 1).all()
    print("%.0f and %.0f us" % tuple(us))
    assert us[1] < 6 * us[0]


def test_verify_more_blocks_than_31_bits_of_threads():
    """Rows whose statistics take more than 2^31 threads: the counters that they clear on the way are those of the
    sequences, whatever a block's number."""
    t = torch()
    n, b, vocab = 4300000, 1000, 2
    note("verify, many rows", n, b, vocab)
    rng = np.random.default_rng(13)
    x, y = (t.from_numpy(rng.normal(size=(n, vocab)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
    q_start = (np.arange(b + 1) * (n // b)).astype(np.int32)
    tokens, picks = rng.integers(0, vocab, n).astype(np.int32), rng.random(b).astype(np.float32)
    accept = t.full((n,), float("nan"), device="cuda")       # no draft stands
    batch = trs.VerifyBatch(dev_i32(q_start), dev_i32(tokens), accept, dev_f32(picks))
    ws = t.full((trs.dc_verify_workspace_bytes(vocab, n, b),), 0xA5, dtype=t.uint8, device="cuda")
    out, count = t.zeros(n, dtype=t.int32, device="cuda"), t.zeros(b, dtype=t.int32, device="cuda")
    trs.dc_verify_drafts(batch, x, y, out, count, ws)
    t.cuda.synchronize()
    rows = (q_start[:-1, None] + np.arange(2)).reshape(-1)   # a sequence's first row and its draft decide
    px, py = (a[t.from_numpy(rows).cuda().long()].double().cpu().numpy() for a in (x, y))
    want, _, _, margin = step.verify(px, py, np.arange(0, 2 * b + 1, 2), tokens[rows], np.full(2 * b, np.nan), picks, None)
    assert margin > 1e-11
    got = out.cpu().numpy().reshape(b, -1)
    assert got[:, 0].tolist() == want[::2] and (got[:, 1:] == -1).all() and (count == 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verify_rows_behind_32_bits(dtype):
    """Rows whose offsets pass 2^32 elements."""
    t = torch()
    note("verify, far rows", dtype)
    v = Verify(15, [3, 2, 4], 2500, dtype, True, "hot").upload()
    stride = (1 << 29) + 16
    far = []
    for a in (v.target, v.dr):
        room = t.empty(stride * (v.n - 1) + 2500, dtype=a.dtype, device="cuda").as_strided((v.n, 2500), (stride, 1))
        far.append(room.copy_(a))
    assert stride * (v.n - 1) >= 1 << 32
    v.target, v.dr = far
    v.run()
    t.cuda.synchronize()
    v.compare()


def test_verify_binding_refusals():
    t = torch()
    v = Verify(12, [2, 2], 64, "f32", True).upload()
    z = lambda *s, **k: t.zeros(*s, **{**dict(device="cuda"), **k})  # noqa: E731
    for kw in (dict(target=v.target.double()), dict(target=v.target[:, :63]), dict(draft=v.dr.bfloat16()), dict(draft=v.dr[1:]),
               dict(target=z(64, 4).t()), dict(out=z(3, dtype=t.int32)), dict(out=z(4)), dict(count=z(3, dtype=t.int32)),
               dict(prob=z(4, dtype=t.float64)), dict(ws=t.zeros(1 << 20, dtype=t.uint8)), dict(out=t.zeros(4, dtype=t.int32))):
        f = {**dict(batch=v.batch, target=v.target, draft=v.dr, out=v.out, count=v.count, ws=v.ws, prob=v.prob), **kw}
        with pytest.raises(ValueError):
            trs.dc_verify_drafts(**f)
    with pytest.raises(trs.DcError):
        trs.dc_verify_drafts(v.batch, v.target, v.dr, v.out, v.count, v.ws[:256])
    with pytest.raises(ValueError):
        trs.VerifyBatch(z(4, dtype=t.int32), z(4, dtype=t.int32), z(4), z(2))
    empty = trs.VerifyBatch(z(1, dtype=t.int32), z(0, dtype=t.int32), z(0), z(0))
    trs.dc_verify_drafts(empty, z(0, 64), None, z(0, dtype=t.int32), z(0, dtype=t.int32), v.ws)
    none = trs.VerifyBatch(z(3, dtype=t.int32), z(0, dtype=t.int32), z(0), z(2))
    count = z(2, dtype=t.int32) + 5
    trs.dc_verify_drafts(none, z(0, 64), None, z(0, dtype=t.int32), count, v.ws)
    assert count.tolist() == [0, 0]


# ------------------------------------------------------------ page tables
class Table:
    """Tables on the device and the oracle's beside them."""

    def __init__(self, pages, kv_len, refs, page):
        t = torch()
        self.ref = step.Tables(np.asarray(pages).tolist(), list(map(int, kv_len)), list(map(int, refs)), page)
        self.pages, self.lens, self.refs = dev_i32(pages), dev_i32(kv_len), dev_i32(refs)
        self.table = trs.KvTable(self.pages, self.lens, self.refs, page)
        self.status = t.zeros(1, dtype=t.int32, device="cuda")
        self.copies = t.full((len(kv_len), 2), -5, dtype=t.int32, device="cuda")

    def resize(self, new):
        trs.dc_kv_resize(self.table, dev_i32(new), self.copies, self.status)
        copies = self.ref.resize(list(map(int, new)))
        self.check()
        assert self.copies.tolist() == copies

    def fork(self, src, dst):
        trs.dc_kv_fork(self.table, dev_i32(src), dev_i32(dst), self.status)
        self.ref.fork(list(map(int, src)), list(map(int, dst)))
        self.check()

    def check(self):
        assert self.lens.tolist() == self.ref.kv_len
        assert self.pages.tolist() == self.ref.pages
        assert self.refs.tolist() == self.ref.refs
        assert self.status.item() == trs.DC_KV_FULL * self.ref.full + trs.DC_KV_BAD * self.ref.bad


def start_table(rng, seqs, width, page, num_pages, held=0):
    refs = np.zeros(num_pages, np.int32)
    refs[rng.permutation(num_pages)[:held]] = rng.integers(1, 4, held)
    return Table(np.full((seqs, width), -1, np.int32), np.zeros(seqs, np.int32), refs, page)


@pytest.mark.parametrize("seqs,width,page,num_pages,held,seed", [
    (1, 1, 16, 1, 0, 0), (3, 4, 16, 9, 2, 1), (7, 20, 32, 131, 40, 2), (65, 9, 16, 700, 100, 3), (40, 70, 64, 4099, 3500, 4),
    (1500, 6, 16, 9001, 1000, 5), (5, 300, 1024, 20000, 19000, 6)])
def test_tables_walk(seqs, width, page, num_pages, held, seed):
    """Random growth, release and branching, pools that run out among them."""
    note("tables", seqs, width, page, num_pages)
    rng = np.random.default_rng(seed)
    t = start_table(rng, seqs, width, page, num_pages, held)
    most = width * page
    for k in range(12):
        lens = np.array(t.ref.kv_len)
        if k % 3 == 2:
            empty, some = np.nonzero(lens == 0)[0], np.nonzero(lens > 0)[0]
            n = min(empty.size, 1 + seqs // 3)
            if n and some.size:
                t.fork(rng.choice(some, n), rng.permutation(empty)[:n])
            continue
        new = np.where(rng.random(seqs) < 0.5, lens + rng.integers(0, 3 * page, seqs), lens)
        new = np.where(rng.random(seqs) < 0.2, rng.integers(0, most + 1, seqs), new)
        new = np.where(rng.random(seqs) < 0.25, 0, new)
        t.resize(np.clip(new, 0, most))
    t.resize(np.zeros(seqs, np.int32))
    assert (t.lens == 0).all() and (t.pages == -1).all()


@pytest.mark.parametrize("seqs,width,page,num_pages,held,seed", [
    (40, 200, 16, 32767, 9000, 7), (40, 200, 16, 32768, 28000, 8), (40, 200, 16, 32770, 9000, 9), (1100, 3, 32, 2501, 3, 10)])
def test_tables_give_back_many(seqs, width, page, num_pages, held, seed):
    """Long sequences closed in great numbers, in pools around the size up to which their pages are counted first."""
    test_tables_walk(seqs, width, page, num_pages, held, seed)


def test_tables_running_out():
    note("tables, running out")
    t = Table([[2, 5, -1, -1], [2, 5, -1, -1], [-1] * 4, [7, -1, -1, -1]], [20, 20, 0, 16], [1, 0, 2, 1, 1, 2, 0, 1, 0], 16)
    t.resize([40, 21, 16, 16])         # 0 needs an exchange and one more, 1 an exchange: three of three; 2 finds none
    assert t.status.item() == trs.DC_KV_FULL and t.lens.tolist() == [40, 21, 0, 16]
    t.status.zero_()
    t.ref.full = False
    t.resize([0, 0, 64, 16])           # what is given back can be taken in the same call
    assert t.status.item() == 0 and t.lens.tolist() == [0, 0, 64, 16]
    t.resize([64, 0, 64, 17])          # too few: what 0 was dealt goes back, and 3 gets none
    assert t.lens.tolist() == [0, 0, 64, 16]


def test_tables_numbers_out_of_range():
    """Lengths, rows and page numbers that cannot be: the sequence or entry is left out, nothing else is touched."""
    note("tables, out of range")
    t = Table([[0, 1], [99, -4], [2, 3], [-1, -1]], [32, 20, 40, 0], [1, 1, 1, 1, 0, 0], 16)
    t.resize([16, 0, 8, 16])           # row 2's length is no length; row 1 gives back pages that are none
    assert t.lens.tolist() == [16, 0, 40, 16] and t.status.item() == trs.DC_KV_BAD
    t.resize([33, -1, 0, 16])
    t.fork([0, 0, 4, -1, 0, 2], [0, 4, 1, 1, 3, 1])
    assert t.lens.tolist() == [16, 0, 40, 16]
    t = Table([[5, 9, -1], [-1] * 3], [20, 0], [0] * 9, 16)    # a branch of a row with a bad page; a last page that is bad
    t.fork([0], [1])
    t.resize([30, 40])
    assert t.status.item() == trs.DC_KV_BAD


@pytest.mark.parametrize("n", [6, 400])
def test_fork_same_row_twice(n):
    """A row that is dst twice takes the first branch alone, a row that is both src and dst none."""
    note("tables, rows named twice", n)
    rng = np.random.default_rng(n)
    t = start_table(rng, n + 4, 3, 16, 16, 2)
    t.resize(np.array([40, 20, 0, 0] + [0] * n))
    src = np.concatenate([[0, 1, 2, 0, 1, 3], rng.integers(0, 6, n - 6)])
    dst = np.concatenate([[2, 2, 5, 4, 5, 3], rng.integers(4, n + 4, n - 6)])
    t.fork(src, dst)
    assert t.status.item() == trs.DC_KV_BAD and t.lens[:6].tolist() == [40, 20, 40, 0, 40, 0]
    t.resize(np.zeros(n + 4, np.int32))
    assert (t.refs.cpu().numpy() > 0).sum() == 2


def test_tables_captured():
    """A captured fork and resize follow the lengths that changed; new_len may be kv_len itself."""
    t = torch()
    note("tables, captured")
    rng = np.random.default_rng(2)
    a = start_table(rng, 9, 8, 16, 300, 50)
    a.resize(np.array([40, 17, 64] + [0] * 6))
    src, dst, new = dev_i32([0, 1, 2]), dev_i32([3, 4, 5]), t.zeros(9, dtype=t.int32, device="cuda")
    g = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(g):
        trs.dc_kv_resize(a.table, new, a.copies, a.status)
        trs.dc_kv_fork(a.table, src, dst, a.status)
    for k in range(4):
        n = np.concatenate([rng.integers(1, 128, 3), [0, 0, 0], rng.integers(0, 128, 3)])
        new.copy_(dev_i32(n))
        g.replay()
        t.cuda.synchronize()
        copies = a.ref.resize(n.tolist())
        assert a.copies.tolist() == copies
        a.ref.fork([0, 1, 2], [3, 4, 5])
        a.check()
    trs.dc_kv_resize(a.table, a.lens, a.copies, a.status)
    a.check()
    assert (a.copies == -1).all()


def test_tables_many_sequences():
    note("tables, many")
    rng = np.random.default_rng(1)
    a = start_table(rng, 16384, 3, 16, 60000, 5000)
    a.resize(rng.integers(0, 49, 16384))
    a.resize(rng.integers(0, 49, 16384))


@pytest.mark.parametrize("at", [0, 700, 1500])
@pytest.mark.parametrize("shared", [False, True])
def test_tables_give_back_a_large_part(at, shared):
    """A pool that runs out behind thousands of a sequence's pages, among the first 1024 sequences and behind them, with
    and without an exchange of its last page: all of them are free again, and another sequence takes them."""
    note("tables, a large part", at, shared)
    seqs, width, page = 1600, 5000, 16
    rng = np.random.default_rng(at)
    pages, lens = np.full((seqs, width), -1, np.int32), np.zeros(seqs, np.int32)
    refs = np.where(rng.random(9001) < 0.5, 0, 1).astype(np.int32)
    held = np.nonzero(refs)[0]
    pages[at, :2], lens[at] = held[:2], 20                   # a partly filled last page
    if shared:
        pages[at + 1, :2], lens[at + 1] = held[:2], 20
        refs[held[:2]] = 2
    t = Table(pages, lens, refs, page)
    new = lens.copy()
    new[at] = width * page                                   # 4998 or 4999 of about 4500 free ones
    new[at + 3] = 40                                         # behind it: gets none
    t.resize(new)
    assert t.status.item() == trs.DC_KV_FULL and t.lens.tolist() == lens.tolist()
    new[at] = lens[at]
    t.status.zero_()
    t.ref.full = False
    new[at + 2], new[at + 3] = 4000 * page, 0
    t.resize(new)
    assert t.status.item() == 0 and t.lens[at + 2].item() == 4000 * page


def test_tables_giving_back_a_part_takes_as_long_as_keeping_it():
    t = torch()
    note("tables, a part's time")
    us = []
    for num in (8192, 8000):
        pages, lens = t.full((1, 8192), -1, dtype=t.int32, device="cuda"), t.zeros(1, dtype=t.int32, device="cuda")
        refs, copies = t.zeros(num, dtype=t.int32, device="cuda"), t.zeros(1, 2, dtype=t.int32, device="cuda")
        table, new, status = trs.KvTable(pages, lens, refs, 16), dev_i32([8192 * 16]), t.zeros(1, dtype=t.int32, device="cuda")

        def empty():
            pages.fill_(-1)
            for x in (lens, refs, status):
                x.zero_()

        us.append(shortest(lambda: trs.dc_kv_resize(table, new, copies, status), empty))
        assert status.item() == (trs.DC_KV_FULL if num < 8192 else 0) and bool((refs == (num == 8192)).all())
    print("%.1f and %.1f us" % tuple(us))
    assert us[1] < 10 * us[0]


def test_tables_of_nearly_2_to_the_31_pages():
    """The most pages that 31 bits number, all held but a few at either end: what is read ahead ends with the counts."""
    t = torch()
    num = 2 ** 31 - 1
    note("tables, pages", num)
    refs = t.ones(num, dtype=t.int32, device="cuda")
    refs[5], refs[num - 3:] = 0, 0
    pages, lens = t.full((3, 4), -1, dtype=t.int32, device="cuda"), t.zeros(3, dtype=t.int32, device="cuda")
    table, status = trs.KvTable(pages, lens, refs, 16), t.zeros(1, dtype=t.int32, device="cuda")
    copies = t.zeros(3, 2, dtype=t.int32, device="cuda")
    trs.dc_kv_resize(table, dev_i32([20, 16, 30]), copies, status)
    assert pages[:, 0].tolist() == [5, num - 2, -1] and pages[0, 1].item() == num - 3 and lens.tolist() == [20, 16, 0]
    assert refs[num - 3:].tolist() == [1, 1, 0] and refs[5].item() == 1 and status.item() == trs.DC_KV_FULL
    trs.dc_kv_resize(table, dev_i32([0, 0, 64]), copies, status)
    assert pages.tolist() == [[-1] * 4, [-1] * 4, [5, num - 3, num - 2, num - 1]] and lens.tolist() == [0, 0, 64]


# ------------------------------------------------------------------ pages
class Layers:
    """Pools of `layers` layers, every slot different: [layer] of [pages][heads][page][dim] codes on the host."""

    def __init__(self, seed, layers, pages, heads, page, dim, kv, order="hsd", gap=0):
        t = torch()
        rng = np.random.default_rng(seed)
        dt, ty = (np.uint16, t.bfloat16) if kv == "bf16" else (np.uint8, t.float8_e4m3fn)
        self.int = t.int16 if kv == "bf16" else t.uint8
        shape = (layers, 2, pages, heads, page, dim)
        self.host = rng.integers(0, 256 if kv == "e4m3" else 65536, shape).astype(dt)
        dev = t.from_numpy(self.host.view(np.int16 if kv == "bf16" else np.uint8)).cuda()
        if order == "shd":      # rows of all heads side by side
            dev = dev.transpose(3, 4).contiguous().transpose(3, 4)
        if gap:                 # room behind every head's rows and between pages
            wide = t.zeros(layers, 2, pages, heads + 1, page + gap, dim, dtype=dev.dtype, device="cuda")
            wide[:, :, :, :heads, :page] = dev
            self.wide = wide
            dev = wide[:, :, :, :heads, :page]
        self.dev = dev.view(ty)
        self.layers = trs.KvLayers([trs.KvCache(x[0], x[1]) for x in self.dev.unbind(0)])

    def check(self):
        got = self.dev.view(self.int).contiguous().cpu().numpy().view(self.host.dtype)
        assert np.array_equal(got, self.host)


COPY = [
    # layers, heads, page, dim, kv, order, gap, pairs
    (1, 1, 16, 64, "e4m3", "hsd", 0, 1),
    (3, 2, 16, 128, "bf16", "hsd", 0, 5),
    (2, 5, 32, 64, "bf16", "shd", 0, 9),
    (2, 3, 64, 128, "e4m3", "shd", 0, 4),
    (40, 8, 16, 128, "bf16", "hsd", 3, 7),
    (1, 40, 128, 128, "bf16", "hsd", 0, 3),
    (2, 7, 1024, 64, "e4m3", "hsd", 1, 2),
    (128, 1, 16, 64, "bf16", "hsd", 0, 2),
]


@pytest.mark.parametrize("layers,heads,page,dim,kv,order,gap,pairs", COPY)
def test_copy(layers, heads, page, dim, kv, order, gap, pairs):
    note("copy", layers, heads, page, dim, kv, order, gap, pairs)
    t = torch()
    pages = 2 * pairs + 3
    p = Layers(pairs, layers, pages, heads, page, dim, kv, order, gap)
    ids = np.random.default_rng(layers).permutation(pages)[:2 * pairs].reshape(-1, 2).astype(np.int32)
    bad = np.array([[-1, -1], [0, pages], [pages, 0], [-1, 0], [1 << 30, 1], [ids[0, 0], ids[0, 0]]], np.int32)
    trs.dc_kv_copy(p.layers, dev_i32(np.concatenate([ids, bad])))
    t.cuda.synchronize()
    for a, b in ids:
        p.host[:, :, b] = p.host[:, :, a]
    p.check()
    if gap:   # what lies between is as it was
        assert (p.wide[:, :, :, heads:] == 0).all() and (p.wide[:, :, :, :, page:] == 0).all()
    # one source for several pages
    trs.dc_kv_copy(p.layers, dev_i32([[ids[0, 0], x] for x in ids[:, 1]]))
    for b in ids[:, 1]:
        p.host[:, :, b] = p.host[:, :, ids[0, 0]]
    p.check()


COMPACT = [
    # layers, heads, page, dim, kv, order, lengths, share kept
    (1, 1, 16, 64, "bf16", "hsd", [1], 1.0),
    (2, 2, 16, 128, "bf16", "hsd", [100, 0, 17, 400], 0.5),
    (3, 17, 16, 64, "e4m3", "shd", [77, 130], 0.8),
    (1, 33, 32, 128, "bf16", "shd", [300, 64], 0.3),
    (2, 4, 64, 128, "e4m3", "hsd", [1000, 65, 2], 0.1),
    (2, 3, 16, 64, "bf16", "hsd", [200, 90], 1.0),
]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("layers,heads,page,dim,kv,order,lens,share", COMPACT)
def test_compact(layers, heads, page, dim, kv, order, lens, share, inplace):
    note("compact", layers, heads, page, dim, kv, order, lens, share, inplace)
    rng = np.random.default_rng(sum(lens) + heads)
    count = [-(-n // page) for n in lens]
    width = max(count) + 1
    pages = 2 * sum(count) + 2
    p = Layers(3, layers, pages, heads, page, dim, kv, order, gap=1 if order == "hsd" else 0)
    perm = rng.permutation(pages)
    tables = [np.full((len(lens), width), -1, np.int32) for _ in range(2)]
    at = 0
    for t in tables:
        for b, m in enumerate(count):
            t[b, :m] = perm[at:at + m]
            at += m
    kept = [np.sort(rng.permutation(n)[:int(n * share)]) for n in lens]
    if len(kept) > 1 and not inplace:
        kept[1] = rng.permutation(np.concatenate([kept[1], kept[1][:2]]))[:lens[1]]   # any order, the same token twice
    start = np.concatenate([[0], np.cumsum([k.size for k in kept])]).astype(np.int32)
    keep = np.concatenate(kept).astype(np.int32)
    keep = np.concatenate([keep, [0, 1, 2]]).astype(np.int32)      # behind the last sequence's: not looked at
    to = tables[0] if inplace else tables[1]
    trs.dc_kv_compact(p.layers, dev_i32(tables[0]), dev_i32(start), dev_i32(keep), None if inplace else dev_i32(to))
    torch().cuda.synchronize()
    for l in range(layers):
        for side in range(2):
            p.host[l, side] = step.compact(p.host[l, side], tables[0], start, keep, to, page)
    p.check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_behind_32_bits(kv):
    """Pages whose offsets pass 2^32 bytes and elements, keys and values of two layers in the room between each other's:
    copied, and compacted to other pages and in place."""
    t = torch()
    note("pages, far", kv)
    heads, page, dim, pages, layers, stride = 3, 16, 64, 18, 2, (1 << 28) + 8192
    p = Layers(5, layers, pages, heads, page, dim, kv)
    room = t.empty(stride * pages, dtype=p.dev.dtype, device="cuda")
    size = heads * page * dim
    shape, strides = (layers, 2, pages, heads, page, dim), (2 * size, size, stride, page * dim, dim, 1)
    far = room.as_strided(shape, strides)
    far.view(p.int).copy_(p.dev.view(p.int))
    p.dev = far
    p.layers = trs.KvLayers([trs.KvCache(x[0], x[1]) for x in far.unbind(0)])
    assert stride * (pages - 1) > 1 << 32
    trs.dc_kv_copy(p.layers, dev_i32([[17, 1], [2, 16], [15, 14]]))
    for a, b in ((17, 1), (2, 16), (15, 14)):
        p.host[:, :, b] = p.host[:, :, a]
    p.check()
    src, dst = np.array([[17, 0, 16], [3, 15, -1]], np.int32), np.array([[4, 13, -1], [12, 5, -1]], np.int32)
    start, keep = np.array([0, 20, 29], np.int32), np.concatenate([np.arange(1, 41, 2), np.arange(0, 27, 3)]).astype(np.int32)
    for to in (dst, None):
        trs.dc_kv_compact(p.layers, dev_i32(src), dev_i32(start), dev_i32(keep), None if to is None else dev_i32(to))
        for l in range(layers):
            for side in range(2):
                p.host[l, side] = step.compact(p.host[l, side], src, start, keep, src if to is None else to, page)
        p.check()


def test_compact_numbers_out_of_range():
    note("compact, out of range")
    p = Layers(4, 2, 6, 2, 16, 64, "bf16")
    src, dst = np.array([[0, 99], [1, -1]], np.int32), np.array([[3, 4], [-7, 5]], np.int32)
    start, keep = np.array([0, 20, 40], np.int32), np.concatenate([[5, -1, 1 << 30, 17, 3], np.arange(15), np.arange(20)]).astype(np.int32)
    trs.dc_kv_compact(p.layers, dev_i32(src), dev_i32(start), dev_i32(keep), dev_i32(dst))
    torch().cuda.synchronize()
    for l in range(2):
        for side in range(2):
            p.host[l, side] = step.compact(p.host[l, side], src, start, keep, dst, 16)
    p.check()


# ---------------------------------------------------------- 4-bit floats
def mx4_case(rng, rows, cols, size=1.0):
    """A random matrix in the format: (fp64 values, view)."""
    codes, scale = step.mx4_quantize(vals(bits(rng.normal(size=(rows, cols)) * size * np.exp(rng.normal(size=(rows, 1))))))
    return step.mx4_matrix(codes, scale), trs.Mx4View(rows, cols, torch().from_numpy(step.mx4_pack(codes, scale)).cuda())


def mx4_empty(rows, cols, fill=0xEE):
    t = torch()
    return trs.Mx4View(rows, cols, t.full((trs.dc_mx4_bytes(rows, cols),), fill, dtype=t.uint8, device="cuda"))


@pytest.mark.parametrize("rows,cols,stride", [(1, 128, 128), (16, 512, 512), (17, 640, 648), (63, 1152, 1152), (128, 384, 1024),
                                              (200, 2048, 2048)])
def test_mx4_pack(rows, cols, stride):
    t = torch()
    note("mx4 pack", rows, cols, stride)
    rng = np.random.default_rng(rows)
    x = rng.normal(size=(rows, cols)) * np.exp(3 * rng.normal(size=(rows, 1)))
    x[0, 32:64] = 0.0
    x[-1, 96:128] = -0.0
    x[0, :32] *= 2.0 ** -120
    x[rows // 2, 64:96] = rng.integers(-12, 13, 32) / 4.0 * 4.0 ** rng.integers(-20, 20)     # ties
    b = bits(x)
    wide = t.full((rows, stride), float("nan"), dtype=t.bfloat16, device="cuda")
    wide[:, :cols] = dev_bits(b)
    view, flag = mx4_empty(rows, cols), t.full((1,), 9, dtype=t.int32, device="cuda")
    trs.dc_mx4_pack_device(wide[:, :cols], view, flag)
    t.cuda.synchronize()
    codes, scale = step.mx4_quantize(vals(b))
    assert flag.item() == 0
    assert np.array_equal(view.buf.cpu().numpy(), step.mx4_pack(codes, scale))
    back = t.full((rows, stride), 3.0, dtype=t.bfloat16, device="cuda")
    trs.dc_mx4_dequant(view, back[:, :cols])
    assert np.array_equal(vals(host_bits(back[:, :cols])), step.mx4_matrix(codes, scale)) and (back[:, cols:] == 3).all()
    other = mx4_empty(rows, cols, 0x11)
    trs.dc_mx4_pack_device(back[:, :cols], other)            # what the format holds, it keeps
    back2 = t.zeros_like(back)
    trs.dc_mx4_dequant(other, back2[:, :cols])
    assert np.array_equal(host_bits(back2[:, :cols]), host_bits(back[:, :cols]))


def test_mx4_pack_of_the_longest_rows():
    """One row of as many columns as 31 bits hold, 512 of them over and over; the last ones are 384."""
    t = torch()
    cols = 2 ** 31 - 128
    note("mx4 pack, longest row", cols)
    part = bits(np.random.default_rng(2).normal(size=(1, 512)))
    x = dev_bits(part)[0].repeat(2 ** 22)[:cols].view(1, cols)
    view, flag = mx4_empty(1, cols), t.ones(1, dtype=t.int32, device="cuda")
    trs.dc_mx4_pack_device(x, view, flag)
    one = step.mx4_pack(*step.mx4_quantize(vals(part)))
    codes, words = t.from_numpy(one[:4096]).cuda().view(t.int64), t.from_numpy(one[4096:].copy()).cuda().view(t.int32)
    n = cols * 8
    got, scales = view.buf[:n].view(t.int64), view.buf[n:].view(t.int32)
    assert flag.item() == 0 and scales.numel() == 64 * 2 ** 22
    assert bool((got[:512 * (2 ** 22 - 1)].view(-1, 512) == codes).all()) and t.equal(got[512 * (2 ** 22 - 1):], codes[:384])
    assert bool((scales[:-64].view(-1, 64) == words).all()) and t.equal(scales[-64:], words & 0xFFFFFF)


def test_mx4_pack_every_bit_pattern():
    """Every bf16 number as the largest of a block and beside a larger one; infinities and NaN make a block NaN."""
    t = torch()
    note("mx4 pack, every bit pattern")
    every = np.arange(1 << 16, dtype=np.uint16)
    alone = np.zeros((1 << 16, 32), np.uint16)
    alone[np.arange(1 << 16), every % 32] = every
    beside = alone.copy()
    finite = np.isfinite(vals(every))
    e = (every >> 7) & 255
    up = np.minimum(e + (every & 3), 254).astype(np.uint16) << 7 | 0x55        # up to 8 times as large
    beside[np.arange(1 << 16), (every + 5) % 32] = up
    x = np.concatenate([alone, beside]).reshape(-1, 512)
    view, flag = mx4_empty(*x.shape), t.zeros(1, dtype=t.int32, device="cuda")
    trs.dc_mx4_pack_device(dev_bits(x), view, flag)
    t.cuda.synchronize()
    codes, scale = step.mx4_quantize(vals(x))
    assert flag.item() == 1 and (scale == 255).sum() == 2 * (~finite).sum()
    assert np.array_equal(view.buf.cpu().numpy(), step.mx4_pack(codes, scale))
    back = t.zeros(x.shape, dtype=t.bfloat16, device="cuda")
    trs.dc_mx4_dequant(view, back)
    assert np.array_equal(vals(host_bits(back)), step.mx4_matrix(codes, scale), equal_nan=True)


def mx4_tolerance(w, x, y):
    """One rounding to bf16; the sums: a matrix-core product adds 32 or 128 products in at most 36 (132) roundings of
    2^-23, so at most cols + cols/8 of them in a row, and 8 more for the waves."""
    return BF16 * np.abs(y) + (w.shape[1] * 1.125 + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


MX4 = [(1, 128, 128), (1, 512, 1152), (3, 384, 4096), (16, 128, 1280), (17, 256, 256), (33, 640, 384), (64, 128, 2048),
       (65, 1920, 640), (200, 384, 256), (130, 1408, 896)]


def close(got, want, tol, what):
    err = np.abs(got - want)
    rel = np.linalg.norm(err) / np.linalg.norm(want)
    print("[%s] worst error / bound %.3f, rel L2 %.2e" % (what, (err / tol).max(), rel), flush=True)
    assert (err <= tol).all()
    assert rel <= BF16      # the rounding at its bound everywhere; it takes 0.42 of that where values are spread evenly


@pytest.mark.parametrize("t_,out,inn", MX4)
def test_apply_mx4(t_, out, inn):
    t = torch()
    note("mx4", t_, out, inn)
    rng = np.random.default_rng(t_ + out)
    w, view = mx4_case(rng, out, inn)
    x = vals(bits(rng.normal(size=(t_, inn))))
    xd = dev_bits(bits(x))
    y = t.full((t_ + 1, out), float("nan"), dtype=t.bfloat16, device="cuda")
    trs.dc_apply_mx4(view, xd, y[:t_])
    t.cuda.synchronize()
    first = host_bits(y).copy()
    want = x @ w.T
    close(vals(first[:t_]), want, mx4_tolerance(w, x, want), "mx4")
    assert np.isnan(vals(first[t_:])).all()
    y.zero_()
    trs.dc_apply_mx4(view, xd, y[:t_])
    assert np.array_equal(host_bits(y)[:t_], first[:t_])


@pytest.mark.parametrize("t_,out,inn", MX4 + [(300, 256, 512), (257, 640, 1536), (511, 384, 640), (1030, 1152, 2176)])
def test_apply_mx4q(t_, out, inn):
    t = torch()
    note("mx4q", t_, out, inn)
    rng = np.random.default_rng(t_ + inn)
    w, view = mx4_case(rng, out, inn)
    x = vals(bits(rng.normal(size=(t_, inn)) * np.exp(rng.normal(size=(1, inn)))))
    xq = mx4_empty(t_, inn)
    trs.dc_mx4_pack_device(dev_bits(bits(x)), xq)
    y = t.full((t_ + 1, out), float("nan"), dtype=t.bfloat16, device="cuda")
    trs.dc_apply_mx4q(view, xq, y[:t_])
    t.cuda.synchronize()
    first = host_bits(y).copy()
    x4 = step.mx4_matrix(*step.mx4_quantize(x))
    want = x4 @ w.T
    close(vals(first[:t_]), want, mx4_tolerance(w, x4, want), "mx4q")
    assert np.isnan(vals(first[t_:])).all()
    y.zero_()
    trs.dc_apply_mx4q(view, xq, y[:t_])
    assert np.array_equal(host_bits(y)[:t_], first[:t_])


# Every tile of the products with bf16 activations (by the rules in launch_mx4 and launch_mx4_few).
@pytest.mark.parametrize("t_,out,inn", [
    (1, 4096, 512), (7, 11008, 640), (16, 8320, 384), (2, 32000, 256), (13, 12416, 896), (3, 8192, 256),   # 16 to 64 rows, up to 16 tokens
    (32, 4096, 1152), (17, 128, 2176), (64, 4096, 1280), (50, 4224, 640), (100, 4096, 896),       # 32 x 16, 32 x 32
    (20, 11008, 1152), (128, 4224, 1408), (64, 11008, 640), (250, 4096, 384), (60, 32000, 128),   # 64 x 32 of 8 and of 4 waves
    (500, 4096, 1152), (130, 11008, 512), (700, 8064, 640), (64, 32000, 1664)])                   # 128 x 64
def test_apply_mx4_tiles(t_, out, inn):
    t = torch()
    note("mx4 tiles", t_, out, inn)
    rng = np.random.default_rng(t_ + out + inn)
    w, view = mx4_case(rng, out, inn)
    xd = dev_bits(bits(rng.normal(size=(t_, inn)).astype(np.float32)))
    wd = t.from_numpy(w).cuda()
    y = t.full((t_ + 1, out), float("nan"), dtype=t.bfloat16, device="cuda")
    trs.dc_apply_mx4(view, xd, y[:t_])
    t.cuda.synchronize()
    first = y.clone()
    want = xd.double() @ wd.t().contiguous()
    tol = BF16 * want.abs() + (inn * 1.125 + 8) * 2.0 ** -23 * (xd.double().abs() @ wd.abs().t().contiguous())
    err = (y[:t_].double() - want).abs()
    assert bool((err <= tol).all()) and float(err.norm() / want.norm()) <= BF16
    assert bool(y[t_:].isnan().all())
    y.zero_()
    trs.dc_apply_mx4(view, xd, y[:t_])
    assert t.equal(y[:t_], first[:t_])


# Every tile of the product (by the rule in launch_mx4q): one or several for a block, columns of 1, 2, 3 and 0 more
# than whole groups of 512, and fewer than 512; rows and tokens that end inside a tile.
@pytest.mark.parametrize("t_,out,inn", [
    (32, 4096, 4096), (17, 4224, 3968),                                              # 16 x 32
    (100, 6400, 1536), (300, 6400, 640), (100, 6400, 1280), (700, 8064, 256), (3000, 1152, 384),   # 32 x 64
    (390, 4224, 1024), (520, 8064, 640), (520, 8064, 768), (520, 8064, 896), (4100, 3200, 128),    # 64 x 64
    (1500, 4224, 512), (1500, 4224, 640), (1500, 4224, 768), (390, 4096, 896), (1100, 6400, 256),  # 64 x 128
    (2600, 4096, 1536), (2600, 4096, 1664), (390, 6400, 768), (520, 4096, 896), (900, 4096, 384),  # 128 x 128
    (5000, 6400, 1536), (2000, 8064, 1152), (5000, 6400, 1792), (5000, 6528, 1408)])               # 256 x 256
def test_apply_mx4q_tiles(t_, out, inn):
    t = torch()
    note("mx4q tiles", t_, out, inn)
    rng = np.random.default_rng(t_ + out + inn)
    w, view = mx4_case(rng, out, inn)
    x = vals(bits(rng.normal(size=(t_, inn)).astype(np.float32)))
    xq = mx4_empty(t_, inn)
    trs.dc_mx4_pack_device(dev_bits(bits(x)), xq)
    x4 = t.from_numpy(step.mx4_matrix(*step.mx4_quantize(x))).cuda()
    wd = t.from_numpy(w).cuda()
    y = t.full((t_ + 1, out), float("nan"), dtype=t.bfloat16, device="cuda")
    trs.dc_apply_mx4q(view, xq, y[:t_])
    t.cuda.synchronize()
    first = y.clone()
    want = x4 @ wd.t().contiguous()
    tol = BF16 * want.abs() + (inn * 1.125 + 8) * 2.0 ** -23 * (x4.abs() @ wd.abs().t().contiguous())
    err = (y[:t_].double() - want).abs()
    assert bool((err <= tol).all()) and float(err.norm() / want.norm()) <= BF16
    assert bool(y[t_:].isnan().all())
    y.zero_()
    trs.dc_apply_mx4q(view, xq, y[:t_])
    assert t.equal(y[:t_], first[:t_])


# The form that a call takes (csrc/step.h), and calls of each: tokens that end inside
# a tile, columns of 1, 2, 3 and 0 more than whole groups of 512.
MX4_FORMS = ["%d x 16" % (16 * r) for r in (1, 2, 3, 4)] + ["few " + x for x in ("32 x 16", "32 x 32", "64 x 32 of 8 waves", "64 x 32", "128 x 64")]
MX4Q_FORMS = ["16 x 16", "16 x 32", "32 x 32", "32 x 64", "64 x 64", "64 x 128", "128 x 128", "256 x 256"]


def mx4_form(t_, out, inn):
    L = trs.lib()
    return MX4_FORMS[L._ZN2dc13mx4_row_tilesEii(out, t_) - 1 if t_ <= 16 else 4 + L._ZN2dc12mx4_few_tileEiii(out, inn, t_)]


def mx4q_form(t_, out, inn):
    return MX4Q_FORMS[trs.lib()._ZN2dc9mx4q_tileEiii(out, inn, t_)]


MX4_CALLS = {
    "16 x 16": [(5, 1152, 512), (15, 128, 640), (2, 1152, 256), (9, 128, 384)],
    "32 x 16": [(1, 4224, 512), (5, 4224, 640), (9, 4224, 256), (15, 6272, 384)],
    "48 x 16": [(2, 8320, 512), (5, 8320, 640), (9, 8320, 256), (15, 11008, 384)],
    "64 x 16": [(1, 12416, 512), (5, 12416, 640), (9, 12416, 256), (15, 32000, 384)],
    "few 32 x 16": [(17, 128, 1024), (17, 128, 1152), (19, 1152, 1792), (17, 128, 1408)],
    "few 32 x 32": [(17, 128, 512), (50, 1152, 640), (61, 1152, 256), (17, 128, 384)],
    "few 64 x 32 of 8 waves": [(33, 4224, 512), (33, 4224, 640), (50, 4224, 256), (33, 4224, 384)],
    "few 64 x 32": [(33, 11008, 512), (33, 11008, 640), (33, 11008, 768), (33, 11008, 384)],
    "few 128 x 64": [(65, 11008, 512), (17, 128, 128), (33, 11008, 256), (65, 11008, 384)],
}
MX4Q_CALLS = {
    "16 x 16": [(17, 128, 1024), (17, 128, 1152), (15, 384, 1280), (17, 128, 896)],
    "16 x 32": [(50, 1152, 2560), (61, 1152, 2176), (19, 2176, 2304), (33, 2048, 2432)],
    "32 x 32": [(17, 128, 512), (50, 1152, 640), (61, 1152, 256), (17, 128, 384)],
    "32 x 64": [(100, 11008, 1024), (33, 32000, 640), (33, 32000, 768), (100, 6400, 1408)],
    "64 x 64": [(33, 32000, 1024), (100, 6400, 1664), (700, 11008, 256), (33, 32000, 896)],
    "64 x 128": [(4100, 384, 1024), (65, 11008, 2176), (1100, 6400, 256), (4100, 384, 896)],
    "128 x 128": [(65, 32000, 512), (65, 32000, 640), (65, 32000, 768), (100, 32000, 384)],
    "256 x 256": [(5300, 5888, 1408), (4500, 10496, 1280), (5800, 7936, 1536), (1100, 11136, 1664)],
}


@pytest.mark.parametrize("form,t_,out,inn", [(f, *c) for f, cs in MX4_CALLS.items() for c in cs])
def test_apply_mx4_forms(form, t_, out, inn):
    assert mx4_form(t_, out, inn) == form
    test_apply_mx4_tiles(t_, out, inn)


@pytest.mark.parametrize("form,t_,out,inn", [(f, *c) for f, cs in MX4Q_CALLS.items() for c in cs])
def test_apply_mx4q_forms(form, t_, out, inn):
    assert mx4q_form(t_, out, inn) == form
    test_apply_mx4q_tiles(t_, out, inn)


# The largest tile: two or three for a block, columns of whole groups of 512 and of 1, 2 and 3 more.
@pytest.mark.parametrize("t_,out,inn", [(5300, 5888, 1408), (4500, 10496, 1280), (5800, 7936, 1536), (6300, 6912, 1664), (4600, 6272, 2048)])
def test_apply_mx4q_largest_tiles(t_, out, inn):
    test_apply_mx4q_tiles(t_, out, inn)


@pytest.mark.parametrize("t_,out,inn,four", [(530001, 128, 4096, False), (300001, 8064, 128, True), (270001, 8064, 128, False)])
def test_mx4_rows_behind_32_bits(t_, out, inn, four):
    """Activations of more than 2^31 entries, results that pass 2^32 bytes: rows at either end, around the borders and between."""
    t = torch()
    note("mx4, far rows", t_, out, inn, four)
    rng = np.random.default_rng(out)
    w, view = mx4_case(rng, out, inn)
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    x = t.randn(t_, inn, generator=g, device="cuda", dtype=t.bfloat16)
    y = t.full((t_ + 1, out), float("nan"), dtype=t.bfloat16, device="cuda")
    assert max(t_ * inn, t_ * out) > 1 << 31
    if four:
        xq = mx4_empty(t_, inn)
        trs.dc_mx4_pack_device(x, xq)
        trs.dc_apply_mx4q(view, xq, y[:t_])
    else:
        trs.dc_apply_mx4(view, x, y[:t_])
    ends = [k * (1 << 31) // n for n in (inn, out) for k in (1, 2) if k * (1 << 31) // n < t_]
    rows = np.unique(np.concatenate([np.arange(40), t_ - 1 - np.arange(300), *[e + np.arange(-40, 40) for e in ends], rng.integers(0, t_, 300)]))
    rows = rows[(rows >= 0) & (rows < t_)]
    at = t.from_numpy(rows).cuda()
    xs = x[at].double().cpu().numpy()
    if four:
        xs = step.mx4_matrix(*step.mx4_quantize(xs))
    want = xs @ w.T
    assert (np.abs(y[at].double().cpu().numpy() - want) <= mx4_tolerance(w, xs, want)).all()
    assert bool(y[t_].isnan().all()) and not any(bool(part.isnan().any()) for part in y[:t_].split(1 << 15))


@pytest.mark.parametrize("t_", [1, 20, 70, 300])
def test_mx4_values_that_are_not_finite(t_):
    """A NaN block reaches its row, an x that is not finite its token; neither reaches further."""
    t = torch()
    note("mx4, not finite", t_)
    rng = np.random.default_rng(t_)
    out, inn = 384, 1280
    w = vals(bits(rng.normal(size=(out, inn))))
    w[130, 700] = np.inf
    x = vals(bits(rng.normal(size=(t_, inn))))
    x[t_ // 2, 1279] = np.nan
    codes, scale = step.mx4_quantize(w)
    view = trs.Mx4View(out, inn, t.from_numpy(step.mx4_pack(codes, scale)).cuda())
    w4 = step.mx4_matrix(codes, scale)
    xq = mx4_empty(t_, inn)
    trs.dc_mx4_pack_device(dev_bits(bits(x)), xq)
    x4 = step.mx4_matrix(*step.mx4_quantize(x))
    for xs, call, arg in ((x, trs.dc_apply_mx4, dev_bits(bits(x))), (x4, trs.dc_apply_mx4q, xq)):
        y = t.zeros(t_, out, dtype=t.bfloat16, device="cuda")
        call(view, arg, y)
        got = vals(host_bits(y))
        bad = np.zeros((t_, out), bool)
        bad[t_ // 2], bad[:, 130] = True, True
        assert np.array_equal(np.isnan(got), bad)
        want = np.where(bad, 0.0, np.nan_to_num(xs) @ np.nan_to_num(w4).T)
        tol = mx4_tolerance(np.nan_to_num(w4), np.nan_to_num(xs), want)
        assert (np.abs(np.where(bad, 0.0, got) - want) <= tol).all()


@pytest.mark.parametrize("low", [0, 252])
def test_mx4_scales_at_their_ends(low):
    """The smallest and the largest scales that the packer makes, against activations that bring the sums back."""
    t = torch()
    note("mx4, scales", low)
    rng = np.random.default_rng(low)
    out, inn, t_ = 128, 256, 5
    codes = rng.integers(0, 16, (out, inn))
    scale = np.full((out, inn // 32), low) + rng.integers(0, 1 + (low == 0), (out, inn // 32))
    view = trs.Mx4View(out, inn, t.from_numpy(step.mx4_pack(codes, scale)).cuda())
    w = step.mx4_matrix(codes, scale)
    x = vals(bits(rng.normal(size=(t_, inn)) * 2.0 ** (100 if low == 0 else -100)))
    want = x @ w.T
    y = t.zeros(t_, out, dtype=t.bfloat16, device="cuda")
    trs.dc_apply_mx4(view, dev_bits(bits(x)), y)
    # the products' own sizes; subnormal ones (2^-126) may count as zero
    assert (np.abs(vals(host_bits(y)) - want) <= mx4_tolerance(w, x, want)).all()
    xq = mx4_empty(t_, inn)
    trs.dc_mx4_pack_device(dev_bits(bits(x)), xq)
    x4 = step.mx4_matrix(*step.mx4_quantize(x))
    want = x4 @ w.T
    trs.dc_apply_mx4q(view, xq, y)
    assert (np.abs(vals(host_bits(y)) - want) <= mx4_tolerance(w, x4, want)).all()


@pytest.mark.parametrize("t_", [1, 9, 16, 17, 40, 100, 300, 520])
@pytest.mark.parametrize("least", [250, 253])
def test_mx4_numbers_larger_than_bf16_holds(t_, least):
    """Scales up to the last one, 254: the products are those of the formula where the numbers themselves pass bf16's
    largest, among small ones, blocks without a number and one that is NaN."""
    t = torch()
    note("mx4, large scales", t_, least)
    rng = np.random.default_rng(t_ + least)
    out, inn = 1152, 640
    codes = rng.integers(0, 16, (out, inn))
    scale = rng.integers(least, 255, (out, inn // 32))
    scale[rng.random(scale.shape) < 0.1] = 128
    codes.reshape(out, -1, 32)[rng.random(scale.shape) < 0.1] = 0
    scale[7, 3] = 255
    view = trs.Mx4View(out, inn, t.from_numpy(step.mx4_pack(codes, scale)).cuda())
    w = step.mx4_matrix(codes, scale)
    x = vals(bits(rng.normal(size=(t_, inn)) * 2.0 ** -100))
    y = t.zeros(t_, out, dtype=t.bfloat16, device="cuda")
    xq = mx4_empty(t_, inn)
    trs.dc_mx4_pack_device(dev_bits(bits(x)), xq)
    x4 = step.mx4_matrix(*step.mx4_quantize(x))
    for xs, call, arg in ((x, trs.dc_apply_mx4, dev_bits(bits(x))), (x4, trs.dc_apply_mx4q, xq)):
        call(view, arg, y)
        got = vals(host_bits(y))
        assert np.isnan(got[:, 7]).all()
        got[:, 7] = 0.0
        w0 = np.nan_to_num(w)
        w0[7] = 0.0
        want = xs @ w0.T
        # four products at a quarter for one: five times the sums' roundings at most
        tol = BF16 * np.abs(want) + 5 * (inn * 1.125 + 8) * 2.0 ** -23 * (np.abs(xs) @ np.abs(w0).T)
        assert (np.abs(got - want) <= tol).all()
    back = t.zeros(out, inn, dtype=t.bfloat16, device="cuda")
    trs.dc_mx4_dequant(view, back)
    want = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
    assert np.array_equal(vals(host_bits(back)), want, equal_nan=True)


def test_mx4_captured():
    t = torch()
    note("mx4, captured")
    rng = np.random.default_rng(1)
    w, view = mx4_case(rng, 256, 640)
    x, xq = dev_bits(bits(rng.normal(size=(40, 640)))), mx4_empty(40, 640)
    flag = t.zeros(1, dtype=t.int32, device="cuda")
    ys = [t.zeros(40, 256, dtype=t.bfloat16, device="cuda") for _ in range(4)]

    def both(y, z):
        trs.dc_apply_mx4(view, x, y)
        trs.dc_mx4_pack_device(x, xq, flag)
        trs.dc_apply_mx4q(view, xq, z)

    both(*ys[2:])
    side, g = t.cuda.Stream(), t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(g, stream=side):
        both(*ys[:2])
    for k in range(4):
        x.copy_(dev_bits(bits(rng.normal(size=(40, 640)))))
        if k == 2:
            x[3, 5] = float("inf")
        t.cuda.synchronize()
        with t.cuda.stream(side):
            g.replay()
        t.cuda.synchronize()
        assert flag.item() == (k == 2)
        both(*ys[2:])
        t.cuda.synchronize()
        assert all(np.array_equal(host_bits(a), host_bits(b)) for a, b in zip(ys[:2], ys[2:]))


def test_mx4_binding_refusals():
    t = torch()
    _, view = mx4_case(np.random.default_rng(0), 128, 256)
    z = lambda *s: t.zeros(*s, dtype=t.bfloat16, device="cuda")  # noqa: E731
    for bad in (lambda: trs.dc_apply_mx4(view, z(2, 128), z(2, 128)), lambda: trs.dc_apply_mx4(view, z(2, 256), z(2, 256)),
                lambda: trs.dc_apply_mx4(view, z(4, 256)[::2], z(2, 128)), lambda: trs.dc_apply_mx4(view, z(2, 256).float(), z(2, 128)),
                lambda: trs.dc_apply_mx4(view, z(2, 256).cpu(), z(2, 128)), lambda: trs.dc_mx4_dequant(view, z(128, 128)),
                lambda: trs.dc_mx4_pack_device(z(128, 128), view), lambda: trs.Mx4View(0, 256, view.buf), lambda: trs.Mx4View(129, 256, view.buf),
                lambda: trs.dc_apply_mx4q(view, view, z(5, 128))):
        with pytest.raises(ValueError):
            bad()
    trs.dc_apply_mx4(view, z(0, 256), z(0, 128))


# ------------------------------------------------------------ all together
def test_step_of_branching_chats():
    """Two chats of a layer branch; the branches' last pages are exchanged and copied; the head at 4 bits gives the
    logits of the drafted tokens, which are verified; lengths follow what stood, on the device; a chat then keeps part of
    its tokens.  Eagerly and as a graph."""
    t = torch()
    note("step")
    rng = np.random.default_rng(21)
    page, heads, dim, hidden, vocab, layers_ = 16, 2, 64, 256, 640, 2
    nq = 4                                                       # input tokens of a chat in the step, 3 of them drafts
    lens0 = [37, 20, 0, 0, 0]
    pages = np.full((5, 6), -1, np.int32)
    pages[0, :3], pages[1, :2] = [9, 4, 7], [1, 6]
    refs = np.zeros(24, np.int32)
    refs[[9, 4, 7, 1, 6]] = 1
    src, dst = dev_i32([0, 0, 1]), dev_i32([2, 3, 4])
    w, head = mx4_case(rng, vocab, hidden, 0.2)
    n = 5 * nq
    q_start = np.arange(6, dtype=np.int32) * nq
    x = vals(bits(rng.normal(size=(n, hidden))))
    xd = dev_bits(bits(x))
    tokens, accept, picks = rng.integers(0, vocab, n).astype(np.int32), rng.random(n).astype(np.float32), rng.random(5).astype(np.float32)
    logits = vals(bits(x @ w.T))
    tokens[1:] = np.where(rng.random(n - 1) < 0.6, logits.argmax(1)[:-1], tokens[1:])   # likely drafts, most of them
    temp = np.array([0.7, 1.0, 0.0, 0.5, 1.3], np.float32)
    batch = trs.VerifyBatch(dev_i32(q_start), dev_i32(tokens), dev_f32(accept), dev_f32(picks), dev_f32(temp))
    vws = t.empty(trs.dc_verify_workspace_bytes(vocab, n, 5), dtype=t.uint8, device="cuda")

    def run(captured):
        tab = Table(pages, lens0, refs, page)
        pool = Layers(31, layers_, 24, heads, page, dim, "bf16")
        y = t.zeros(n, vocab, dtype=t.bfloat16, device="cuda")
        out, count = (t.full((k,), -9, dtype=t.int32, device="cuda") for k in (n, 5))
        new, after = t.zeros(5, dtype=t.int32, device="cuda"), t.zeros(5, dtype=t.int32, device="cuda")

        def body():
            trs.dc_kv_fork(tab.table, src, dst, tab.status)
            t.add(tab.lens, nq, out=new)
            trs.dc_kv_resize(tab.table, new, tab.copies, tab.status)
            trs.dc_kv_copy(pool.layers, tab.copies)
            trs.dc_apply_mx4(head, xd, y)
            trs.dc_verify_drafts(batch, y, None, out, count, vws)
            t.sub(tab.lens, nq, out=after)
            t.add(after, count, out=after)                       # the first input token and the drafts that stood
            trs.dc_kv_resize(tab.table, after, tab.copies2, tab.status)

        tab.copies2 = t.zeros_like(tab.copies)
        if captured:
            g = t.cuda.CUDAGraph()
            t.cuda.synchronize()
            with t.cuda.graph(g):
                body()
            g.replay()
        else:
            body()
        t.cuda.synchronize()
        return tab, pool, y, out, count

    tab, pool, y, out, count = run(False)
    r = tab.ref
    r.fork([0, 0, 1], [2, 3, 4])
    copies = r.resize([a + nq for a in r.kv_len])
    assert tab.copies.tolist() == copies and sum(a >= 0 for a, _ in copies) == 5
    for a, b in copies:
        pool.host[:, :, b] = pool.host[:, :, a]
    pool.check()
    got = vals(host_bits(y))
    want = x @ w.T
    assert (np.abs(got - want) <= mx4_tolerance(w, x, want)).all()
    o, _, c, margin = step.verify(got, None, q_start, tokens, accept, picks, temp.astype(np.float64))
    assert margin > 1e-11 and out.tolist() == o and count.tolist() == c and 5 < sum(c) < n
    r.resize([a - nq + k for a, k in zip(r.kv_len, c)])
    tab.check()
    assert not r.full and not r.bad
    # chat 0 keeps every other token of its own pages
    keep = np.arange(0, r.kv_len[3], 2, dtype=np.int32)
    own = np.array([r.pages[3]], np.int32)
    fresh = np.full_like(own, -1)
    free = [p for p in range(24) if r.refs[p] == 0][:-(-keep.size // page)]
    fresh[0, :len(free)] = free
    trs.dc_kv_compact(pool.layers, dev_i32(own), dev_i32([0, keep.size]), dev_i32(keep), dev_i32(fresh))
    for l in range(layers_):
        for s in range(2):
            pool.host[l, s] = step.compact(pool.host[l, s], own, [0, keep.size], keep, fresh, page)
    pool.check()
    tab2, pool2, y2, out2, count2 = run(True)
    assert t.equal(y, y2) and t.equal(out, out2) and t.equal(count, count2)
    assert t.equal(tab.pages, tab2.pages) and t.equal(tab.refs, tab2.refs) and t.equal(tab.lens, tab2.lens)
