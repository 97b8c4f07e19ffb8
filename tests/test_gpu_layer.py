"""The decoder-layer operators on the GPU against the fp64 oracle: appending rotated keys and values to a paged cache,
attention over shared prefixes, products with a 4-bit backbone, and a layer's step that runs them together.

Every unused slot of a cache holds NaN, so that anything read from where it must not be shows."""
import os

import numpy as np
import pytest

import synth
import tenant_rank_serving_amd as trs
from gpu_util import dev_i32, note, torch, upload, workspace
from oracle import apply as oap
from oracle import layer

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


def dev_bf16(a):
    t = torch()
    return t.from_numpy(np.ascontiguousarray(bits(a)).view(np.int16)).cuda().view(t.bfloat16)


def host_bits(x):
    t = torch()
    return x.contiguous().view(t.int16).cpu().numpy().view(np.uint16)


class Pool:
    """A cache of NaN on the host ([pages][heads][page][dim] bits or codes) and its values."""

    def __init__(self, kv, pages, heads, page, dim, rng, nhd=False, together=False):
        t = torch()
        self.kv, self.nhd = kv, nhd
        self.nan = 0x7FC1 if kv == "bf16" else 0x7F
        dt = np.uint16 if kv == "bf16" else np.uint8
        self.k = np.full((pages, heads, page, dim), self.nan, dt)
        self.v = self.k.copy()
        self.ks = self.vs = None
        if kv == "e4m3":
            self.ks = rng.uniform(0.005, 0.03, heads).astype(np.float32)
            self.vs = rng.uniform(0.005, 0.03, heads).astype(np.float32)
        self.together = together

    def put(self, which, table, n, x, page):
        """Rows 0 .. n-1 of a sequence: x [n][heads][dim] (values)."""
        pool, sc = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        i = np.arange(n)
        if self.kv == "bf16":
            pool[np.asarray(table)[i // page], :, i % page] = bits(x)
        else:
            c = layer.e4m3_code(np.asarray(x, np.float64) / sc[:, None].astype(np.float64))
            pool[np.asarray(table)[i // page], :, i % page] = c

    def values(self, which):
        pool, sc = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        if self.kv == "bf16":
            return vals(pool)
        return layer.e4m3_value(pool) * sc.astype(np.float64)[None, :, None, None]

    def upload(self):
        t = torch()
        dt = np.int16 if self.kv == "bf16" else np.uint8
        ty = t.bfloat16 if self.kv == "bf16" else t.float8_e4m3fn
        both = [a.view(dt) for a in (self.k, self.v)]
        if self.nhd:
            both = [np.ascontiguousarray(a.transpose(0, 2, 1, 3)) for a in both]
        if self.together:   # keys and values of a page side by side in one allocation
            one = t.from_numpy(np.ascontiguousarray(np.stack(both, 1))).cuda().view(ty)
            self.dk, self.dv = one[:, 0], one[:, 1]
        else:
            self.dk, self.dv = (t.from_numpy(a).cuda().view(ty) for a in both)
        if self.nhd:
            self.dk, self.dv = self.dk.transpose(1, 2), self.dv.transpose(1, 2)
        f = lambda a: None if a is None else t.from_numpy(a).cuda()  # noqa: E731
        return trs.KvCache(self.dk, self.dv, f(self.ks), f(self.vs))

    def download(self):
        t = torch()
        ty, dt = (t.int16, np.uint16) if self.kv == "bf16" else (t.uint8, np.uint8)
        return [x.contiguous().view(ty).cpu().numpy().view(dt) for x in (self.dk, self.dv)]


# ----------------------------------------------------------------- append
APPEND = [
    # n, hq, hkv, dim, page, kv, rot, interleaved, nhd, farthest position
    (1, 32, 32, 128, 16, "bf16", 128, False, False, 4096),
    (7, 8, 2, 128, 64, "bf16", 64, True, True, 100),
    (33, 4, 4, 64, 16, "e4m3", 64, False, False, 200000),
    (65, 6, 2, 64, 32, "e4m3", 32, True, True, 1000),
    (600, 8, 8, 128, 16, "bf16", 128, False, True, 1 << 30),
    (530, 5, 1, 128, 1024, "e4m3", 112, False, False, 5000),
    (3, 0, 3, 128, 16, "bf16", 16, False, False, 50),
    (9, 3, 3, 64, 16, "bf16", 0, False, False, 50),
]


@pytest.mark.parametrize("n,hq,hkv,dim,page,kv,rot,inter,nhd,far", APPEND)
def test_append(n, hq, hkv, dim, page, kv, rot, inter, nhd, far):
    note("append", n, hq, hkv, dim, page, kv, rot, inter, nhd)
    t = torch()
    rng = np.random.default_rng(n + dim)
    pages = (n + page - 1) // page + 3
    pool = Pool(kv, pages, hkv, page, dim, rng, nhd, together=n % 2 == 1)
    cache = pool.upload()
    rows = rng.normal(size=(n, hq + 2 * hkv, dim)) * 2
    if n > 2:
        rows[2, hq + hkv, :4] = [np.inf, -np.inf, np.nan, 3e38]   # values reach the cache as they are
    fused = dev_bf16(rows.reshape(n, -1))
    x = vals(host_bits(fused)).reshape(n, hq + 2 * hkv, dim)
    q, k, v = fused.split([hq * dim, hkv * dim, hkv * dim], dim=1)
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    if n > 4:
        slots[1], slots[3] = -1, pages * page   # neither is stored
    pos = rng.integers(0, far, n).astype(np.int32)
    pos[0] = far - 1
    freq = 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    rope = trs.Rope(t.from_numpy(freq).cuda(), inter) if rot else None
    wide = t.full((n, hq * dim + 8), 7.0, dtype=t.bfloat16, device="cuda")   # rows of another stride
    q_out = wide[:, :hq * dim] if hq else None
    trs.dc_kv_append(cache, q if hq else None, k, v, dev_i32(pos) if rot else None, t.from_numpy(slots).cuda(), rope, q_out)
    t.cuda.synchronize()
    assert (wide[:, hq * dim:] == 7).all()
    ref = layer.rotate(x[:, :hq + hkv], pos, freq, inter)
    # the angle's fp32 fraction of half a turn (2^-24 pi), sine, cosine and three roundings of fp32: below 2^-20 of
    # the pair's entries; then one rounding to bf16
    size = np.abs(x).max(-1)[..., None]
    if hq:
        got = vals(host_bits(q_out)).reshape(n, hq, dim)
        err = np.abs(got - ref[:, :hq])
        assert (err <= BF16 * np.abs(ref[:, :hq]) + 2.0 ** -20 * size[:, :hq]).all()
        assert np.array_equal(got[..., rot:], x[:, :hq, rot:])
    gk, gv = pool.download()
    used = np.zeros((pages, page), bool)
    for i in range(n):
        if not 0 <= slots[i] < pages * page:
            continue
        p, s = divmod(int(slots[i]), page)
        used[p, s] = True
        if kv == "bf16":
            assert (np.abs(vals(gk[p, :, s]) - ref[i, hq:]) <= BF16 * np.abs(ref[i, hq:]) + 2.0 ** -20 * size[i, hq:hq + hkv]).all()
            assert np.array_equal(gv[p, :, s], host_bits(v).reshape(n, hkv, dim)[i])
            continue
        # x / scale in fp32 (2^-24), rounded to 3 bits behind the leading one (2^-4), or to a multiple of 2^-9
        for got, want, sc in ((gk, ref[i, hq:], pool.ks), (gv, x[i, hq + hkv:], pool.vs)):
            w = want / sc.astype(np.float64)[:, None]
            g = layer.e4m3_value(got[p, :, s])
            nan = np.isnan(w)
            assert np.array_equal(np.isnan(g), nan)
            w = np.clip(w, -448, 448)
            slack = 2.0 ** -20 * size[i, hq:hq + hkv] / sc[:, None] if got is gk else 0.0
            assert (np.abs(g - w)[~nan] <= (np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10) * (1 + 2.0 ** -20) + slack)[~nan]).all()
    for g in (gk, gv):
        assert (g.transpose(0, 2, 1, 3)[~used] == pool.nan).all()   # every other slot is as it was


def test_append_in_place_and_by_itself():
    """q rotated onto itself, in the middle of a fused row; angle 0 leaves everything as it is."""
    t = torch()
    note("append in place")
    rng = np.random.default_rng(5)
    n, hq, hkv, dim = 20, 4, 2, 128
    pool = Pool("bf16", 4, hkv, 16, dim, rng)
    cache = pool.upload()
    fused = dev_bf16(rng.normal(size=(n, (hq + 2 * hkv) * dim)))
    before = host_bits(fused).copy()
    q, k, v = fused[:, :hq * dim], fused[:, hq * dim:(hq + hkv) * dim], fused[:, (hq + hkv) * dim:]
    rope = trs.Rope(t.rand(64, dtype=t.float64, device="cuda"))
    slots = t.arange(n, dtype=t.int64, device="cuda")
    zero = t.zeros(n, dtype=t.int32, device="cuda")
    trs.dc_kv_append(cache, q, k, v, zero, slots, rope, q)
    assert np.array_equal(host_bits(fused), before)
    pos = t.arange(n, dtype=t.int32, device="cuda")
    out = t.empty((n, hq * dim), dtype=t.bfloat16, device="cuda")
    trs.dc_kv_append(cache, q, k, v, pos, slots, rope, out)
    trs.dc_kv_append(cache, q, k, v, pos, slots, rope, q)
    t.cuda.synchronize()
    assert np.array_equal(host_bits(q), host_bits(out))
    assert np.array_equal(host_bits(fused)[:, hq * dim:], before[:, hq * dim:])


# -------------------------------------------------------------- attention
class Case:
    """Sequences, groups and a cache with random contents, on the host and the GPU."""

    def __init__(self, seed, nq, kv_len, groups, prefix, hq, hkv, dim, page, kv, nhd=False, std=1.0, bounds=None):
        t = torch()
        rng = np.random.default_rng(seed)
        self.nq, self.kv_len, self.groups, self.prefix = list(nq), list(kv_len), list(groups), list(prefix)
        self.hq, self.hkv, self.dim, self.page = hq, hkv, dim, page
        pg = lambda n: (n + page - 1) // page  # noqa: E731
        total = sum(map(pg, kv_len)) + sum(map(pg, prefix)) + 2
        perm = rng.permutation(total)
        self.pool = Pool(kv, total, hkv, page, dim, rng, nhd, together=not nhd)
        at = 0
        self.tables, self.ptables = [], []
        for lens, tables in ((kv_len, self.tables), (prefix, self.ptables)):
            for n in lens:
                tables.append(perm[at:at + pg(n)])
                at += pg(n)
                for w in "kv":
                    self.pool.put(w, tables[-1], n, rng.normal(size=(n, hkv, dim)) * (std if w == "k" else 1.0), page)
        n = sum(nq)
        self.n = n
        self.q = vals(bits(rng.normal(size=(n, hq, dim)) * std))
        self.scale = dim ** -0.5
        # -1 (no page) past a sequence's pages, and columns beyond the longest
        def table(tabs):
            w = max([len(x) for x in tabs] + [0]) + 2
            a = np.full((max(1, len(tabs)), w), -1, np.int32)
            for i, x in enumerate(tabs):
                a[i, :len(x)] = x
            return dev_i32(a)
        self.q_start = dev_i32(np.concatenate([[0], np.cumsum(self.nq)]))
        gq = [sum(self.nq[a:b]) for a, b in zip(groups[:-1], groups[1:])]
        kw = {}
        if prefix:
            kw = dict(group_start=dev_i32(groups), prefix_len=dev_i32(prefix), prefix_pages=table(self.ptables),
                      max_prefix=max(prefix), max_group_q=max(gq))
        b = bounds or {}
        self.dlen = dev_i32(self.kv_len)
        self.batch = trs.AttnBatch(self.q_start, self.dlen, table(self.tables), b.get("max_q", max(self.nq + [0])),
                                   b.get("max_kv", max(self.kv_len + [0])), **kw)
        self.reload()

    def reload(self):
        self.cache = self.pool.upload()

    def run(self, extra=3):
        """The output bits [n + extra][hq][dim]; the rows behind the last sequence hold a mark."""
        t = torch()
        n = self.n + extra
        q = np.zeros((n, self.hq * self.dim))
        q[:self.n] = self.q.reshape(self.n, -1)
        self.dq = dev_bf16(q)
        self.dy = t.full((n, self.hq * self.dim), -5.0, dtype=t.bfloat16, device="cuda")
        self.ws = t.full((trs.dc_attention_workspace_bytes(self.cache, self.batch, self.hq, n),), 255, dtype=t.uint8, device="cuda")
        trs.dc_attention(self.cache, self.dq, self.batch, self.scale, self.dy, self.ws)
        t.cuda.synchronize()
        y = host_bits(self.dy).reshape(n, self.hq, self.dim)
        assert (vals(y[self.n:]) == -5.0).all(), "rows behind the last sequence were written"
        return y[:self.n]

    def reference(self):
        """(y, tolerance) [n][hq][dim].

        Let a weight's relative error be e: its rounding to bf16 (2^-8) and, before it, the score's error.  The score
        is an fp32 sum of dim products (each of the at most dim + 8 roundings 2^-23 of sum |q_i k_i|), scaled and
        subtracted from the running maximum (3 roundings of 2^-23 of at most the same size); an exponential to 2^-22.
        Numerator and denominator hold the same weights, so y moves by at most e / (1 - e) sum w |v - y|.  The fp32
        sums over m keys cost (m + 40) 2^-23 of sum w |v|; the result is rounded once (2^-8)."""
        k, v = self.pool.values("k"), self.pool.values("v")
        ys, tols = [], []
        at = 0
        for b, n in enumerate(self.nq):
            own = self.kv_len[b]
            kk, vv = (layer.gather(a, self.tables[b], own, self.page) for a in (k, v))
            see = np.arange(own)[None] <= np.arange(n)[:, None] + own - n
            for g in range(len(self.prefix)):
                if self.groups[g] <= b < self.groups[g + 1]:
                    pk, pv = (layer.gather(a, self.ptables[g], self.prefix[g], self.page) for a in (k, v))
                    kk, vv = np.concatenate([pk, kk]), np.concatenate([pv, vv])
                    see = np.concatenate([np.ones((n, self.prefix[g]), bool), see], 1)
            y, spread, size, reach = layer.attend(self.q[at:at + n], kk, vv, see, self.scale)
            e = BF16 + 2.0 ** -22 + (self.dim + 11) * 2.0 ** -23 * self.scale * reach[..., None] * 1.4427
            ys.append(y)
            tols.append(e / (1 - e) * spread + (kk.shape[0] + 40) * 2.0 ** -23 * size + BF16 * 1.01 * np.abs(y))
            at += n
        z = np.zeros((0, self.hq, self.dim))
        return np.concatenate(ys + [z]), np.concatenate(tols + [z])

    def check(self):
        got = vals(self.run())
        y, tol = self.reference()
        err = np.abs(got - y)
        worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
        rel = float(np.linalg.norm(got - y) / max(np.linalg.norm(y), 1e-300)) if err.size else 0.0
        print("[attention] worst error / bound %.3f, rel L2 %.2e" % (worst, rel), flush=True)
        assert np.isfinite(got).all()
        assert (err <= tol).all()


ATT = {
    "one key": dict(nq=[1], kv_len=[1], groups=[0], prefix=[], hq=4, hkv=4, dim=128, page=16, kv="bf16"),
    "one sequence": dict(nq=[1], kv_len=[1000], groups=[0], prefix=[], hq=8, hkv=8, dim=128, page=16, kv="bf16"),
    "no key at all": dict(nq=[1, 2], kv_len=[0, 1], groups=[0], prefix=[], hq=8, hkv=2, dim=64, page=16, kv="bf16"),
    "odd lengths": dict(nq=[1, 1, 1, 1, 1, 1], kv_len=[15, 16, 17, 31, 33, 129], groups=[0], prefix=[], hq=12, hkv=4,
                        dim=128, page=16, kv="bf16"),
    "e4m3": dict(nq=[1, 1, 1], kv_len=[15, 64, 333], groups=[0], prefix=[], hq=12, hkv=4, dim=128, page=32, kv="e4m3", nhd=True),
    "dim 64": dict(nq=[1, 1, 1], kv_len=[15, 64, 333], groups=[0], prefix=[], hq=12, hkv=4, dim=64, page=32, kv="bf16", nhd=True),
    "dim 64 e4m3": dict(nq=[1, 3, 1], kv_len=[15, 64, 333], groups=[0], prefix=[], hq=6, hkv=1, dim=64, page=64, kv="e4m3"),
    "one group": dict(nq=[1] * 5, kv_len=[0, 1, 40, 17, 300], groups=[0, 5], prefix=[777], hq=8, hkv=2, dim=128, page=16, kv="bf16"),
    "groups, some without sequences or prefix": dict(
        nq=[1, 2, 1, 0, 1, 4, 1], kv_len=[5, 2, 40, 17, 300, 4, 0], groups=[1, 1, 3, 3, 6], prefix=[50, 0, 31, 260],
        hq=16, hkv=2, dim=128, page=32, kv="bf16"),
    "groups e4m3": dict(nq=[1] * 9, kv_len=[3] * 4 + [90] * 5, groups=[0, 4, 9], prefix=[513, 40], hq=8, hkv=2, dim=128,
                        page=16, kv="e4m3", nhd=True),
    "many rows on a prefix": dict(nq=[1] * 40, kv_len=[1 + i for i in range(40)], groups=[0, 37, 40], prefix=[400, 33],
                                  hq=8, hkv=4, dim=128, page=16, kv="bf16"),
    "many rows on a prefix, dim 64": dict(nq=[1] * 40, kv_len=[1 + i for i in range(40)], groups=[0, 37, 40], prefix=[400, 33],
                                          hq=8, hkv=4, dim=64, page=16, kv="e4m3"),
    "drafted tokens": dict(nq=[5, 8, 0, 3, 1], kv_len=[40, 8, 9, 200, 77], groups=[0, 2, 5], prefix=[100, 35], hq=8, hkv=8,
                           dim=128, page=16, kv="bf16"),
    "drafted tokens, more rows": dict(nq=[5, 8, 0, 3, 8], kv_len=[40, 8, 9, 200, 77], groups=[0, 2, 5], prefix=[100, 35], hq=20,
                                      hkv=4, dim=128, page=16, kv="bf16"),
    "queries before any key": dict(nq=[6, 20], kv_len=[2, 0], groups=[0], prefix=[], hq=8, hkv=2, dim=128, page=16, kv="bf16"),
    "a short prompt": dict(nq=[70], kv_len=[70], groups=[0], prefix=[], hq=4, hkv=2, dim=128, page=16, kv="bf16"),
    "prompts": dict(nq=[130, 33, 257, 1, 0], kv_len=[130, 90, 300, 17, 5], groups=[0, 1, 4], prefix=[70, 129], hq=32, hkv=32,
                    dim=128, page=16, kv="bf16"),
    "prompts, shared heads": dict(nq=[100, 33], kv_len=[130, 33], groups=[1, 2], prefix=[70], hq=64, hkv=64, dim=64, page=32,
                                  kv="bf16"),
    "prompts e4m3": dict(nq=[100, 33, 64], kv_len=[130, 33, 64], groups=[0, 2], prefix=[45], hq=144, hkv=48, dim=128, page=64,
                         kv="e4m3"),
    "prompts e4m3, dim 64": dict(nq=[100, 3], kv_len=[99, 33], groups=[0, 2], prefix=[45], hq=128, hkv=64, dim=64, page=64,
                                 kv="e4m3"),
    "large scores": dict(nq=[1, 40, 3], kv_len=[500, 80, 9], groups=[0, 3], prefix=[200], hq=8, hkv=4, dim=128, page=16, kv="bf16",
                         std=6.0),
    "loose bounds": dict(nq=[1, 1], kv_len=[5, 70], groups=[0], prefix=[], hq=8, hkv=4, dim=128, page=16, kv="bf16",
                         bounds=dict(max_q=3, max_kv=96)),
}


@pytest.mark.parametrize("name", list(ATT))
def test_attention(name):
    note("attention", name)
    Case(len(name), **ATT[name]).check()


def test_attention_of_a_batch_without_keys():
    """No key anywhere, a bound of none and a page table without columns: zeros."""
    t = torch()
    note("attention, no keys")
    c = Case(1, nq=[2, 1], kv_len=[0, 0], groups=[0], prefix=[], hq=4, hkv=2, dim=128, page=16, kv="bf16")
    c.batch = trs.AttnBatch(c.q_start, c.dlen, t.empty((2, 0), dtype=t.int32, device="cuda"), 2, 0)
    assert (vals(c.run()) == 0).all()


@pytest.mark.parametrize("name", ["drafted tokens", "prompts", "many rows on a prefix", "groups e4m3"])
def test_attention_repeats_bit_for_bit(name):
    note("attention twice", name)
    c = Case(3, **ATT[name])
    a = c.run()
    assert np.array_equal(a, c.run())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", ["drafted tokens, more rows", "prompts, shared heads"])
def test_attention_does_not_see_later_tokens(name, kv):
    """A later query token's key and value of infinity and NaN reach that token and those behind it only."""
    t = torch()
    note("attention, later tokens", name, kv)
    c = Case(4, **dict(ATT[name], kv=kv))
    clean = c.run().copy()
    b, n = 0, c.nq[0]
    j = n - 2                                    # its key is own key kv_len - n + j
    i = c.kv_len[b] - n + j
    p, s = c.tables[b][i // c.page], i % c.page
    nan, inf = (0x7FC0, 0x7F80) if kv == "bf16" else (0x7F, 0xFF)
    c.pool.v[p, :, s, ::2] = nan
    c.pool.v[p, :, s, 1::2] = inf
    c.pool.k[p, :, s, 3] = nan
    c.reload()
    got = c.run()
    assert np.array_equal(got[:j], clean[:j])
    assert np.isnan(vals(got[j:n])).all()
    assert np.array_equal(got[n:], clean[n:])


def test_attention_infinite_value_that_is_seen():
    note("attention, infinities")
    c = Case(5, nq=[1], kv_len=[40], groups=[0], prefix=[], hq=2, hkv=2, dim=128, page=16, kv="bf16")
    p, s = c.tables[0][1], 4
    c.pool.v[p, 0, s, 5] = 0x7F80
    c.reload()
    y = vals(c.run())
    assert y[0, 0, 5] == np.inf and np.isfinite(np.delete(y[0, 0], 5)).all() and np.isfinite(y[0, 1]).all()


def test_attention_page_numbers_outside_the_cache():
    """A table entry outside the cache spoils its own sequence only."""
    note("attention, bad pages")
    c = Case(6, nq=[1, 1, 1], kv_len=[100, 200, 60], groups=[0, 2], prefix=[50], hq=8, hkv=2, dim=128, page=16, kv="bf16")
    good = c.run().copy()
    t = torch()
    pages = c.batch._keep[2]
    pages[1, 3], pages[1, 5] = 1 << 30, -7
    t.cuda.synchronize()
    got = c.run()
    assert np.array_equal(got[[0, 2]], good[[0, 2]])


def test_attention_lengths_beyond_the_bounds_stay_inside():
    """Lengths above the host's bounds are cut; the other sequences are as before."""
    note("attention, lengths past the bounds")
    c = Case(7, nq=[1, 1, 1], kv_len=[100, 96, 60], groups=[0], prefix=[], hq=8, hkv=2, dim=128, page=16, kv="bf16")
    good = c.run().copy()
    c.dlen[1] = 1 << 30
    got = c.run()
    assert np.array_equal(got[[0, 2]], good[[0, 2]])
    c.dlen[1] = -4
    got = c.run()
    assert np.array_equal(got[[0, 2]], good[[0, 2]]) and (vals(got[1]) == 0).all()


def test_attention_far_pages():
    """A cache whose pages lie beyond 2^32 bytes."""
    t = torch()
    note("attention, a cache of 6 GB")
    rng = np.random.default_rng(8)
    hkv, page, dim, n = 8, 64, 128, 200
    pages = (6 << 30) // (2 * hkv * page * dim * 2)
    one = t.zeros((pages, 2, hkv, page, dim), dtype=t.bfloat16, device="cuda")
    table = np.array([pages - 1, 3, pages - 2, pages // 2], np.int32)
    cache = trs.KvCache(one[:, 0], one[:, 1])
    k, v = (vals(bits(rng.normal(size=(n, hkv, dim)))) for _ in range(2))
    slots = table[np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
    trs.dc_kv_append(cache, None, dev_bf16(k.reshape(n, -1)), dev_bf16(v.reshape(n, -1)), None, t.from_numpy(slots).cuda(),
                     None, None)
    q = vals(bits(rng.normal(size=(1, hkv, dim))))
    batch = trs.AttnBatch(dev_i32([0, 1]), dev_i32([n]), dev_i32(table[None]), 1, n)
    y = t.empty((1, hkv * dim), dtype=t.bfloat16, device="cuda")
    ws = t.empty(trs.dc_attention_workspace_bytes(cache, batch, hkv, 1), dtype=t.uint8, device="cuda")
    trs.dc_attention(cache, dev_bf16(q.reshape(1, -1)), batch, dim ** -0.5, y, ws)
    want, spread, size, _ = layer.attend(q, k, v, np.ones((1, n), bool), dim ** -0.5)
    assert (np.abs(vals(host_bits(y)).reshape(1, hkv, dim) - want) <= 1.1 * BF16 * (spread + np.abs(want)) + 1e-4 * size).all()


def test_attention_captured_and_replayed():
    """A captured step follows the lengths, tables and tokens that change between its replays."""
    t = torch()
    note("attention, captured")
    c = Case(9, nq=[1, 1, 1, 1], kv_len=[100, 200, 60, 5], groups=[0, 2, 4], prefix=[50, 120], hq=8, hkv=2, dim=128, page=16, kv="bf16")
    c.run()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        trs.dc_attention(c.cache, c.dq, c.batch, c.scale, c.dy, c.ws)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        trs.dc_attention(c.cache, c.dq, c.batch, c.scale, c.dy, c.ws)
    for step, lens in enumerate(([100, 200, 60, 5], [99, 7, 0, 4], [1, 200, 60, 5], [100, 199, 33, 2])):
        c.dlen.copy_(dev_i32(lens))
        c.dq.copy_(c.dq.roll(1, 0))
        c.dy.fill_(-5.0)
        g.replay()
        t.cuda.synchronize()
        got = c.dy.clone()
        c.ws.fill_(255)
        trs.dc_attention(c.cache, c.dq, c.batch, c.scale, c.dy, c.ws)
        t.cuda.synchronize()
        assert t.equal(got.view(t.int16), c.dy.view(t.int16)), step


def test_attention_on_two_streams():
    """Two calls at once, each with its own workspace and output, as one after the other."""
    t = torch()
    note("attention, two streams")
    cs = [Case(10 + i, nq=[1] * 8, kv_len=[300 + i] * 8, groups=[0, 8], prefix=[500], hq=8, hkv=8, dim=128, page=16, kv="bf16")
          for i in range(2)]
    want = [c.run().copy() for c in cs]
    streams = [t.cuda.Stream() for _ in cs]
    t.cuda.synchronize()
    for _ in range(3):
        for c in cs:
            c.dy.fill_(0)
        t.cuda.synchronize()
        for c, s in zip(cs, streams):
            with t.cuda.stream(s):
                trs.dc_attention(c.cache, c.dq, c.batch, c.scale, c.dy, c.ws)
        t.cuda.synchronize()
        for c, w in zip(cs, want):
            assert np.array_equal(host_bits(c.dy).reshape(-1, c.hq, c.dim)[:c.n], w)


# ------------------------------------------------------------------ 4-bit
def w4_case(rng, out, inn):
    codes = rng.integers(0, 16, size=(out, inn))
    scale = np.exp(rng.normal(size=(inn // 128, out)) * 0.5 - 5).astype(np.float16)
    zero = rng.integers(0, 16, size=(inn // 128, out)).astype(np.float16)
    t = torch()
    buf = layer.w4_pack(codes, scale, zero)
    assert buf.size == trs.dc_w4_bytes(out, inn)
    return codes, scale, zero, trs.W4View(out, inn, t.from_numpy(buf).cuda())


def w4_reference(codes, scale, zero, x):
    """(y, tolerance): the fp32 sums hold codes of up to 143 times |x| (and as much again taken off), each through at
    most 36 + 8 roundings of 2^-23; the sums over the groups add one each; the result is rounded once."""
    y = x @ layer.w4_matrix(codes, scale, zero).T
    mag = np.zeros_like(y)
    for g in range(scale.shape[0]):
        mag += np.abs(x[:, 128 * g:128 * g + 128]).sum(1)[:, None] * scale[g].astype(np.float64)
    return y, BF16 * np.abs(y) + (44 * 2 * 143 + scale.shape[0] * 16) * 2.0 ** -23 * mag


@pytest.mark.parametrize("t_,out,inn", [(1, 128, 128), (1, 512, 1152), (3, 384, 4096), (16, 128, 1280), (17, 256, 256),
                                        (33, 640, 384), (64, 128, 2048), (65, 1920, 640), (200, 384, 256)])
def test_w4(t_, out, inn):
    t = torch()
    note("w4", t_, out, inn)
    rng = np.random.default_rng(t_ + out)
    codes, scale, zero, view = w4_case(rng, out, inn)
    x = vals(bits(rng.normal(size=(t_, inn))))
    y = t.full((t_, out), float("nan"), dtype=t.bfloat16, device="cuda")
    xd = dev_bf16(x)
    trs.dc_apply_w4(view, xd, y)
    t.cuda.synchronize()
    first = host_bits(y).copy()
    want, tol = w4_reference(codes, scale, zero, x)
    err = np.abs(vals(first) - want)
    print("[w4] worst error / bound %.3f, rel L2 %.2e" % ((err / tol).max(), np.linalg.norm(err) / np.linalg.norm(want)), flush=True)
    assert (err <= tol).all()
    trs.dc_apply_w4(view, xd, y)
    assert np.array_equal(host_bits(y), first)


def test_w4_pack():
    """The device packer against the oracle's quantizer at 4 bits, edge groups included."""
    from oracle import quant
    t = torch()
    note("w4 pack")
    rng = np.random.default_rng(3)
    out, inn = 256, 384
    w = vals(bits(rng.normal(size=(out, inn)) * 0.02))
    w[0, :128] = 0.0
    w[1, :128] = 0.5
    w[2, :128] = -np.abs(w[2, :128])
    w[3, 128:256] = np.abs(w[3, 128:256])
    w[4, :128] = vals(bits(1e-9 * np.ones(128)))   # the scale is below fp16's smallest: 1
    dst = t.empty(trs.dc_w4_bytes(out, inn), dtype=t.uint8, device="cuda")
    flag = t.full((1,), 9, dtype=t.int32, device="cuda")
    trs.dc_w4_pack_device(dev_bf16(w), dst, flag)
    codes, scale, zero = (np.stack(a) for a in zip(*(quant.quantize_vector(r, 4) for r in w)))
    scale, zero = scale.T, np.abs(zero.T)   # -0.0 counts as 0
    assert int(flag.item()) == 0
    assert np.array_equal(dst.cpu().numpy(), layer.w4_pack(codes.astype(np.int64), scale, zero))
    for bad in (np.nan, np.inf, 3e38):
        w2 = w.copy()
        w2[17, 200] = bad
        trs.dc_w4_pack_device(dev_bf16(w2), dst, flag)
        assert int(flag.item()) == 1


# ------------------------------------------------------------ all together
def test_layer_step_of_many_tenants():
    """q, k and v of a grouped-query layer by the multi-tenant call, rotated and appended, attention over the tenants'
    shared prompts, and the output matrix at 4 bits: each operator against its oracle on the inputs it had."""
    t = torch()
    note("layer step")
    rng = np.random.default_rng(11)
    hq, hkv, dim, hidden, page = 4, 2, 64, 256, 16
    shapes = [(hq * dim, hidden), (hkv * dim, hidden), (hkv * dim, hidden)]
    ids = np.array([0, 0, 0, 1, 1, 2], np.int32)            # sorted by tenant: its sequences are a group
    T = ids.size
    ds = [[synth.small_delta(50 + 10 * j + k, *sh, 2, 8, 22) for k in range(3)] for j, sh in enumerate(shapes)]
    views = [[upload(d.spec, d) for d in row] for row in ds]
    x = vals(bits(rng.normal(size=(T, hidden))))
    ys = [t.empty((T, sh[0]), dtype=t.int16, device="cuda") for sh in shapes]
    ws = t.empty(trs.dc_group_workspace_bytes([d.spec for row in ds for d in row], 3, T), dtype=t.uint8, device="cuda")
    xb = t.from_numpy(bits(x).view(np.int16)).cuda()
    w = [t.from_numpy(synth.base_weight(rng, *sh).view(np.int16)).cuda() for sh in shapes]

    lens = np.array([20, 1, 33, 7, 16, 40], np.int32)       # with the new token
    prefix = [70, 33, 5]
    c = Case(12, nq=[1] * T, kv_len=lens, groups=[0, 3, 5, 6], prefix=prefix, hq=hq, hkv=hkv, dim=dim, page=page, kv="bf16")
    for b in range(T):                                      # the new token's slot is still empty
        i = lens[b] - 1
        for a in (c.pool.k, c.pool.v):
            a[c.tables[b][i // page], :, i % page] = c.pool.nan
    c.reload()
    pos = np.array([prefix[ids[b]] + lens[b] - 1 for b in range(T)], np.int32)
    slots = np.array([c.tables[b][(lens[b] - 1) // page] * page + (lens[b] - 1) % page for b in range(T)], np.int64)
    freq = 10000.0 ** (-np.arange(dim // 2) * 2.0 / dim)
    rope = trs.Rope(t.from_numpy(freq).cuda())
    att = t.empty((T, hq * dim), dtype=t.bfloat16, device="cuda")
    aws = t.empty(trs.dc_attention_workspace_bytes(c.cache, c.batch, hq, T), dtype=t.uint8, device="cuda")
    codes, scale, zero, o4 = w4_case(rng, hidden, hq * dim)
    out = t.empty((T, hidden), dtype=t.bfloat16, device="cuda")
    idd, posd, slotd = dev_i32(ids), dev_i32(pos), t.from_numpy(slots).cuda()

    def step():
        trs.dc_apply_multitenant_group(views, w, xb, idd, ys, ws)
        trs.dc_kv_append(c.cache, ys[0], ys[1], ys[2], posd, slotd, rope, att)
        trs.dc_attention(c.cache, att, c.batch, dim ** -0.5, out4, aws)
        trs.dc_apply_w4(o4, out4, out)

    out4 = t.empty((T, hq * dim), dtype=t.bfloat16, device="cuda")
    step()
    t.cuda.synchronize()
    q, k, v = (vals(y.cpu().numpy().view(np.uint16)).reshape(T, -1, dim) for y in ys)
    qr = layer.rotate(q, pos, freq, False)
    got_q = vals(host_bits(att)).reshape(T, hq, dim)
    assert (np.abs(got_q - qr) <= BF16 * np.abs(qr) + 2.0 ** -20 * np.abs(q).max()).all()
    gk, gv = c.pool.download()
    kr = layer.rotate(k, pos, freq, False)
    for b in range(T):
        p, s = divmod(int(slots[b]), page)
        assert (np.abs(vals(gk[p, :, s]) - kr[b]) <= BF16 * np.abs(kr[b]) + 2.0 ** -20 * np.abs(k).max()).all()
        assert np.array_equal(vals(gv[p, :, s]), v[b])
    c.pool.k, c.pool.v, c.q = gk, gv, got_q                 # attention on what it was given
    want, tol = c.reference()
    got = vals(host_bits(out4)).reshape(T, hq, dim)
    assert (np.abs(got - want) <= tol).all()
    want, tol = w4_reference(codes, scale, zero, got.reshape(T, -1))
    assert (np.abs(vals(host_bits(out)) - want) <= tol).all()
    # the whole step captured: the same bits on every replay
    first = host_bits(out).copy()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step()
    for _ in range(3):
        out.zero_()
        g.replay()
        t.cuda.synchronize()
        assert np.array_equal(host_bits(out), first)


# ------------------------------------------------- further calls of each
def test_append_every_bit_pattern():
    """Without a rotation every bf16 number, subnormal ones and infinities included, passes as it is (NaN as some NaN)."""
    t = torch()
    note("append, every bit pattern")
    n, dim = 512, 128
    pool = Pool("bf16", n // 16, 1, 16, dim, np.random.default_rng(0))
    cache = pool.upload()
    every = np.arange(1 << 16, dtype=np.uint16)
    x = t.from_numpy(every.view(np.int16).reshape(n, dim)).cuda().view(t.bfloat16)
    out = t.zeros_like(x)
    trs.dc_kv_append(cache, x, x, x, None, t.arange(n, dtype=t.int64, device="cuda"), None, out)
    t.cuda.synchronize()
    nan = np.isnan(vals(every))
    for got in [host_bits(out)] + pool.download():
        got = got.reshape(-1)
        assert np.array_equal(got[~nan], every[~nan]) and np.isnan(vals(got[nan])).all()


def test_append_captured_on_another_stream():
    """Replays follow the positions and slots that changed since; every other slot stays."""
    t = torch()
    note("append, captured")
    rng = np.random.default_rng(6)
    n, hq, hkv, dim, pages = 5, 4, 2, 64, 3
    rope = trs.Rope(t.rand(dim // 2, dtype=t.float64, device="cuda"))
    q, k, v = (dev_bf16(rng.normal(size=(n, h * dim))) for h in (hq, hkv, hkv))
    pos, slots = t.zeros(n, dtype=t.int32, device="cuda"), t.zeros(n, dtype=t.int64, device="cuda")
    pools = [Pool("bf16", pages, hkv, 16, dim, rng) for _ in range(2)]
    caches = [p.upload() for p in pools]
    outs = [t.zeros_like(q) for _ in range(2)]
    side = t.cuda.Stream()
    g = t.cuda.CUDAGraph()
    slots.copy_(t.arange(n))
    t.cuda.synchronize()
    with t.cuda.graph(g, stream=side):
        trs.dc_kv_append(caches[0], q, k, v, pos, slots, rope, outs[0])
    for step in range(4):
        pos.copy_(dev_i32(rng.integers(0, 5000, n)))
        slots.copy_(t.from_numpy(rng.permutation(pages * 16)[:n].astype(np.int64)))
        t.cuda.synchronize()
        with t.cuda.stream(side):
            g.replay()
        trs.dc_kv_append(caches[1], q, k, v, pos, slots, rope, outs[1])
        t.cuda.synchronize()
        assert np.array_equal(host_bits(outs[0]), host_bits(outs[1])), step
        for a, b in zip(*(p.download() for p in pools)):
            assert np.array_equal(a, b), step


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq", [[1, 1], [1] * 6, [1] * 12, [5, 3], [5, 8], [9, 1, 14]])
def test_attention_rows_of_every_number(nq, dim, kv):
    """4 query heads a kv head: up to 16, up to 32 and more rows of own keys and of a prefix."""
    note("attention, rows", nq, dim, kv)
    own = [200 + 37 * i for i in range(len(nq))]
    Case(len(nq) + dim, nq=nq, kv_len=own, groups=[0, len(nq)], prefix=[301], hq=8, hkv=2, dim=dim, page=16, kv=kv).check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [2, 5])
def test_attention_of_few_rows_does_not_see_later_tokens(heads, dim, kv):
    """12 and 30 rows of a kv head: infinities and NaN of a later token reach it and those behind it only."""
    note("attention, later tokens, few rows", heads, dim, kv)
    c = Case(heads, nq=[6, 3], kv_len=[150, 40], groups=[0], prefix=[], hq=2 * heads, hkv=2, dim=dim, page=16, kv=kv)
    clean = c.run().copy()
    i = 150 - 6 + 4                              # the key of query token 4
    p, s = c.tables[0][i // c.page], i % c.page
    nan, inf = (0x7FC0, 0x7F80) if kv == "bf16" else (0x7F, 0xFF)
    c.pool.v[p, :, s, ::2] = nan
    c.pool.v[p, :, s, 1::2] = inf
    c.reload()
    got = c.run()
    assert np.array_equal(got[:4], clean[:4]) and np.array_equal(got[6:], clean[6:])
    assert not np.isfinite(vals(got[4:6])).any()


@pytest.mark.parametrize("name", ["odd lengths", "one key", "groups e4m3", "drafted tokens, more rows", "prompts",
                                  "prompts, shared heads"])
def test_attention_rows_in_front_of_the_first_sequence(name):
    """They stay as they are, like those behind the last; the sequences' results do not depend on where they lie."""
    t = torch()
    note("attention, rows in front", name)
    c = Case(21, **ATT[name])
    want = c.run().copy()
    c.q_start.add_(2)
    c.dq[2:c.n + 2] = c.dq[:c.n].clone()
    c.dq[:2] = float("nan")
    c.dy.fill_(-5.0)
    trs.dc_attention(c.cache, c.dq, c.batch, c.scale, c.dy, c.ws)
    t.cuda.synchronize()
    got = host_bits(c.dy).reshape(-1, c.hq, c.dim)
    assert (vals(got[:2]) == -5.0).all() and (vals(got[c.n + 2:]) == -5.0).all()
    assert np.array_equal(got[2:c.n + 2], want)


def test_attention_two_graphs_on_one_workspace():
    """Nothing is kept in a workspace: two captured calls that use the same one, replayed in turn."""
    t = torch()
    note("attention, one workspace")
    cs = [Case(30 + i, **ATT[n]) for i, n in enumerate(["groups e4m3", "many rows on a prefix"])]
    want = [c.run().copy() for c in cs]
    ws = max((c.ws for c in cs), key=lambda w: w.numel())
    graphs = []
    for c in cs:
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            trs.dc_attention(c.cache, c.dq, c.batch, c.scale, c.dy, ws)
        graphs.append(g)
    for step in range(3):
        for c in cs:
            c.dy.fill_(-5.0)
        for g in graphs[::1 if step % 2 else -1]:
            g.replay()
        t.cuda.synchronize()
        for c, w in zip(cs, want):
            assert np.array_equal(host_bits(c.dy).reshape(-1, c.hq, c.dim)[:c.n], w), step


@pytest.mark.parametrize("t_", [1, 40])
def test_w4_captured_and_what_is_not_finite(t_):
    """Replays follow x; a token that is not finite spoils its own row only; nothing behind y's rows is written."""
    t = torch()
    note("w4 captured", t_)
    rng = np.random.default_rng(40 + t_)
    out, inn = 384, 640
    view = w4_case(rng, out, inn)[3]
    x = dev_bf16(rng.normal(size=(t_ + 1, inn)))
    y = t.full((t_ + 2, out), -5.0, dtype=t.bfloat16, device="cuda")
    want = t.empty((t_, out), dtype=t.bfloat16, device="cuda")
    g = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(g):
        trs.dc_apply_w4(view, x[:t_], y[:t_])
    for step in range(3):
        x.copy_(x.roll(1, 0))
        g.replay()
        trs.dc_apply_w4(view, x[:t_], want)
        t.cuda.synchronize()
        assert np.array_equal(host_bits(y[:t_]), host_bits(want)) and (y[t_:] == -5).all(), step
    x[0, 77] = float("inf")
    g.replay()
    t.cuda.synchronize()
    assert not t.isfinite(y[0]).any() and np.array_equal(host_bits(y[1:t_]), host_bits(want[1:]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_of_a_single_prompt(kv):
    """64 blocks of 128 rows: few keys are walked whole, more are split."""
    for own in (256, 900):
        note("attention, one prompt", own, kv)
        Case(50 + own, nq=[256], kv_len=[own], groups=[0], prefix=[], hq=32, hkv=8, dim=64, page=16, kv=kv).check()


# 4 rows of a kv head; 20; 40: each walk of the keys.  With large scores most weights are 0 in 32 bits and the running
# maximum jumps by more than 2^149.
@pytest.mark.parametrize("std", [1.0, 12.0])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gq", [4, 20, 40])
def test_attention_every_visible_infinity(gq, dim, std):
    """An infinite value that a row sees makes its result infinite (every weight is positive), whichever key it is, the
    heaviest and the lightest included; two of different signs make NaN.  The other elements stay as they are."""
    note("attention, every visible infinity", gq, dim, std)
    n, keys, hkv, page = 71, 70, 2, 16
    c = Case(gq + dim, nq=[1] * n, kv_len=[keys] * n, groups=[0], prefix=[], hq=gq * hkv, hkv=hkv, dim=dim, page=page, kv="bf16", std=std)
    at = lambda b, i: (c.tables[b][i // page], 0, i % page, 7 * b % dim)  # noqa: E731
    spots = [(b, b, 0x7F80 if b % 2 else 0xFF80) for b in range(keys)] + [(keys, 1, 0x7F80), (keys, 40, 0xFF80)]
    for b, i, _ in spots:
        c.pool.v[at(b, i)] = 0
    y, tol = c.reference()
    for b, i, w in spots:
        c.pool.v[at(b, i)] = w
    c.reload()
    got = vals(c.run())
    rest = np.ones(got.shape, bool)
    for b in range(n):
        e = 7 * b % dim
        rest[b, :gq, e] = False
        want = np.nan if b == keys else np.inf if b % 2 else -np.inf
        assert np.array_equal(got[b, :gq, e], np.full(gq, want), equal_nan=True), (b, got[b, :gq, e])
    assert (np.abs(got - y) <= tol)[rest].all()


@pytest.mark.parametrize("prefix", [0, 150])
@pytest.mark.parametrize("std", [1.0, 12.0])
def test_attention_visible_infinities_of_a_prompt(prefix, std):
    """A block that walks all keys of its rows: an infinite value reaches every token that sees it, own key or prefix, and
    nothing else."""
    note("attention, visible infinities of a prompt", prefix, std)
    heads, n, own, page, dim = 64, 70, 200, 16, 64
    c = Case(prefix + 3, nq=[n], kv_len=[own], groups=[0, 1] if prefix else [0], prefix=[prefix] if prefix else [], hq=heads, hkv=heads,
             dim=dim, page=page, kv="bf16", std=std)
    spots = []                                   # head, key (of the prefix and the own keys behind it), element
    for h in range(heads):
        i = h * 5 % (prefix + own)
        t, j = (c.ptables[0], i) if i < prefix else (c.tables[0], i - prefix)
        spots.append((h, i, (t[j // page], h, j % page, 3 * h % dim)))
    for _, _, s in spots:
        c.pool.v[s] = 0
    y, tol = c.reference()
    for _, _, s in spots:
        c.pool.v[s] = 0x7F80
    c.reload()
    got = vals(c.run())
    for h, i, s in spots:
        sees = i - prefix <= np.arange(n) + own - n
        assert (got[sees, h, s[3]] == np.inf).all(), (h, i)
        y[sees, h, s[3]] = got[sees, h, s[3]] = 0.0
    assert (np.abs(got - y) <= tol).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gq", [4, 20, 40])
def test_attention_large_finite_values(gq, dim):
    """Values up to 2^115 by the number of keys stay finite (a weight is 2^12 at most, so the sums stay below 2^128)."""
    note("attention, large finite values", gq, dim)
    c = Case(gq, nq=[1, 2], kv_len=[70, 66], groups=[0], prefix=[], hq=2 * gq, hkv=2, dim=dim, page=16, kv="bf16", std=3.0)
    v = vals(c.pool.v)
    v *= 2.0 ** 115 / 70 / np.nanmax(np.abs(v))
    c.pool.v = bits(v)
    c.reload()
    c.check()


# The tile that the launcher takes (16-row tiles of the matrix x 16-token tiles of a block), tokens, rows, inputs: each tile,
# with rows that fill the last block in part (of 3 and 6 row tiles; rows come by 8) and tokens that do.
W4_TILES = [((1, 1), 5, 640, 1152), ((2, 1), 3, 4224, 256), ((3, 1), 7, 8320, 256), ((3, 1), 16, 11008, 128), ((4, 1), 9, 12416, 256),
            ((4, 1), 64, 4096, 256), ((6, 1), 2, 16640, 256), ((8, 1), 33, 8320, 256), ((2, 2), 17, 4224, 1152), ((4, 2), 19, 8448, 256),
            ((6, 2), 17, 16640, 256), ((6, 2), 64, 11008, 128), ((8, 2), 45, 12416, 256), ((8, 2), 33, 12544, 1152)]


def w4_tile(tokens, out):
    """The launcher's rule once more."""
    def cost(tile):
        rt, tok = tile[0], 16 * tile[1]
        blocks = -(-out // 16 // rt) * -(-tokens // tok)
        return (blocks + 255) // 256 * (17 * rt + 4 * min(tokens, tok))
    return min([(1, 1), (2, 1), (3, 1), (4, 1), (6, 1), (8, 1), (2, 2), (4, 2), (6, 2), (8, 2)], key=cost)


@pytest.mark.parametrize("tile,t_,out,inn", W4_TILES)
def test_w4_every_tile(tile, t_, out, inn):
    src = open(os.path.join(os.path.dirname(trs.__file__), "csrc", "k_w4.hip")).read()
    assert "const int64_t cost = (blocks + 255) / 256 * (17 * rt + 4 * (a.T < tok ? a.T : tok));" in src, "another rule: other cases"
    assert w4_tile(t_, out) == tile
    test_w4(t_, out, inn)


def test_w4_tiles_are_all_there():
    assert len({c[0] for c in W4_TILES}) == 10


# Paths that only long keys or other numbers of heads take.  A range of keys is at most 1/64 of them and holds 128 or more;
# a wave keeps 64 page numbers at a time, 1024 keys of pages of 16.
PATHS = {
    # more than 64 partial sums of a row, and the most there are, 64 of the prefix and 64 of the own keys
    "72 ranges": dict(nq=[1], kv_len=[9000], groups=[0, 1], prefix=[9000], hq=8, hkv=4, page=16),
    "128 ranges": dict(nq=[1], kv_len=[8192], groups=[0, 1], prefix=[16384], hq=8, hkv=4, page=16),
    # between 17 and 64 of them, some of them without keys
    "20 ranges": dict(nq=[2, 1], kv_len=[1500, 300], groups=[0, 2], prefix=[1900], hq=6, hkv=6, page=64),
    # long queries: a block of 128 rows walks 69 pages
    "a prompt on 69 pages": dict(nq=[40], kv_len=[1100], groups=[0], prefix=[], hq=140, hkv=140, page=16),
    "a prompt on a prefix of 67 pages": dict(nq=[40], kv_len=[50], groups=[0, 1], prefix=[1060], hq=140, hkv=140, page=16),
    # 36 rows of a sequence, 5 blocks of 128 from the 16 of its group (ranges of the prefix); from 3 groups
    "drafted tokens on one prefix, ranges": dict(nq=[9] * 16, kv_len=[20 + i for i in range(16)], groups=[0, 16], prefix=[700], hq=32,
                                                 hkv=8, page=16),
    "drafted tokens on 3 prefixes, ranges": dict(nq=[9] * 15 + [0], kv_len=[9 + i for i in range(16)], groups=[0, 7, 8, 16],
                                                 prefix=[500, 900, 411], hq=64, hkv=16, page=32),
    # one range of 69 pages, by 1 and by 20 rows a kv head; of a prefix too
    "a token on 69 pages": dict(nq=[1, 1], kv_len=[1100, 1030], groups=[0], prefix=[], hq=128, hkv=128, page=16),
    "20 heads on 69 pages": dict(nq=[1, 1], kv_len=[1100, 1030], groups=[0], prefix=[], hq=2560, hkv=128, page=16),
    "tokens on 4 prefixes of 69 pages": dict(nq=[1] * 5, kv_len=[3, 90, 1, 0, 17], groups=[0, 1, 2, 3, 5],
                                             prefix=[1100, 1040, 30, 1090], hq=128, hkv=128, page=16),
}


@pytest.mark.parametrize("name,dim,kv", [(name, dim, kv) for name in PATHS for dim in (64, 128) for kv in ("bf16", "e4m3")
                                         if "ranges" in name or (dim == 128) == (kv == "bf16")])
def test_attention_long_paths(name, dim, kv):
    note("attention, long paths", name, dim, kv)
    Case(len(name), dim=dim, kv=kv, **PATHS[name]).check()


@pytest.mark.parametrize("t_", [1, 40])
def test_w4_large_entries(t_):
    """A group whose entries sum to less than 2^120 (143 of them, the largest code, stay below 2^128); beside it a token
    with entries that may overflow spoils its own row only."""
    t = torch()
    note("w4, large entries", t_)
    rng = np.random.default_rng(t_)
    out, inn = 256, 384
    codes, scale, zero, view = w4_case(rng, out, inn)
    x = vals(bits(rng.uniform(0.5, 0.99, size=(t_ + 1, inn)) * 2.0 ** 113 * np.where(rng.random((t_ + 1, 1)) < 0.5, 1, rng.choice([-1, 1], (t_ + 1, inn)))))
    assert np.abs(x).reshape(t_ + 1, -1, 128).sum(-1).max() < 2.0 ** 120
    x[t_] *= 2.0 ** 5
    y = t.empty((t_ + 1, out), dtype=t.bfloat16, device="cuda")
    trs.dc_apply_w4(view, dev_bf16(x), y)
    want, tol = w4_reference(codes, scale, zero, x)
    assert (np.abs(vals(host_bits(y)) - want) <= tol)[:t_].all()
