"""The operators that close a decode step in fp64 numpy and plain Python: verification of drafted tokens, page tables,
pages, microscaled 4-bit floating point.  Written from the formulas; used by tests only."""
import numpy as np


# ----------------------------------------------------------- verification
def distribution(logits, t):
    """softmax(logits / t) in fp64, all on the first largest one for t <= 0; None if there is no distribution."""
    x = np.asarray(logits, np.float64)
    if np.isnan(x).any() or not np.isfinite(x.max()):
        return None
    if not t > 0:
        p = np.zeros(x.size)
        p[int(x.argmax())] = 1.0
        return p
    with np.errstate(under="ignore"):
        e = np.exp((x - x.max()) / np.float64(min(np.float64(t), 3.4028234663852886e38)))
    return e / e.sum()


def pick(w, r):
    """(lowest i with w_i > 0 whose running sum passes r sum(w), how far r sum(w) is from the nearest border)."""
    c = np.cumsum(w)
    aim = np.float64(r) * c[-1]
    at = np.nonzero((c > aim) & (w > 0))[0]
    i = int(at[0]) if at.size else int(np.nonzero(w > 0)[0][-1])
    return i, float(np.abs(c[:-1] - aim).min() / c[-1]) if c.size > 1 else 1.0


def verify(target, draft, q_start, tokens, accept, picks, temperature):
    """out, prob [N] (None where a row is of no sequence), count [B], and the smallest relative distance of any
    comparison to its border."""
    n, vocab = np.shape(target)
    out, prob, count, margin = [None] * n, [None] * n, [], 1.0
    for b in range(len(q_start) - 1):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        for r in range(lo, hi):
            out[r], prob[r] = -1, 0.0
        t = 1.0 if temperature is None else float(temperature[b])
        got = 0
        for r in range(lo, hi):
            p = distribution(target[r], t)
            if p is None:
                break
            w = p
            if r + 1 < hi:
                d = int(tokens[r + 1])
                inside = 0 <= d < vocab
                if draft is None or not t > 0:
                    q = np.zeros(vocab)
                    if inside:
                        q[d] = 1.0
                else:
                    q = distribution(draft[r], t)
                if inside and q is not None:
                    left, right = float(accept[r]) * q[d], p[d]
                    if t > 0 and max(left, right) > 0:
                        margin = min(margin, abs(left - right) / max(left, right))
                    if left < right if t > 0 else p[d] == 1.0:   # greedy: no random number
                        out[r], prob[r] = d, p[d]
                        got += 1
                        continue
                if q is not None:
                    rest = np.maximum(p - q, 0.0)
                    w = rest if rest.sum() > 0 else p
            i, m = pick(w, picks[b])
            if t > 0:
                margin = min(margin, m)
            out[r], prob[r] = i, p[i]
            got += 1
            break
        count.append(got)
    return out, prob, count, margin


# ------------------------------------------------------------ page tables
class Tables:
    """Page tables as lists; rows keep -1 behind their pages."""

    def __init__(self, pages, kv_len, refs, page):
        self.pages, self.kv_len, self.refs = [list(r) for r in pages], list(kv_len), list(refs)
        self.page, self.full, self.bad = page, False, False

    def _count(self, n):
        return -(-n // self.page)

    def _ok(self, p):
        return 0 <= p < len(self.refs)

    def resize(self, new_len):
        most = len(self.pages[0]) * self.page
        copies = [[-1, -1] for _ in self.pages]
        fine = [0 <= a <= most and 0 <= b <= most for a, b in zip(self.kv_len, new_len)]
        self.bad |= not all(fine)
        for b, row in enumerate(self.pages):
            if fine[b]:
                for i in range(self._count(new_len[b]), self._count(self.kv_len[b])):
                    if self._ok(row[i]):
                        self.refs[row[i]] -= 1
                    else:
                        self.bad = True
                    row[i] = -1
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        plan, short = [], False
        for b, row in enumerate(self.pages):
            need, swap = 0, False
            if fine[b] and new_len[b] > self.kv_len[b]:
                need = self._count(new_len[b]) - self._count(self.kv_len[b])
                if self.kv_len[b] % self.page:
                    p = row[self.kv_len[b] // self.page]
                    if self._ok(p):
                        swap = self.refs[p] > 1
                    else:
                        self.bad = True
            plan.append((need + swap, swap))
        fallen = []
        for b, row in enumerate(self.pages):
            need, swap = plan[b]
            if not fine[b]:
                continue
            short |= need > len(free)
            if need and short:
                self.full = True
                continue
            if swap:
                i = self.kv_len[b] // self.page
                copies[b] = [row[i], free[0]]
                fallen.append(row[i])
                row[i] = free.pop(0)
                self.refs[row[i]] = 1
            for i in range(self._count(self.kv_len[b]), self._count(new_len[b])):
                row[i] = free.pop(0)
                self.refs[row[i]] = 1
            self.kv_len[b] = new_len[b]
        for p in fallen:
            self.refs[p] -= 1
        return copies

    def fork(self, src, dst):
        for i, (s, d) in enumerate(zip(src, dst)):
            n = len(self.pages)
            if s in dst or d in dst[:i] or not (0 <= s < n and 0 <= d < n and s != d and self.kv_len[d] == 0
                    and 0 <= self.kv_len[s] <= len(self.pages[0]) * self.page):
                self.bad = True
                continue
            for i in range(self._count(self.kv_len[s])):
                self.pages[d][i] = self.pages[s][i]
                if self._ok(self.pages[s][i]):
                    self.refs[self.pages[s][i]] += 1
                else:
                    self.bad = True
            self.kv_len[d] = self.kv_len[s]


def compact(pool, source, start, keep, target, page):
    """pool [pages][heads][page][dim] after kept tokens moved; sources are read before anything is written."""
    new = pool.copy()
    width = len(source[0])
    for b in range(len(start) - 1):
        for j in range(start[b], start[b + 1]):
            a, z = int(keep[j]), j - start[b]
            if not (0 <= a < width * page and 0 <= z < width * page):
                continue
            p, q = source[b][a // page], target[b][z // page]
            if 0 <= p < pool.shape[0] and 0 <= q < pool.shape[0]:
                new[q, :, z % page] = pool[p, :, a % page]
    return new


# ---------------------------------------------------------- 4-bit floats
POINTS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize(x):
    """(codes [rows][cols], scale bytes [rows][cols/32]) of fp64 values."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    s = np.maximum(np.frexp(np.maximum(top, 2.0 ** -140))[1] - 1 - 2 + 127, 0)
    v = np.abs(b) / 2.0 ** (s[..., None] - 127.0)
    d = np.abs(v[..., None] - POINTS)
    best = d.min(-1, keepdims=True)
    tie = d == best                      # of two equally near points the even code
    c = np.where(tie.sum(-1) == 2, np.where(tie.argmax(-1) % 2 == 0, tie.argmax(-1), tie.argmax(-1) + 1), d.argmin(-1))
    c = c | (np.signbit(b) << 3)
    return np.where(bad[..., None], 0, c).reshape(x.shape), np.where(bad, 255, s)


def mx4_matrix(codes, scale):
    """The fp64 values (NaN throughout a block of scale 255)."""
    c = np.asarray(codes)
    v = POINTS[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(np.asarray(scale) == 255, np.nan, 2.0 ** (np.asarray(scale, np.float64) - 127.0))
    return (v.reshape(c.shape[0], -1, 32) * s[..., None]).reshape(c.shape)


def mx4_pack(codes, scale):
    """Bytes of the format."""
    rows, cols = codes.shape
    tiles = -(-rows // 16)
    out = np.zeros((tiles, cols // 128, 4, 16, 16), np.uint8)
    sc = np.zeros((tiles, -(-cols // 512), 4, 16, 4), np.uint8)
    for r in range(rows):
        q = np.asarray(codes[r], np.uint8).reshape(cols // 128, 4, 16, 2)
        out[r // 16, :, :, r % 16] = q[..., 0] | q[..., 1] << 4
        for g in range(cols // 128):
            sc[r // 16, g // 4, :, r % 16, g % 4] = scale[r][4 * g:4 * g + 4]
    return np.concatenate([out.reshape(-1), sc.reshape(-1)])
