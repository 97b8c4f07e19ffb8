"""The oracle of the operators that close a decode step against hand-worked values and plain identities (CPU)."""
import numpy as np

from oracle import step


def test_distribution():
    assert np.allclose(step.distribution([0.0, np.log(3.0)], 1.0), [0.25, 0.75])
    assert np.allclose(step.distribution([0.0, np.log(9.0)], 2.0), [0.25, 0.75])
    assert step.distribution([1.0, 5.0, 5.0], 0.0).tolist() == [0, 1, 0] == step.distribution([1.0, 5.0, 5.0], -1.0).tolist()
    assert step.distribution([-np.inf, 0.0], 1.0).tolist() == [0, 1]
    assert step.distribution([-np.inf, -np.inf], 1.0) is None and step.distribution([np.nan, 0.0], 0.0) is None
    assert step.distribution([np.inf, 0.0], 1.0) is None


def test_verify_by_hand():
    l3 = np.log(3.0)
    target = np.array([[0.0, l3], [l3, 0.0], [0.0, l3]])          # p = (1/4, 3/4), (3/4, 1/4), (1/4, 3/4)
    draft = np.array([[l3, 0.0], [l3, 0.0], [0.0, 0.0]])          # q = (3/4, 1/4), twice
    # the first draft 0: stands while u 3/4 < 1/4; else only token 1 is left of p - q
    for u, want in ((0.3, [0, 0]), (0.34, [1, -1])):
        out, prob, count, _ = step.verify(target[:2], draft[:2], [0, 2], [9, 0], [u, 0.5], [0.7], None)
        assert out == want and count == [2 if u == 0.3 else 1]
        assert np.allclose(prob, [0.25, 0.75] if u == 0.3 else [0.75, 0.0])
    # looked-up drafts: 1 stands while u < 3/4, then 1 while u < 1/4, then p itself
    out, prob, count, _ = step.verify(target, None, [0, 3], [0, 1, 1], [0.74, 0.2, 0.9], [0.25], None)
    assert out == [1, 1, 1] and count == [3] and np.allclose(prob, [0.75, 0.25, 0.75])
    out, _, count, _ = step.verify(target, None, [0, 3], [0, 1, 1], [0.74, 0.26, 0.9], [0.99], None)
    assert out == [1, 0, -1] and count == [2]                     # 1 fell: only 0 is left
    # rows of no sequence, a sequence without rows, a token outside the vocabulary, a row without a distribution
    out, _, count, _ = step.verify(target, None, [1, 1, 3], [0, 0, 7], [0, 0.0, 0], [0.5, 0.5], [1.0, 1.0])
    assert out == [None, 0, -1] and count == [0, 1]
    out, _, count, _ = step.verify(np.array([[np.nan, 0.0]]), None, [0, 1], [0], [0], [0], None)
    assert out == [-1] and count == [0]


def test_verified_tokens_follow_the_target():
    """Whatever the draft's distribution, the first token of a step is distributed as p."""
    rng = np.random.default_rng(0)
    t, d = rng.normal(size=(2, 2, 5))
    p, q = step.distribution(t[0], 1.0), step.distribution(d[0], 1.0)
    hits, n = np.zeros(5), 20000
    for _ in range(n):
        tok = rng.choice(5, p=q)
        hits[step.verify(t, d, [0, 2], [0, tok], rng.random(2), rng.random(1), None)[0][0]] += 1
    assert np.abs(hits / n - p).max() < 5 * np.sqrt(0.25 / n)     # five standard deviations


def test_tables_by_hand():
    t = step.Tables([[4, 1, -1], [-1, -1, -1], [-1, -1, -1]], [20, 0, 0], [0, 1, 0, 3, 1, 0], 16)
    t.fork([0, 0], [1, 2])
    assert t.pages[1] == [4, 1, -1] and t.kv_len == [20, 20, 20] and t.refs == [0, 3, 0, 3, 3, 0]
    copies = t.resize([20, 21, 40])
    # rows 1 and 2 get fresh last pages, lowest numbers first; row 2 another one
    assert copies == [[-1, -1], [1, 0], [1, 2]] and t.pages == [[4, 1, -1], [4, 0, -1], [4, 2, 5]]
    assert t.refs == [1, 1, 1, 3, 3, 1] and not t.full and not t.bad
    assert t.resize([33, 0, 40]) == [[-1, -1]] * 3                # row 1 gives 0 back, row 0 takes it
    assert t.pages[0] == [4, 1, 0] and t.pages[1] == [-1] * 3 and t.refs == [1, 1, 1, 3, 2, 1]
    t.resize([33, 1, 20])                                         # 5 is given back and taken
    assert t.pages[1] == [5, -1, -1] and t.kv_len == [33, 1, 20]
    t.resize([33, 17, 33])
    assert t.full and t.kv_len == [33, 1, 20] and t.pages[2] == [4, 2, -1]
    t.fork([0], [2])
    assert t.bad


def test_compact_by_hand():
    pool = np.arange(4 * 16).reshape(4, 1, 16, 1)
    new = step.compact(pool, [[2, 0]], [0, 3], [1, 5, 17], [[2, 0]], 16)
    assert new[2, 0, :4, 0].tolist() == [33, 37, 1, 35] and np.array_equal(new[[0, 1, 3]], pool[[0, 1, 3]])


def test_mx4():
    x = np.zeros((1, 128))
    x[0, :8] = [6.0, 0.25, 0.75, -2.5, 3.5, 5.0, 0.26, -0.1]      # exponent 2: the scale is 1, ties go to the even code
    x[0, 32] = 7.9                                                # 6 is the largest
    x[0, 64:66] = [2.0 ** -126, 2.0 ** -128]
    x[0, 96] = np.inf
    codes, scale = step.mx4_quantize(x)
    assert scale.tolist() == [[127, 127, 0, 255]]
    v = step.mx4_matrix(codes, scale)
    assert v[0, :8].tolist() == [6.0, 0.0, 1.0, -2.0, 4.0, 4.0, 0.5, 0.0] and np.signbit(v[0, 7]) and v[0, 32] == 6.0
    assert v[0, 64:66].tolist() == [2.0 ** -126, 2.0 ** -128] and np.isnan(v[0, 96:]).all()
    assert np.array_equal(step.mx4_matrix(np.arange(16)[None].repeat(2, 0).reshape(1, 32), [[127]])[0, 8:16],
                          -step.POINTS)
    every = np.tile(np.arange(16), 8)[None]
    assert np.array_equal(step.mx4_quantize(step.mx4_matrix(every, [[100] * 4]))[0], every)


def test_mx4_format_positions():
    codes, scale = np.zeros((17, 640), np.int64), np.zeros((17, 20), np.int64)
    codes[16, 128 * 3 + 32 * 2 + 7] = 9          # tile 1, group 3, block 2, row 0, element 7: the high half of byte 3
    scale[3, 4 * 4 + 1] = 77                     # tile 0, columns 512 + 32 ..: group 4 = byte 0 of the second word
    buf = step.mx4_pack(codes, scale)
    assert buf[((5 + 3) * 64 + 2 * 16 + 0) * 16 + 3] == 9 << 4 and np.count_nonzero(buf[:2 * 5 * 1024]) == 1
    sc = buf[2 * 5 * 1024:]
    assert sc.size == 2 * 2 * 256 and sc[((0 * 2 + 1) * 64 + 1 * 16 + 3) * 4] == 77 and np.count_nonzero(sc) == 1
