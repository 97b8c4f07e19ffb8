"""Argument checks of the operators that close a decode step, on the CPU: device entry points are called only with
arguments that the host refuses (or nothing to do), with made-up addresses, so no kernel is ever launched."""
import ctypes

import pytest

import tenant_rank_serving_amd as trs
from tenant_rank_serving_amd import _lib

E = trs


@pytest.fixture(scope="module")
def L():
    return trs.lib()


def make(struct, defaults, kw):
    return struct(*({**defaults, **kw}[n] for n, _ in struct._fields_))


# ----------------------------------------------------------- verification
def batch(**kw):
    return make(_lib.dc_verify_batch, dict(seqs=3, q_start=0x1000, tokens=0x1100, accept=0x1200, pick=0x1300, temperature=0x1400), kw)


def verify(L, b=None, dtype=0, vocab=1000, target=0x100000, ts=1000, draft=0x200000, ds=1000, n=9, out=0x10000, count=0x10100,
           prob=0x10200, ws=0x400000, nws=1 << 20):
    return L.dc_verify_drafts(ctypes.byref(b if b is not None else batch()), dtype, vocab, target, ts, draft, ds, n, out, count,
                              prob, ws, nws, None)


def test_verify_with_nothing_to_do(L):
    empty = batch(seqs=0, q_start=None, tokens=None, accept=None, pick=None, temperature=None)
    assert verify(L, empty) == E.DC_OK and verify(L, empty, draft=None, ds=0, prob=None, count=None) == E.DC_OK
    assert verify(L, empty, dtype=1, n=0) == E.DC_OK


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), E.DC_ERR_INVALID_ARG), (dict(dtype=2), E.DC_ERR_INVALID_ARG), (dict(vocab=0), E.DC_ERR_SHAPE),
    (dict(vocab=-5), E.DC_ERR_SHAPE), (dict(target=None), E.DC_ERR_INVALID_ARG), (dict(ts=999), E.DC_ERR_SHAPE),
    (dict(ds=999), E.DC_ERR_SHAPE), (dict(target=0x100001), E.DC_ERR_ALIGN), (dict(dtype=1, target=0x100002), E.DC_ERR_ALIGN),
    (dict(draft=0x200001), E.DC_ERR_ALIGN), (dict(out=None), E.DC_ERR_INVALID_ARG), (dict(out=0x10002), E.DC_ERR_ALIGN),
    (dict(count=None), E.DC_ERR_INVALID_ARG), (dict(count=0x10101), E.DC_ERR_ALIGN), (dict(prob=0x10202), E.DC_ERR_ALIGN),
    (dict(ws=None), E.DC_ERR_INVALID_ARG), (dict(ws=0x400080), E.DC_ERR_ALIGN), (dict(nws=255), E.DC_ERR_BUFFER),
    (dict(b=batch(seqs=-1)), E.DC_ERR_INVALID_ARG), (dict(b=batch(q_start=None)), E.DC_ERR_INVALID_ARG),
    (dict(b=batch(tokens=None)), E.DC_ERR_INVALID_ARG), (dict(b=batch(accept=None)), E.DC_ERR_INVALID_ARG),
    (dict(b=batch(pick=None)), E.DC_ERR_INVALID_ARG), (dict(b=batch(pick=0x1302)), E.DC_ERR_ALIGN),
    (dict(b=batch(temperature=0x1401)), E.DC_ERR_ALIGN),
    (dict(vocab=(1 << 30) + 1, ts=1 << 31, ds=1 << 31), E.DC_ERR_UNSUPPORTED), (dict(n=1 << 24), E.DC_ERR_UNSUPPORTED),
    (dict(n=1 << 20, ts=1 << 27), E.DC_ERR_UNSUPPORTED), (dict(b=batch(seqs=1 << 24)), E.DC_ERR_UNSUPPORTED),
    # outputs that lie in one another, in what is read, in the workspace
    (dict(out=0x10100 - 32), E.DC_ERR_INVALID_ARG), (dict(prob=0x10000), E.DC_ERR_INVALID_ARG), (dict(out=0x1100), E.DC_ERR_INVALID_ARG),
    (dict(out=0x100000 + 2 * 9000 - 4), E.DC_ERR_INVALID_ARG), (dict(prob=0x200000), E.DC_ERR_INVALID_ARG),
    (dict(count=0x1308), E.DC_ERR_INVALID_ARG), (dict(out=0x400000), E.DC_ERR_INVALID_ARG), (dict(ws=0x100000), E.DC_ERR_INVALID_ARG),
    (dict(ws=0x200000 + 0x4600), E.DC_ERR_INVALID_ARG),
])
def test_verify_refusals(L, kw, want):
    assert verify(L, **kw) == want


def test_verify_most_sequences(L):
    """Launches have fewer than 2^32 threads: up to 4 per 32 logits of a sequence's row, 1024 at least."""
    size = L.dc_verify_workspace_bytes
    assert size(10, 9, (1 << 22) - 1) > 0 and size(10, 9, 1 << 22) == 0
    assert size(100003, 9, (1 << 22) // 13) > 0 and size(100003, 9, (1 << 22) // 13 + 1) == 0
    assert verify(L, batch(seqs=1 << 22)) == E.DC_ERR_UNSUPPORTED


def test_verify_workspace(L):
    size = L.dc_verify_workspace_bytes
    assert size(1000, 9, 3) % 256 == 0 and size(1000, 9, 3) >= 9 * 2 * 16 + 3 * 20
    assert [size(0, 1, 1), size(10, -1, 1), size(10, 1, -1), size((1 << 30) + 1, 1, 1), size(10, 1 << 24, 1)] == [0] * 5
    assert size(10, 0, 0) >= 256 and size(100003, 576, 64) > size(100003, 575, 64)
    need = size(1000, 9, 3)
    assert verify(L, nws=need - 1) == E.DC_ERR_BUFFER


def test_verify_workspace_of_a_larger_call_serves_a_smaller(L):
    """The size falls with none of its arguments, pieces of either length among them; calls are looked at up to the check
    behind the workspace's (an output in the logits)."""
    size = L.dc_verify_workspace_bytes
    for vocab in (1, 50, 2034, 2035, 8178, 8179, 32000, 100003, 128256, 1 << 22, 1 << 30):
        for seqs in (0, 1, 64, 3000):
            if seqs * (vocab // 8192 + 2) >= 1 << 22:
                continue
            all_n = sorted({n for n in [*range(0, 700), 1023, 1024, 4000, 65536] if 2 * n * (vocab // 8192 + 2) < 1 << 24})
            sizes = [size(vocab, n, seqs) for n in all_n]
            assert sizes == sorted(sizes) and sizes[0] > 0, (vocab, seqs)
    for n in (1, 2, 31, 32, 33, 40, 127, 128, 129, 255, 256, 257, 511, 512, 513, 2000):
        for seqs in (1, n):
            sizes = [size(v, n, seqs) for v in range(1, 140000, 97)]
            assert sizes == sorted(sizes), (n, seqs)
    for n in (1, 127, 128, 600):
        sizes = [size(32000, n, s) for s in range(0, 2000)]
        assert sizes == sorted(sizes), n
    for vocab, most in ((32000, 128), (32000, 200), (100003, 40), (128256, 32), (2, 600)):
        for n in range(1, most + 1):
            assert verify(L, batch(seqs=1), vocab=vocab, ts=vocab, ds=vocab, target=1 << 40, draft=1 << 41, out=1 << 40,
                          n=n, ws=1 << 42, nws=size(vocab, most, 1)) == E.DC_ERR_INVALID_ARG, (vocab, most, n)


# ------------------------------------------------------------ page tables
def table(**kw):
    return make(_lib.dc_kv_table, dict(seqs=4, width=10, page=16, num_pages=100, pages=0x1000, kv_len=0x2000, refs=0x3000), kw)


def resize(L, t=None, new=0x4000, copies=0x5000, status=0x6000):
    return L.dc_kv_resize(ctypes.byref(t if t is not None else table()), new, copies, status, None)


def fork(L, t=None, src=0x4000, dst=0x5000, n=0, status=0x6000):
    return L.dc_kv_fork(ctypes.byref(t if t is not None else table()), src, dst, n, status, None)


TABLES = [
    (dict(seqs=-1), E.DC_ERR_INVALID_ARG), (dict(width=-1), E.DC_ERR_INVALID_ARG), (dict(page=8), E.DC_ERR_SHAPE),
    (dict(page=24), E.DC_ERR_SHAPE), (dict(page=2048), E.DC_ERR_SHAPE), (dict(num_pages=0), E.DC_ERR_SHAPE),
    (dict(width=1 << 27), E.DC_ERR_SHAPE), (dict(pages=None), E.DC_ERR_INVALID_ARG), (dict(kv_len=None), E.DC_ERR_INVALID_ARG),
    (dict(refs=None), E.DC_ERR_INVALID_ARG), (dict(refs=0x3008), E.DC_ERR_ALIGN), (dict(pages=0x1002), E.DC_ERR_ALIGN),
    (dict(kv_len=0x2001), E.DC_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,want", TABLES)
def test_table_refusals(L, kw, want):
    assert resize(L, table(**kw)) == want and fork(L, table(**kw), n=1) == want


def test_tables_with_nothing_to_do(L):
    assert resize(L, table(seqs=0, pages=None, kv_len=None), None, None) == E.DC_OK
    assert fork(L) == E.DC_OK and fork(L, src=None, dst=None) == E.DC_OK


@pytest.mark.parametrize("kw,want", [
    (dict(new=None), E.DC_ERR_INVALID_ARG), (dict(copies=None), E.DC_ERR_INVALID_ARG), (dict(status=None), E.DC_ERR_INVALID_ARG),
    (dict(new=0x4001), E.DC_ERR_ALIGN), (dict(copies=0x5002), E.DC_ERR_ALIGN), (dict(status=0x6001), E.DC_ERR_ALIGN),
    (dict(t=table(seqs=16385)), E.DC_ERR_UNSUPPORTED), (dict(t=table(seqs=16384, width=65536)), E.DC_ERR_UNSUPPORTED),
    (dict(copies=0x3000 + 396), E.DC_ERR_INVALID_ARG), (dict(status=0x1000 + 156), E.DC_ERR_INVALID_ARG),
    (dict(new=0x1000), E.DC_ERR_INVALID_ARG), (dict(new=0x2004), E.DC_ERR_INVALID_ARG), (dict(copies=0x4000), E.DC_ERR_INVALID_ARG),
    (dict(t=table(kv_len=0x1000)), E.DC_ERR_INVALID_ARG),
])
def test_resize_refusals(L, kw, want):
    assert resize(L, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), E.DC_ERR_INVALID_ARG), (dict(n=1, src=None), E.DC_ERR_INVALID_ARG), (dict(n=1, dst=None), E.DC_ERR_INVALID_ARG),
    (dict(n=1, src=0x4001), E.DC_ERR_ALIGN), (dict(n=1, dst=0x5002), E.DC_ERR_ALIGN), (dict(n=1 << 24), E.DC_ERR_UNSUPPORTED),
    (dict(n=1, src=0x2000), E.DC_ERR_INVALID_ARG), (dict(n=4, dst=0x3000 - 8), E.DC_ERR_INVALID_ARG),
    (dict(n=1, status=0x4000), E.DC_ERR_INVALID_ARG),
    (dict(n=16385), E.DC_ERR_UNSUPPORTED),
])
def test_fork_refusals(L, kw, want):
    assert fork(L, **kw) == want


# ------------------------------------------------------------------ pages
def cache(**kw):
    return make(_lib.dc_kv_cache, dict(dtype=0, heads=4, dim=128, page=16, num_pages=10, page_stride=4 * 16 * 128,
                                       head_stride=16 * 128, slot_stride=128, k=0x10000, v=0x4000000, k_scale=None, v_scale=None), kw)


def layers(*kws):
    return (_lib.dc_kv_cache * len(kws))(*[cache(**kw) for kw in kws])


def copy(L, ls=None, n_layers=None, copies=0x1000, n=0):
    ls = ls if ls is not None else layers({}, dict(k=0x8000000, v=0x9000000))
    return L.dc_kv_copy(ls, len(ls) if n_layers is None else n_layers, copies, n, None)


def compact(L, ls=None, n_layers=None, source=0x1000, seqs=2, width=8, start=0x2000, keep=0x3000, n=0, to=0x4000):
    ls = ls if ls is not None else layers({}, dict(k=0x8000000, v=0x9000000))
    return L.dc_kv_compact(ls, len(ls) if n_layers is None else n_layers, source, seqs, width, start, keep, n, to, None)


def test_pages_with_nothing_to_do(L):
    assert copy(L) == E.DC_OK and copy(L, copies=None) == E.DC_OK
    assert compact(L) == E.DC_OK and compact(L, n=5, seqs=0) == E.DC_OK and compact(L, n=5, width=0) == E.DC_OK
    assert copy(L, layers(*[{}] * 128)) == E.DC_OK


LAYERS = [
    (layers(dict(dtype=3)), E.DC_ERR_INVALID_ARG), (layers(dict(dim=96)), E.DC_ERR_SHAPE), (layers({}, dict(v=None)), E.DC_ERR_INVALID_ARG),
    (layers({}, dict(k=0x8)), E.DC_ERR_ALIGN), (layers({}, dict(num_pages=11)), E.DC_ERR_SHAPE),
    (layers({}, dict(page_stride=5 * 16 * 128)), E.DC_ERR_SHAPE), (layers({}, dict(dtype=1)), E.DC_ERR_SHAPE),
    (layers({}, dict(dim=64)), E.DC_ERR_SHAPE), (layers({}, dict(heads=2)), E.DC_ERR_SHAPE),
    (layers({}, dict(head_stride=128, slot_stride=512)), E.DC_ERR_SHAPE),
    (layers({}, dict(page=32, num_pages=10, page_stride=4 * 32 * 128, head_stride=32 * 128)), E.DC_ERR_SHAPE),
    (layers(*[{}] * 129), E.DC_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("ls,want", LAYERS)
def test_layer_refusals(L, ls, want):
    assert copy(L, ls, n=1) == want and compact(L, ls, n=1) == want


def test_page_refusals(L):
    assert copy(L, n_layers=0) == E.DC_ERR_INVALID_ARG and copy(L, n=-1) == E.DC_ERR_INVALID_ARG
    assert copy(L, n=1, copies=None) == E.DC_ERR_INVALID_ARG and copy(L, n=1, copies=0x1002) == E.DC_ERR_ALIGN
    assert copy(L, n=1 << 23) == E.DC_ERR_UNSUPPORTED
    for kw, want in ((dict(n=-1), E.DC_ERR_INVALID_ARG), (dict(seqs=-1), E.DC_ERR_INVALID_ARG), (dict(width=-1), E.DC_ERR_INVALID_ARG),
                     (dict(n=1, source=None), E.DC_ERR_INVALID_ARG), (dict(n=1, start=None), E.DC_ERR_INVALID_ARG),
                     (dict(n=1, keep=None), E.DC_ERR_INVALID_ARG), (dict(n=1, source=0x1002), E.DC_ERR_ALIGN),
                     (dict(n=1, to=0x4001), E.DC_ERR_ALIGN), (dict(n=1, to=0x1000), E.DC_ERR_INVALID_ARG),
                     (dict(n=1, width=1 << 28), E.DC_ERR_SHAPE), (dict(n=INT_MAX, seqs=1), E.DC_ERR_UNSUPPORTED),
                     (dict(n=1, seqs=1 << 23), E.DC_ERR_UNSUPPORTED)):
        assert compact(L, **kw) == want, kw


def test_what_the_pages_hold_is_not_what_a_call_reads(L):
    """Pairs, tables and positions that lie in a page of any layer's keys or values; room between pages is none of them."""
    size = 10 * 4 * 16 * 128 * 2
    pools = (0x10000, 0x4000000, 0x8000000, 0x9000000)          # keys and values of the two layers
    for p in pools:
        for at in (p - 4, p, p + size - 8):
            assert copy(L, n=1, copies=at) == E.DC_ERR_INVALID_ARG, hex(at)
            for kw in (dict(source=at), dict(to=at), dict(start=at), dict(keep=at, n=2)):
                assert compact(L, **{**dict(n=1), **kw}) == E.DC_ERR_INVALID_ARG, (hex(at), kw)
                if "to" not in kw:
                    assert compact(L, **{**dict(n=1, to=None), **kw}) == E.DC_ERR_INVALID_ARG, (hex(at), kw)
    # pages 128 elements further apart than they are long, the last one's end
    wide = layers(dict(page_stride=4 * 16 * 128 + 128))
    page = 4 * 16 * 128 * 2
    for at, want in ((0x10000 + page - 4, E.DC_ERR_INVALID_ARG), (0x10000 + page + 252, E.DC_ERR_INVALID_ARG),
                     (0x10000 + 9 * (page + 256) + page - 4, E.DC_ERR_INVALID_ARG)):
        assert copy(L, wide, n=1, copies=at) == want, hex(at)


INT_MAX = 2 ** 31 - 1


# ---------------------------------------------------------- 4-bit floats
def view(rows=256, cols=384, base=0x1000000):
    return _lib.dc_mx4_view(rows, cols, base)


def apply(L, w=None, x=0x2000000, y=0x3000000, t=0):
    return L.dc_apply_mx4(ctypes.byref(w if w is not None else view()), x, y, t, None)


def applyq(L, w=None, x=None, y=0x3000000):
    return L.dc_apply_mx4q(ctypes.byref(w if w is not None else view()), ctypes.byref(x if x is not None else view(5, 384, 0x2000000)), y,
                           None)


def pack(L, rows=256, cols=384, x=0x2000000, stride=384, dst=0x1000000, n=1 << 30, flag=0x100):
    return L.dc_mx4_pack_device(rows, cols, x, stride, dst, n, flag, None)


def dequant(L, w=None, x=0x2000000, stride=384):
    return L.dc_mx4_dequant(ctypes.byref(w if w is not None else view()), x, stride, None)


def test_mx4_bytes():
    assert trs.dc_mx4_bytes(256, 384) == 256 * 384 // 2 + 16 * 256 and trs.dc_mx4_bytes(1, 640) == 16 * 640 // 2 + 2 * 256
    assert [trs.dc_mx4_bytes(*s) for s in ((0, 128), (-1, 128), (5, 0), (5, 64), (5, 130), (5, -128))] == [0] * 6
    assert trs.dc_mx4_bytes(1 << 20, 1 << 20) == (1 << 39) + (1 << 35)


def test_mx4_bytes_at_the_ends_of_its_arguments(L):
    """Rows and columns up to the last ones that 31 bits hold, in exact arithmetic."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    for rows in (1, 16, 17, 1 << 30, INT_MAX - 15, INT_MAX - 14, INT_MAX):
        for cols in (128, 512, 640, 1 << 30, 2 ** 31 - 640, 2 ** 31 - 512, 2 ** 31 - 384, 2 ** 31 - 128):
            want = up(rows, 16) * 16 * cols // 2 + up(rows, 16) * up(cols, 512) * 256
            assert trs.dc_mx4_bytes(rows, cols) == want, (rows, cols)
    # a buffer one byte short of such a row is refused
    cols = 2 ** 31 - 128
    assert pack(L, rows=1, cols=cols, stride=cols, x=1 << 40, dst=1 << 44, n=trs.dc_mx4_bytes(1, cols) - 1) == E.DC_ERR_BUFFER


def test_mx4_forms_that_the_gpu_tests_name():
    """Every form of the products has its calls in the GPU tests, whatever the rules become: whole and ragged columns, tokens
    that end inside a tile."""
    import test_gpu_step as g
    for forms, calls, of, tokens in ((g.MX4_FORMS, g.MX4_CALLS, g.mx4_form, lambda f: 16 if f in g.MX4_FORMS[:4] else int(f.split()[3])),
                                     (g.MX4Q_FORMS, g.MX4Q_CALLS, g.mx4q_form, lambda f: int(f.split()[2]))):
        assert list(calls) == forms
        for form, cases in calls.items():
            for t, out, inn in cases:
                assert of(t, out, inn) == form, (form, t, out, inn, of(t, out, inn))
                assert t % tokens(form) and out % 128 == 0
            assert {inn // 128 % 4 for _, _, inn in cases} == {0, 1, 2, 3}, form


def test_mx4_refusals(L):
    assert apply(L) == E.DC_OK and pack(L, rows=0) == E.DC_OK and pack(L, rows=0, n=0, flag=None) == E.DC_OK
    size = trs.dc_mx4_bytes(256, 384)
    for w, want in ((view(0), E.DC_ERR_SHAPE), (view(256, 100), E.DC_ERR_SHAPE), (view(base=None), E.DC_ERR_INVALID_ARG),
                    (view(base=0x1000008), E.DC_ERR_ALIGN), (view(1 << 20, 1 << 12), E.DC_ERR_UNSUPPORTED)):
        assert apply(L, w, t=1) == want and applyq(L, w) == want and dequant(L, w, stride=w.cols) == want
        assert w.rows == 256 or applyq(L, x=w) == want
    for kw, want in ((dict(t=-1), E.DC_ERR_INVALID_ARG), (dict(x=None), E.DC_ERR_INVALID_ARG), (dict(y=None), E.DC_ERR_INVALID_ARG),
                     (dict(w=view(130)), E.DC_ERR_SHAPE), (dict(x=0x2000008), E.DC_ERR_ALIGN), (dict(y=0x3000004), E.DC_ERR_ALIGN),
                     (dict(t=1048561), E.DC_ERR_UNSUPPORTED), (dict(t=2, y=0x2000000 + 384 * 4 - 16), E.DC_ERR_INVALID_ARG),
                     (dict(t=1, y=0x1000000 + size - 16), E.DC_ERR_INVALID_ARG), (dict(t=1, y=0x1000000 - 496), E.DC_ERR_INVALID_ARG)):
        assert apply(L, **kw) == want, kw
    for kw, want in ((dict(y=None), E.DC_ERR_INVALID_ARG), (dict(y=0x3000008), E.DC_ERR_ALIGN), (dict(w=view(130)), E.DC_ERR_SHAPE),
                     (dict(x=view(5, 512)), E.DC_ERR_SHAPE), (dict(x=view(1048561, 128), w=view(128, 128)), E.DC_ERR_UNSUPPORTED),
                     (dict(y=0x1000000), E.DC_ERR_INVALID_ARG), (dict(y=0x2000000 + 16), E.DC_ERR_INVALID_ARG)):
        assert applyq(L, **kw) == want, kw
    for kw, want in ((dict(rows=-1), E.DC_ERR_INVALID_ARG), (dict(cols=100), E.DC_ERR_SHAPE), (dict(stride=376), E.DC_ERR_SHAPE),
                     (dict(stride=388), E.DC_ERR_ALIGN), (dict(x=None), E.DC_ERR_INVALID_ARG), (dict(x=0x2000002), E.DC_ERR_ALIGN),
                     (dict(dst=None), E.DC_ERR_INVALID_ARG), (dict(dst=0x1000004), E.DC_ERR_ALIGN), (dict(flag=0x102), E.DC_ERR_ALIGN),
                     (dict(n=size - 1), E.DC_ERR_BUFFER), (dict(dst=0x2000000), E.DC_ERR_INVALID_ARG),
                     (dict(dst=0x2000000 - size + 16), E.DC_ERR_INVALID_ARG), (dict(flag=0x2000000), E.DC_ERR_INVALID_ARG),
                     (dict(flag=0x1000010), E.DC_ERR_INVALID_ARG), (dict(rows=1 << 30, x=1 << 50, n=1 << 60), E.DC_ERR_UNSUPPORTED)):
        assert pack(L, **kw) == want, kw
    for kw, want in ((dict(x=None), E.DC_ERR_INVALID_ARG), (dict(stride=376), E.DC_ERR_SHAPE), (dict(stride=388), E.DC_ERR_ALIGN),
                     (dict(x=0x1000000 + size - 16), E.DC_ERR_INVALID_ARG)):
        assert dequant(L, **kw) == want, kw
