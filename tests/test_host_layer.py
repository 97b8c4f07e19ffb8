"""Argument checks of the decoder-layer operators, on the CPU: device entry points are called only with arguments that
the host refuses (or nothing to do), with made-up addresses, so no kernel is ever launched."""
import ctypes
import os

import pytest

import tenant_rank_serving_amd as trs
from tenant_rank_serving_amd import _lib

E = trs


def cache(**kw):
    f = dict(dtype=0, heads=4, dim=128, page=16, num_pages=10, page_stride=4 * 16 * 128, head_stride=16 * 128,
             slot_stride=128, k=0x10000, v=0x4000000, k_scale=None, v_scale=None)
    f.update(kw)
    return _lib.dc_kv_cache(*(f[n] for n, _ in _lib.dc_kv_cache._fields_))


def rope(**kw):
    f = dict(inv_freq=0x100, rot=128, interleaved=0)
    f.update(kw)
    return _lib.dc_rope(*(f[n] for n, _ in _lib.dc_rope._fields_))


def batch(**kw):
    f = dict(seqs=2, max_q=1, max_kv=100, seq_pages=8, q_start=0x1000, kv_len=0x1100, pages=0x1200, groups=1, max_group_q=2,
             max_prefix=50, prefix_pages_per_group=4, group_start=0x1300, prefix_len=0x1400, prefix_pages=0x1500)
    f.update(kw)
    return _lib.dc_attn_batch(*(f[n] for n, _ in _lib.dc_attn_batch._fields_))


@pytest.fixture(scope="module")
def L():
    return trs.lib()


def append(L, c=None, r=rope(), q=0x8000000, qs=1024, k=0x8100000, ks=512, v=0x8200000, vs=512, pos=0x200, slots=0x300,
           qo=0x8300000, qos=1024, hq=8, n=0):
    return L.dc_kv_append(ctypes.byref(c if c is not None else cache()), ctypes.byref(r) if r is not None else None, q, qs, k, ks,
                          v, vs, pos, slots, qo, qos, hq, n, None)


def test_append_with_nothing_to_do(L):
    assert append(L) == E.DC_OK
    assert append(L, r=None, pos=None) == E.DC_OK
    assert append(L, hq=0, q=None, qo=None, qs=0, qos=0) == E.DC_OK
    # pages of [slots][heads], keys and values in one allocation, e4m3 with scales
    assert append(L, cache(slot_stride=4 * 128, head_stride=128, page_stride=2 * 4 * 16 * 128)) == E.DC_OK
    assert append(L, cache(dtype=1, k_scale=0x40, v_scale=0x80)) == E.DC_OK


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), E.DC_ERR_INVALID_ARG), (dict(k=None), E.DC_ERR_INVALID_ARG), (dict(v=None), E.DC_ERR_INVALID_ARG),
    (dict(heads=0), E.DC_ERR_SHAPE), (dict(dim=96), E.DC_ERR_SHAPE), (dict(dim=256), E.DC_ERR_SHAPE),
    (dict(page=8), E.DC_ERR_SHAPE), (dict(page=48), E.DC_ERR_SHAPE), (dict(page=2048), E.DC_ERR_SHAPE),
    (dict(num_pages=0), E.DC_ERR_SHAPE), (dict(k=0x10008), E.DC_ERR_ALIGN), (dict(v=0x4000001), E.DC_ERR_ALIGN),
    (dict(slot_stride=64), E.DC_ERR_SHAPE), (dict(slot_stride=132), E.DC_ERR_ALIGN), (dict(page_stride=8196), E.DC_ERR_ALIGN),
    (dict(head_stride=1024), E.DC_ERR_SHAPE),                    # heads that overlap
    (dict(page_stride=4 * 16 * 128 - 128), E.DC_ERR_SHAPE),      # pages that overlap
    (dict(k_scale=0x40), E.DC_ERR_INVALID_ARG),                  # scales of a bf16 cache
    (dict(dtype=1, k_scale=0x42), E.DC_ERR_ALIGN),
    (dict(dtype=1, slot_stride=136), E.DC_ERR_ALIGN),            # 16 bytes are 16 elements there
    (dict(slot_stride=1 << 26, head_stride=128, page_stride=1 << 30), E.DC_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 30, page_stride=1 << 40), E.DC_ERR_UNSUPPORTED),
])
def test_cache_refusals(L, kw, want):
    assert append(L, cache(**kw)) == want
    b = batch()
    assert L.dc_attention(ctypes.byref(cache(**kw)), ctypes.byref(b), 0x8000000, 1024, 8, 0.1, 0x8300000, 1024, 2, 0x100, 1 << 30,
                          None) == want
    assert L.dc_attention_workspace_bytes(ctypes.byref(cache(**kw)), ctypes.byref(b), 8, 2) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), E.DC_ERR_INVALID_ARG), (dict(hq=-1), E.DC_ERR_INVALID_ARG),
    (dict(k=None), E.DC_ERR_INVALID_ARG), (dict(v=None), E.DC_ERR_INVALID_ARG), (dict(q=None), E.DC_ERR_INVALID_ARG),
    (dict(qo=None), E.DC_ERR_INVALID_ARG), (dict(slots=None), E.DC_ERR_INVALID_ARG), (dict(pos=None), E.DC_ERR_INVALID_ARG),
    (dict(r=rope(inv_freq=None)), E.DC_ERR_INVALID_ARG), (dict(r=rope(rot=8)), E.DC_ERR_SHAPE),
    (dict(r=rope(rot=144)), E.DC_ERR_SHAPE), (dict(r=rope(rot=40)), E.DC_ERR_SHAPE), (dict(r=rope(inv_freq=0x104)), E.DC_ERR_ALIGN),
    (dict(slots=0x304), E.DC_ERR_ALIGN), (dict(pos=0x202), E.DC_ERR_ALIGN), (dict(q=0x8000008), E.DC_ERR_ALIGN),
    (dict(qs=1028), E.DC_ERR_ALIGN), (dict(qs=1016), E.DC_ERR_SHAPE), (dict(ks=0), E.DC_ERR_SHAPE), (dict(vs=504), E.DC_ERR_SHAPE),
    # overlaps: q_out one row behind q, over k, over v; q in place with another stride
    (dict(n=4, qo=0x8000000 + 2048), E.DC_ERR_INVALID_ARG), (dict(n=4, qo=0x8100000, qos=1024), E.DC_ERR_INVALID_ARG),
    (dict(n=1, qo=0x8200000 - 512), E.DC_ERR_INVALID_ARG), (dict(n=2, qo=0x8000000, qos=2048), E.DC_ERR_INVALID_ARG),
    # a fused matrix whose k columns the written q rows reach into
    (dict(n=4, q=0x8000000, qs=2048, k=0x8000000 + 1024, ks=2048, qo=0x8000000, qos=2048), E.DC_ERR_INVALID_ARG),
])
def test_append_refusals(L, kw, want):
    assert append(L, **kw) == want


def attend(L, c=None, b=None, q=0x8000000, qs=1024, hq=8, scale=0.1, y=0x8300000, ys=1024, n=0, ws=0x100, nws=1 << 30):
    return L.dc_attention(ctypes.byref(c or cache()), ctypes.byref(b or batch()), q, qs, hq, scale, y, ys, n, ws, nws, None)


def test_attention_with_nothing_to_do(L):
    assert attend(L) == E.DC_OK
    assert attend(L, b=batch(seqs=0, q_start=None, kv_len=None, pages=None), n=5) == E.DC_OK
    assert attend(L, b=batch(max_q=0), n=5) == E.DC_OK
    assert attend(L, b=batch(groups=0, group_start=None, prefix_len=None, prefix_pages=None)) == E.DC_OK


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), E.DC_ERR_INVALID_ARG), (dict(hq=0), E.DC_ERR_INVALID_ARG), (dict(hq=6), E.DC_ERR_SHAPE),
    (dict(scale=0.0), E.DC_ERR_INVALID_ARG), (dict(scale=-1.0), E.DC_ERR_INVALID_ARG), (dict(scale=float("nan")), E.DC_ERR_INVALID_ARG),
    (dict(scale=float("inf")), E.DC_ERR_INVALID_ARG), (dict(q=None), E.DC_ERR_INVALID_ARG), (dict(y=None), E.DC_ERR_INVALID_ARG),
    (dict(ws=None), E.DC_ERR_INVALID_ARG), (dict(ws=0x180), E.DC_ERR_ALIGN), (dict(q=0x8000004), E.DC_ERR_ALIGN),
    (dict(ys=1020), E.DC_ERR_SHAPE), (dict(ys=1026), E.DC_ERR_ALIGN), (dict(n=2, y=0x8000000), E.DC_ERR_INVALID_ARG),
    (dict(n=2, nws=256), E.DC_ERR_BUFFER), (dict(n=1 << 30), E.DC_ERR_UNSUPPORTED),
    (dict(b=batch(seqs=-1)), E.DC_ERR_INVALID_ARG), (dict(b=batch(groups=-1)), E.DC_ERR_INVALID_ARG),
    (dict(b=batch(max_kv=-1)), E.DC_ERR_INVALID_ARG), (dict(b=batch(q_start=None)), E.DC_ERR_INVALID_ARG),
    (dict(b=batch(kv_len=None)), E.DC_ERR_INVALID_ARG), (dict(b=batch(pages=None)), E.DC_ERR_INVALID_ARG),
    (dict(b=batch(group_start=None)), E.DC_ERR_INVALID_ARG), (dict(b=batch(prefix_pages=None)), E.DC_ERR_INVALID_ARG),
    (dict(b=batch(prefix_len=0x1402)), E.DC_ERR_ALIGN), (dict(b=batch(max_kv=129)), E.DC_ERR_SHAPE),
    (dict(b=batch(max_prefix=65)), E.DC_ERR_SHAPE), (dict(b=batch(max_q=1 << 28)), E.DC_ERR_UNSUPPORTED),
])
def test_attention_refusals(L, kw, want):
    assert attend(L, **kw) == want


def test_attention_workspace(L):
    c = cache()
    size = lambda n=2, **kw: L.dc_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(batch(**kw)), 8, n)  # noqa: E731
    assert size() > 256 and size() % 256 == 0
    assert size(groups=0, max_kv=64) == 256            # one range of keys: no partial sums
    assert size(n=2, max_kv=100) < size(n=4, max_kv=100)
    need = size()
    assert attend(L, n=2, nws=need - 1) == E.DC_ERR_BUFFER


def w4(L, out=256, inn=384, base=0x1000000, x=0x2000000, y=0x3000000, t=0):
    return L.dc_apply_w4(ctypes.byref(_lib.dc_w4_view(out, inn, base)), x, y, t, None)


def test_w4_refusals(L):
    assert trs.dc_w4_bytes(256, 384) == 256 * 384 // 2 + 4 * 256 * 3
    assert [trs.dc_w4_bytes(*s) for s in ((0, 128), (128, 64), (130, 128), (-128, 128))] == [0] * 4
    assert w4(L) == E.DC_OK
    assert w4(L, t=-1) == E.DC_ERR_INVALID_ARG and w4(L, out=200) == E.DC_ERR_SHAPE
    assert w4(L, base=None) == E.DC_ERR_INVALID_ARG and w4(L, x=None) == E.DC_ERR_INVALID_ARG
    assert w4(L, x=0x2000004) == E.DC_ERR_ALIGN and w4(L, base=0x1000008) == E.DC_ERR_ALIGN
    assert w4(L, t=4, y=0x2000010) == E.DC_ERR_INVALID_ARG
    assert w4(L, out=1 << 16, inn=1 << 15) == E.DC_ERR_UNSUPPORTED
    pack = lambda out=256, inn=384, w=0x1000000, d=0x2000000, n=1 << 30, f=0x100: L.dc_w4_pack_device(out, inn, w, d, n, f, None)  # noqa: E731
    assert pack(out=100) == E.DC_ERR_SHAPE and pack(w=None) == E.DC_ERR_INVALID_ARG and pack(f=None) == E.DC_ERR_INVALID_ARG
    assert pack(d=0x2000008) == E.DC_ERR_ALIGN and pack(n=trs.dc_w4_bytes(256, 384) - 1) == E.DC_ERR_BUFFER


def test_binding_checks_types_and_shapes():
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    c = trs.KvCache(k, k.clone())
    assert (c.c.page_stride, c.c.head_stride, c.c.slot_stride) == (2048, 1024, 64)
    one = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2)   # [pages][slots][heads][dim]
    c = trs.KvCache(one, one.clone(memory_format=torch.preserve_format))
    assert (c.c.page_stride, c.c.head_stride, c.c.slot_stride) == (2048, 64, 128)
    with pytest.raises(ValueError):
        trs.KvCache(k, k.float())
    with pytest.raises(ValueError):
        trs.KvCache(k.float(), k.float())
    with pytest.raises(ValueError):
        trs.KvCache(k, one)
    with pytest.raises(ValueError):
        trs.KvCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), torch.ones(3), torch.ones(2))
    with pytest.raises(ValueError):
        trs.Rope(torch.ones(8))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        trs.AttnBatch(i32(2), i32(2), i32(2, 4), 1, 4)
    with pytest.raises(ValueError):
        trs.AttnBatch(i32(3), i32(2).long(), i32(2, 4), 1, 4)
    with pytest.raises(ValueError):
        trs.AttnBatch(i32(3), i32(2), i32(2, 4), 1, 4, group_start=i32(1), prefix_len=i32(1), prefix_pages=i32(1, 1))
    with pytest.raises(ValueError):
        trs.W4View(128, 128, torch.zeros(100, dtype=torch.uint8))
    with pytest.raises(ValueError):   # rows that are too short for the heads
        trs.dc_kv_append(c, None, torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16), None,
                         torch.zeros(4, dtype=torch.int64), None, None)


def test_more_blocks_than_a_launch_takes(L):
    """Refused before anything is launched (2^32 threads are one too many)."""
    assert append(L, n=1 << 24, q=1 << 40, k=1 << 42, v=1 << 43, qo=1 << 44) == E.DC_ERR_UNSUPPORTED
    few = dict(groups=0, group_start=None, prefix_len=None, prefix_pages=None)
    # a block for every sequence and kv head
    assert attend(L, b=batch(seqs=1 << 22, max_q=1, max_kv=16, **few), n=2, nws=1 << 60) == E.DC_ERR_UNSUPPORTED
    # the rows whose partial sums are joined, four a block
    b = batch(seqs=2, max_q=1, max_kv=100, max_group_q=1)
    q, y = 1 << 40, 1 << 50
    assert attend(L, b=b, q=q, y=y, n=1 << 23, nws=1 << 60) == E.DC_ERR_UNSUPPORTED


def test_strides_beyond_any_memory(L):
    """Rows that would lie 2^48 bytes away: refused, and no product of 64 bits overflows on the way (the rows of q and
    q_out then count as apart)."""
    far = 1 << 40
    assert append(L, n=1 << 23, qs=far, qos=far, q=1 << 40, qo=(1 << 40) + 4096, k=1 << 50, v=1 << 51) == E.DC_ERR_SHAPE
    assert append(L, n=1 << 23, ks=far, q=1 << 40, qo=1 << 41, k=1 << 50, v=1 << 51) == E.DC_ERR_SHAPE
    assert attend(L, n=1 << 23, qs=far, ys=far, q=1 << 40, y=(1 << 40) + 4096, nws=1 << 60) == E.DC_ERR_SHAPE


@pytest.mark.parametrize("scale", [1e-45, 1e-38, 2.4e38, 3.4e38])
def test_attention_scales_out_of_range(L, scale):
    assert attend(L, n=2, scale=scale) == E.DC_ERR_INVALID_ARG


def test_attention_scales_at_the_ends(L):
    assert attend(L, scale=1.2e-38) == E.DC_OK and attend(L, scale=2.3e38) == E.DC_OK


def test_append_of_more_heads_than_a_launch_takes(L):
    assert append(L, hq=1 << 21, qs=1 << 28, qos=1 << 28, n=1, q=1 << 40, qo=1 << 42, k=1 << 43, v=1 << 44) == E.DC_ERR_UNSUPPORTED


def test_empty_calls_through_the_binding(monkeypatch):
    """Tensors without rows have no address; a call with them is a no-op, its other arguments are checked all the same."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(_lib, "_current", lambda device, stream: 0)
    bf16 = dict(dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 16, 64, **bf16)
    c = trs.KvCache(k, k.clone())
    rope = trs.Rope(torch.ones(32, dtype=torch.float64))
    row = torch.zeros(1, 128, **bf16)
    none, pos, slots = row[:0], torch.zeros(0, dtype=torch.int32), torch.zeros(0, dtype=torch.int64)
    for empty in (none, torch.zeros(0, 128, **bf16)):
        assert empty.data_ptr() == 0
        trs.dc_kv_append(c, empty, empty, empty, pos, slots, rope, empty)
        trs.dc_kv_append(c, None, empty, empty, None, slots, None, None)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    for b in (trs.AttnBatch(i32(1), i32(0), i32(1, 4), 1, 64), trs.AttnBatch(i32(3), i32(2), i32(2, 4), 0, 64)):
        trs.dc_attention(c, none, b, 0.125, none, ws)
    view = trs.W4View(128, 128, torch.zeros(trs.dc_w4_bytes(128, 128), dtype=torch.uint8))
    trs.dc_apply_w4(view, none, none)
    with pytest.raises(trs.DcError):
        trs.dc_attention(c, none, trs.AttnBatch(i32(3), i32(2), i32(2, 4), 0, 65), 0.125, none, ws)
    with pytest.raises(ValueError):
        trs.dc_kv_append(c, none[:, :64], none, none, pos, slots, rope, none)


def test_assembly_names_the_registers_it_writes():
    """Inline assembly that writes m0, exec or vcc by name says so, or the compiler may keep something there."""
    import re
    src = os.path.join(os.path.dirname(trs.__file__), "csrc")
    found = 0
    for name in sorted(os.listdir(src)):
        text = open(os.path.join(src, name)).read()
        for m in re.finditer(r"asm volatile\((.*?)\);", text, re.S):
            for reg in ("m0", "exec", "vcc"):
                if re.search(r"[a-z_0-9]+ %s," % reg, m.group(1)):
                    found += 1
                    assert '"%s"' % reg in m.group(1).rsplit(":", 1)[1], (name, m.group(1))
    assert found


# The made-up cache: keys 0x10000 .. 0x38000, values 0x4000000 .. 0x4028000, pages of 0x4000 bytes.
@pytest.mark.parametrize("kw", [
    dict(qo=0x10000), dict(qo=0x38000 - 16), dict(qo=0x4000000), dict(qo=0x10000 - 2048, n=2), dict(qo=0x4020000, qos=1 << 12),
    dict(q=0x20000, qs=1024, qo=0x20000),   # in place, in the cache
])
def test_append_refuses_queries_in_the_cache(L, kw):
    assert append(L, **dict(dict(n=1), **kw)) == E.DC_ERR_INVALID_ARG


def test_append_queries_in_a_gap_of_the_cache(L):
    """Pages with room between them: what fits there is not in the cache (of two tokens, it reaches the next page)."""
    gap = cache(page_stride=2 * 4 * 16 * 128)   # 0x8000 bytes, the upper half is free
    assert append(L, gap, n=3, qo=0x10000 + 0x4000 + 0x3000 + 2048) == E.DC_ERR_INVALID_ARG
    assert append(L, gap, n=1, qo=0x10000 + 0x4000 - 16) == E.DC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(y=0x10000), dict(y=0x4028000 - 16), dict(y=0x4000000 - 2048),        # the output in the cache
    dict(ws=0x10000), dict(ws=0x4020000), dict(ws=0x10000 - 0x2000),          # the workspace in the cache,
    dict(ws=0x8000000), dict(ws=0x8000000 - 0x2000),                          # in the queries,
    dict(ws=0x8300000), dict(y=0x101000, ws=0x100000),                        # in the output
])
def test_attention_refuses_overlaps(L, kw):
    assert 0x2000 < L.dc_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch()), 8, 2) < 0x10000
    assert attend(L, **dict(dict(n=2, ws=0x100000, nws=0x10000), **kw)) == E.DC_ERR_INVALID_ARG


def test_w4_refuses_overlaps(L):
    size = trs.dc_w4_bytes(256, 384)
    assert w4(L, t=1, y=0x1000000) == E.DC_ERR_INVALID_ARG and w4(L, t=1, y=0x1000000 + size - 16) == E.DC_ERR_INVALID_ARG
    pack = lambda w, d: L.dc_w4_pack_device(256, 384, w, d, 1 << 30, 0x100, None)  # noqa: E731
    assert pack(0x1000000, 0x1000000) == E.DC_ERR_INVALID_ARG
    assert pack(0x1000000, 0x1000000 + 2 * 256 * 384 - 16) == E.DC_ERR_INVALID_ARG
    assert pack(0x1000000, 0x1000000 - size + 16) == E.DC_ERR_INVALID_ARG


def test_append_elements_of_a_token_at_the_limit(L):
    """65535 * 4096 elements of q, k and v a token, 16 a unit and 256 units a block along the launch's y."""
    most = 65535 * 4096 // 128 - 2 * 4          # query heads beside 4 + 4 kv heads
    far = dict(q=1 << 40, qs=1 << 29, qo=1 << 42, qos=1 << 29, k=1 << 43, v=1 << 44)
    assert append(L, hq=most, **far) == E.DC_OK
    assert append(L, hq=most + 1, **far) == E.DC_ERR_UNSUPPORTED


def test_attention_reads_a_shared_prefix_for_its_group(L):
    """9 drafted tokens of 64 sequences on one long prefix: 36 rows of 128 in a block of their own, so the blocks of the
    prefix are filled from the group (with partial sums); filled blocks walk it themselves."""
    c = cache(heads=8, page_stride=8 * 16 * 128, num_pages=20000)
    def size(seqs, nq, own, groups, prefix):
        b = batch(seqs=seqs, max_q=nq, max_kv=own, seq_pages=1 << 12, groups=groups, max_group_q=seqs // groups * nq, max_prefix=prefix,
                  prefix_pages_per_group=1 << 12)
        return L.dc_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 32, seqs * nq)
    assert size(64, 9, 300, 1, 16384) > 256 and size(64, 9, 300, 8, 16384) > 256 and size(64, 9, 300, 1, 2048) > 256
    assert size(400000, 9, 16, 100, 16384) == 256   # more rows than a join takes: not refused
    assert size(64, 9, 300, 1, 512) == 256 and size(64, 32, 300, 1, 16384) == 256 and size(8, 1024, 1024, 8, 2048) == 256
