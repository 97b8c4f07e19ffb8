"""Cases of the operators that close a decode step: verifying drafted tokens against the target's probabilities, the
page tables of a cache (forking, growing, freeing, copying, compacting), and products with a backbone in microscaled
4-bit floating point (MXFP4).

own = False computes the plain forms (elementary torch operations); own = True calls the library.
Lengths are a function of the case (not of the seed), so that work(case) can count them.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one chat without drafts: sampling its next token from a 7B model's 32000 logits, where latency counts
        dict(name="verify_1x1_32000", op="verify", b=1, nq=1, vocab=32000, dtype="bf16", draft="none", masked=False),
        # 20 chats check 4 drafted tokens each against the draft model's logits, grammars mask part of some vocabularies
        dict(name="verify_20x5_32000", op="verify", b=20, nq=5, vocab=32000, dtype="bf16", draft="logits", masked=True),
        # 64 chats x 8 drafts, a large vocabulary of an odd size, fp32 logits, drafts looked up in the prompt (no logits)
        dict(name="verify_64x9_100003_f32", op="verify", b=64, nq=9, vocab=100003, dtype="f32", draft="token", masked=False),
        # best-of-n sampling: 48 branches of 16 chats are dropped, and opened and grown again
        dict(name="tables_16x3_branches", op="tables", b=16, fork=3, have=2100, grow=70, page=16, spare=4096),
        # the pages that 4 opened branches write to next, all layers of a 7B model
        dict(name="copy_4_32x32", op="copy", n=4, layers=32, heads=32, d=128, page=16, kv="bf16"),
        # 96 long chats branch: their last pages, grouped-query layers, e4m3 cache
        dict(name="copy_96_32x8_e4m3", op="copy", n=96, layers=32, heads=8, d=128, page=64, kv="e4m3"),
        # one chat keeps half of about a thousand tokens
        dict(name="compact_1x1000_32x8", op="compact", b=1, have=1000, keep=0.5, layers=32, heads=8, d=128, page=16,
             kv="bf16"),
        # 8 chats keep a third of some 4000 tokens each
        dict(name="compact_8x4000_32x8", op="compact", b=8, have=4000, keep=0.33, layers=32, heads=8, d=128, page=64,
             kv="bf16"),
        # one token through the q, k, v or o matrix of a 7B layer
        dict(name="mx4_1_4096x4096", op="mx4", t=1, out=4096, inn=4096),
        # the logits of 64 chats: a 7B model's head
        dict(name="mx4_64_32000x4096", op="mx4", t=64, out=32000, inn=4096),
        # the prompts of 8 x 2048 tokens through the gate or up matrix of a 7B layer, activations in 4 bits too
        dict(name="mx4q_16384_11008x4096", op="mx4q", t=16384, out=11008, inn=4096),
        # laying out the down matrix of a grouped-query model, and what it then stands for
        dict(name="mx4_pack_4096x14336", op="pack", out=4096, inn=14336),
    ]


SHAPES = [(4096, 4096), (1024, 4096), (5120, 5120), (11008, 4096), (4096, 11008), (14336, 4096), (4096, 14336),
          (13824, 5120), (5120, 13824), (32000, 4096), (512, 1152), (1920, 640)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "tables", "copy", "compact", "mx4", "mx4q", "pack"])
    if op == "verify":
        nq = rng.choice([1, 2, 3, 5, 6, 9])
        vocab = rng.choice([32000, _log(rng, 50, 131072)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        draft = "none" if nq == 1 else rng.choice(["logits", "logits", "token"])
        row = vocab * (2 if dtype == "bf16" else 4) * (2 if draft == "logits" else 1)
        return dict(op=op, b=max(1, min(_log(rng, 1, 64), 230000000 // (row * nq))), nq=nq, vocab=vocab, dtype=dtype,
                    draft=draft, masked=rng.random() < 0.4)
    if op == "tables":
        have = _log(rng, 20, 8000)
        return dict(op=op, b=_log(rng, 1, 64), fork=rng.choice([1, 2, 3, 4]), have=have, grow=_log(rng, 1, 300),
                    page=rng.choice([16, 32, 64, 128]), spare=_log(rng, 2000, 60000))
    layers = _log(rng, 1, 40)
    heads = rng.choice([8, 8, 32, 4, 40, 2])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    row = layers * heads * d * (2 if kv == "bf16" else 1) * 2   # bytes of a token
    if op == "copy":
        n = _log(rng, 1, 128)
        return dict(op=op, n=max(1, min(n, 400000000 // (row * page))), layers=layers, heads=heads, d=d, page=page, kv=kv)
    if op == "compact":
        b, keep = _log(rng, 1, 16), rng.choice([0.1, 0.33, 0.5, 0.9])
        have = min(_log(rng, 1, 8192), max(1, int(1000000000 / (row * b * max(keep, 0.33)))))
        return dict(op=op, b=b, have=have, keep=keep, layers=layers, heads=heads, d=d, page=page, kv=kv)
    out, inn = rng.choice(SHAPES)
    if op == "pack":
        return dict(op=op, out=out, inn=inn)
    if op == "mx4":
        return dict(op=op, t=_log(rng, 1, 64), out=out, inn=inn)
    return dict(op=op, t=min(_log(rng, 1, 8192), 16384 * 11008 * 4096 // (out * inn)), out=out, inn=inn)


# ---------------------------------------------------------------- lengths
def _spread(i, lo, hi):
    """A length between lo and hi for item i."""
    return lo + (i * 40503 + 11 * i * i + 7) % 65521 % (hi - lo + 1)


def _pages(n, page):
    return (n + page - 1) // page


def _rows(c):
    """Rows of each sequence of a verification: its drafts and one more; the last sequence has the most."""
    return [c["nq"] if i == c["b"] - 1 else _spread(i, (c["nq"] + 1) // 2, c["nq"]) for i in range(c["b"])]


def _have(c):
    """Tokens of each sequence; the last one takes the bound itself."""
    return [c["have"] if i == c["b"] - 1 else _spread(i, (c["have"] + 1) // 2, c["have"]) for i in range(c["b"])]


def _kept(c):
    return [max(1, int(n * c["keep"])) for n in _have(c)]


def work(c):
    op = c["op"]
    if op == "verify":
        n, e = sum(_rows(c)), 2 if c["dtype"] == "bf16" else 4
        drafts = n - c["b"] if c["draft"] == "logits" else 0   # the last row of a sequence has no draft
        return {"bytes": (n + drafts) * c["vocab"] * e + 16 * n + 20 * c["b"], "flops": 6 * (n + drafts) * c["vocab"]}
    if op == "tables":
        # dropped branches: their entries and counts; opened: entries read and written, counts; grown: new entries
        have = sum(_pages(n, c["page"]) for n in _have(c)) * c["fork"]
        more = sum(_pages(n + c["grow"], c["page"]) - n // c["page"] for n in _have(c)) * c["fork"]
        return {"bytes": 12 * (have + more) + 16 * have + 8 * more + 4 * c["spare"] + 24 * c["b"] * c["fork"], "flops": 0}
    if op in ("copy", "compact"):
        row = c["layers"] * c["heads"] * c["d"] * (2 if c["kv"] == "bf16" else 1) * 2
        tokens = c["n"] * c["page"] if op == "copy" else sum(_kept(c))
        return {"bytes": 2 * tokens * row + 8 * (c["n"] if op == "copy" else tokens), "flops": 0}
    out, inn = c["out"], c["inn"]
    w = out * inn // 2 + out * inn // 32
    if op == "pack":
        return {"bytes": 2 * w + 4 * out * inn, "flops": 0}
    return {"bytes": w + 2 * c["t"] * (inn + out), "flops": 2 * c["t"] * out * inn}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(counts):
    return _i32([sum(counts[:i]) for i in range(len(counts) + 1)])


def prepare(c, seed):
    g = _gen(seed)
    return {"verify": _prepare_verify, "tables": _prepare_tables, "copy": _prepare_copy, "compact": _prepare_compact,
            "mx4": _prepare_product, "mx4q": _prepare_product, "pack": _prepare_pack}[c["op"]](c, g)


def _prepare_verify(c, g):
    rows, v, b = _rows(c), c["vocab"], c["b"]
    n = sum(rows)
    ty = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    # a few likely tokens above a broad floor, as a model's logits are
    target = torch.randn((n, v), generator=g, device=DEV) * 2.0
    target.scatter_add_(1, torch.randint(0, v, (n, 6), generator=g, device=DEV),
                        4.0 + 6.0 * torch.rand((n, 6), generator=g, device=DEV))
    draft = target + torch.randn((n, v), generator=g, device=DEV) * 0.7
    if c["masked"]:   # every third row allows part of the vocabulary only
        hit = torch.rand((n, v), generator=g, device=DEV) < 0.6
        hit[:, v // 2] = False
        hit &= (torch.arange(n, device=DEV) % 3 == 1)[:, None]
        target.masked_fill_(hit, -math.inf)
    target, draft = target.to(ty), draft.to(ty)
    temperature = torch.rand(b, generator=g, device=DEV) * 1.2 + 0.3
    temperature[::5] = 0.0 if b > 1 else 0.8    # greedy chats among the others
    q_start = _starts(rows)
    seq = torch.searchsorted(q_start, torch.arange(n, device=DEV, dtype=torch.int32), right=True) - 1
    # the drafted tokens: drawn from the draft model's distribution (looked-up ones: from something like it)
    t = torch.where(temperature > 0, temperature, 0.01)[seq][:, None]
    noise = -torch.log(-torch.log(torch.rand((n, v), generator=g, device=DEV).clamp_(1e-20, 1 - 1e-7)))
    drawn = (draft.float() / t + noise).argmax(1)
    tokens = torch.roll(drawn, 1).to(torch.int32)    # row j's draft is the input token of row j + 1
    s = dict(c=c, n=n, target=target, draft=draft if c["draft"] == "logits" else None, q_start=q_start, tokens=tokens,
             temperature=temperature, accept=torch.rand(n, generator=g, device=DEV),
             pick=torch.rand(b, generator=g, device=DEV), most=max(rows),
             out=torch.empty(n, dtype=torch.int32, device=DEV), count=torch.empty(b, dtype=torch.int32, device=DEV),
             prob=torch.empty(n, dtype=torch.float32, device=DEV))
    if own:   # the views and the workspace that a serving loop keeps
        import tenant_rank_serving_amd as trs
        s["batch"] = trs.VerifyBatch(q_start, tokens, s["accept"], s["pick"], temperature)
        s["ws"] = torch.empty(trs.dc_verify_workspace_bytes(v, n, b), dtype=torch.uint8, device=DEV)
    return s


def _prepare_tables(c, g):
    b, f, page = c["b"], c["fork"], c["page"]
    have = _have(c)
    width = _pages(c["have"] + c["grow"], page)
    used = sum(_pages(n, page) for n in have)
    num = used + c["spare"] + b * f * (2 + c["grow"] // page)
    perm = torch.randperm(num, generator=g, device=DEV).to(torch.int32).cpu()
    pages = torch.full((b * (1 + f), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(have):
        m = _pages(n, page)
        pages[i, :m] = perm[at:at + m]
        at += m
    refs = torch.zeros(num, dtype=torch.int32)
    refs[perm[:used].long()] = 1
    refs[perm[used:used + c["spare"] // 2].long()] = 2   # held by others
    lens = _i32(have + [0] * (b * f))
    src = torch.arange(b, dtype=torch.int32, device=DEV).repeat_interleave(f)
    dst = torch.arange(b, b * (1 + f), dtype=torch.int32, device=DEV)
    less, more = lens.clone(), lens.clone()
    more[b:] = lens[:b].repeat_interleave(f) + c["grow"]
    s = dict(c=c, pages=pages.to(DEV), lens=lens, refs=refs.to(DEV), src=src, dst=dst, less=less, more=more,
             copies=torch.full((b * (1 + f), 2), -1, dtype=torch.int32, device=DEV),
             none=torch.full((b * (1 + f), 2), -1, dtype=torch.int32, device=DEV),
             status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if own:
        import tenant_rank_serving_amd as trs
        s["table"] = trs.KvTable(s["pages"], lens, s["refs"], page)
    return s


def _pool(c, pages, g):
    """Keys and values of all layers: [layers][2][pages][heads][page][d], in use."""
    shape = (c["layers"], 2, pages, c["heads"], c["page"], c["d"])
    if c["kv"] == "bf16":
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    codes = torch.randint(0, 254, shape, generator=g, device=DEV, dtype=torch.uint8)
    return torch.where(codes >= 127, codes + 1, codes).view(torch.float8_e4m3fn)   # every code that is a number


def _layers(pool):
    import tenant_rank_serving_amd as trs
    return trs.KvLayers([trs.KvCache(x[0], x[1]) for x in pool.unbind(0)])


def _prepare_copy(c, g):
    pages = 2 * c["n"] + 8
    pool = _pool(c, pages, g)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    pairs = perm[:2 * c["n"]].view(-1, 2).contiguous()
    if c["n"] > 8:
        pairs[c["n"] // 3] = -1   # a chat that needs no copy
    s = dict(c=c, pool=pool, pairs=pairs)
    if own:
        s["layers"] = _layers(pool)
    return s


def _prepare_compact(c, g):
    have, kept, page = _have(c), _kept(c), c["page"]
    width = _pages(c["have"], page)
    a, b = sum(_pages(n, page) for n in have), sum(_pages(n, page) for n in kept)
    pool = _pool(c, a + b + 4, g)
    perm = torch.randperm(a + b + 4, generator=g, device=DEV).to(torch.int32).cpu()
    tables, at = [], 0
    for lens in (have, kept):
        t = torch.full((c["b"], width), -1, dtype=torch.int32)
        for i, n in enumerate(lens):
            m = _pages(n, page)
            t[i, :m] = perm[at:at + m]
            at += m
        tables.append(t.to(DEV))
    keep = torch.cat([torch.randperm(n, generator=g, device=DEV)[:m].sort().values for n, m in zip(have, kept)])
    s = dict(c=c, pool=pool, src=tables[0], dst=tables[1], keep=keep.to(torch.int32), start=_starts(kept))
    if own:
        s["layers"] = _layers(pool)
    return s


def _prepare_product(c, g):
    w = torch.randn((c["out"], c["inn"]), generator=g, device=DEV) * 0.02
    codes, scale = _quantized(w)
    x = torch.randn((c["t"], c["inn"]), generator=g, device=DEV)
    x[:, ::97] *= 8.0   # a few large channels, as activations have
    s = dict(c=c, w=_packed(codes, scale), x=x.to(torch.bfloat16),
             y=torch.empty((c["t"], c["out"]), dtype=torch.bfloat16, device=DEV))
    if own:
        import tenant_rank_serving_amd as trs
        s["view"] = trs.Mx4View(c["out"], c["inn"], s["w"])
        if c["op"] == "mx4q":   # room for the activations in 4 bits
            s["xq"] = trs.Mx4View(c["t"], c["inn"], torch.empty(trs.dc_mx4_bytes(c["t"], c["inn"]), dtype=torch.uint8,
                                                               device=DEV))
    return s


def _prepare_pack(c, g):
    w = torch.randn((c["out"], c["inn"]), generator=g, device=DEV) * 0.02
    w *= torch.exp(torch.randn((c["out"], 1), generator=g, device=DEV))
    w[:, 64:96] = 0.0   # blocks without a value
    s = dict(c=c, x=w.to(torch.bfloat16), out=torch.empty((c["out"], c["inn"]), dtype=torch.bfloat16, device=DEV))
    if own:
        import tenant_rank_serving_amd as trs
        s["view"] = trs.Mx4View(c["out"], c["inn"], torch.empty(trs.dc_mx4_bytes(c["out"], c["inn"]), dtype=torch.uint8,
                                                               device=DEV))
        s["flag"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# The MXFP4 format: blocks of 32 columns of a row; the block's scale is 2^(byte - 127) with the byte of its largest
# magnitude's exponent less 2 (never below 0), its codes e2m1 (sign, 2 exponent bits, 1 mantissa bit).  Codes as bytes
# [rows/16][cols/128][4][16][16]: piece (T, G, q, i) holds row 16T + i, columns 128G + 32q + e, code e in the low
# (even e) or high half of byte e/2; then scale bytes [rows/16][cols/512][4][16][4], byte j of (T, H, q, i) being that of
# columns 512H + 128j + 32q .. + 31.  Rows past the last and bytes past the last column are zero.
def _power(n):
    """2^n in fp32, exactly, for whole numbers -126 .. 127."""
    return ((n + 127) << 23).to(torch.int32).view(torch.float32)


def _quantized(x):
    """(codes [rows][cols] int32, scale bytes [rows][cols/32] int32) of finite fp32 values."""
    b = x.view(x.shape[0], -1, 32)
    e = ((b.abs().amax(-1).view(torch.int32) >> 23) - 2).clamp(min=0)
    v = b * _power(127 - e)[..., None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)                # round half to even
    mag = torch.where(q < 2, 2 * q, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.int32)
    sign = torch.signbit(v).to(torch.int32)
    return (mag | sign << 3).view(x.shape), e.to(torch.int32)


def _packed(codes, scale):
    rows, cols = codes.shape
    pad = -rows % 16
    codes = torch.nn.functional.pad(codes.to(torch.uint8), (0, 0, 0, pad))
    scale = torch.nn.functional.pad(scale.to(torch.uint8), (0, -(cols // 32) % 16, 0, pad))
    c = codes.view(-1, 16, cols // 128, 4, 16, 2).permute(0, 2, 3, 1, 4, 5)
    b = (c[..., 0] | c[..., 1] << 4).reshape(-1)
    s = scale.view(scale.shape[0] // 16, 16, -1, 4, 4).permute(0, 2, 4, 1, 3).reshape(-1)
    return torch.cat([b, s])


def _values(buf, rows, cols, ty=torch.float32):
    """What a buffer of the format stands for."""
    up, gc = (rows + 15) // 16 * 16, cols // 128
    nc = up * cols // 2
    b = buf[:nc].view(-1, gc, 4, 16, 16)
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).permute(0, 3, 1, 2, 4).reshape(up, cols)[:rows].to(torch.int32)
    s = buf[nc:].view(up // 16, -1, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(up, -1)[:rows, :cols // 32].to(torch.int32)
    mag = c & 7
    m = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2.0, 2.0 * mag - 8.0)).to(ty)
    m = torch.where((c & 8) > 0, -m, m).view(rows, -1, 32)
    m = torch.where((s == 0)[..., None], m / 2, m)                   # 2^-127 is subnormal
    return (m * _power(s.clamp(min=1) - 127)[..., None].to(ty)).view(rows, cols)


# ------------------------------------------------------------------- runs
def run(s):
    c = s["c"]
    if own:
        return _own(s, c)
    return {"verify": _plain_verify, "tables": _plain_tables, "copy": _plain_copy, "compact": _plain_compact,
            "mx4": _plain_product, "mx4q": _plain_product, "pack": _plain_pack}[c["op"]](s, c)


def _own(s, c):
    import tenant_rank_serving_amd as trs
    op = c["op"]
    if op == "verify":
        trs.dc_verify_drafts(s["batch"], s["target"], s["draft"], s["out"], s["count"], s["ws"], s["prob"])
        return [s["out"], s["count"], s["prob"]]
    if op == "tables":
        trs.dc_kv_resize(s["table"], s["less"], s["none"], s["status"])       # the branches of before go
        trs.dc_kv_fork(s["table"], s["src"], s["dst"], s["status"])           # and are opened again
        trs.dc_kv_resize(s["table"], s["more"], s["copies"], s["status"])     # with room for what they will write
        return [s["pages"], s["lens"], s["refs"], s["copies"], s["status"]]
    if op == "copy":
        trs.dc_kv_copy(s["layers"], s["pairs"])
        return s["pool"]
    if op == "compact":
        trs.dc_kv_compact(s["layers"], s["src"], s["start"], s["keep"], s["dst"])
        return s["pool"]
    if op == "pack":
        trs.dc_mx4_pack_device(s["x"], s["view"], s["flag"])
        trs.dc_mx4_dequant(s["view"], s["out"])
        return s["out"]
    if op == "mx4":
        trs.dc_apply_mx4(s["view"], s["x"], s["y"])
    else:
        trs.dc_mx4_pack_device(s["x"], s["xq"])
        trs.dc_apply_mx4q(s["view"], s["xq"], s["y"])
    return s["y"]


def _softmax(logits, t):
    """exp((l - max) / t) over its sum, in 64 bits (sampling looks for the place of a number among the sums)."""
    x = logits.double()
    x = ((x - x.amax(1, keepdim=True)) / t[:, None]).exp_()
    return x.div_(x.sum(1, keepdim=True))


def _plain_verify(s, c):
    n, v, b = s["n"], c["vocab"], c["b"]
    q_start, target = s["q_start"].long(), s["target"]
    row = torch.arange(n, device=target.device)
    seq = torch.searchsorted(q_start, row, right=True) - 1
    temp = s["temperature"][seq].double()
    greedy = temp <= 0
    t = torch.where(greedy, 1.0, temp)
    index = torch.arange(v, device=target.device)
    best = torch.where(target == target.amax(1, keepdim=True), index, v).amin(1)     # the lowest of equal ones
    p = _softmax(target, t)
    token = torch.roll(s["tokens"], -1).long()                                       # the draft that a row judges
    drafted = row < q_start[1:][seq] - 1
    pt = p.gather(1, token[:, None])[:, 0]
    if s["draft"] is None:
        q, qt = None, torch.ones_like(pt)
    else:
        q = _softmax(s["draft"], t)
        qt = q.gather(1, token[:, None])[:, 0]
    stands = torch.where(greedy, token == best, s["accept"].double() * qt < pt) & drafted
    j = torch.arange(s["most"], device=target.device)
    at = (q_start[:-1, None] + j).clamp(max=n - 1)
    inside = q_start[:-1, None] + j < q_start[1:, None]
    kept = torch.cumprod(torch.where(inside, stands[at], False).to(torch.int32), 1).sum(1)
    last = q_start[:-1] + kept                                                       # the row that gives a new token
    w = p[last]
    fell = drafted[last]                                                             # its draft did not stand
    if q is None:
        less = torch.nn.functional.one_hot(token[last], v)
    else:
        less = q[last]
    rest = (w - less).clamp_(min=0.0)
    rest = torch.where((rest.sum(1) > 0)[:, None], rest, w)
    w = torch.where(fell[:, None], rest, w)
    cum = w.cumsum(1)
    new = torch.where(cum > s["pick"].double()[:, None] * cum[:, -1:], index, v).amin(1)
    new = torch.where(new < v, new, torch.where(w > 0, index, -1).amax(1))
    new = torch.where(greedy[last], best[last], new)
    place = row - q_start[seq]
    s["out"].copy_(torch.where(place < kept[seq], token, torch.where(place == kept[seq], new[seq], -1)))
    s["count"].copy_(kept + 1)
    pn = torch.where(greedy[last], 1.0, p[last].gather(1, new[:, None])[:, 0])       # what the target gave each token
    pt = torch.where(greedy, 1.0, pt)
    s["prob"].copy_(torch.where(place < kept[seq], pt, torch.where(place == kept[seq], pn[seq], 0.0)))
    return [s["out"], s["count"], s["prob"]]


def _resize(s, c, want, copies):
    """Sequences take `want` tokens: pages behind them are given back, missing ones taken, lowest numbers first; a last
    page that others hold is exchanged before tokens are added to it."""
    page, pages, lens, refs = c["page"], s["pages"], s["lens"], s["refs"]
    rows, width = pages.shape
    i = torch.arange(width, device=pages.device)
    old, new = (lens + page - 1) // page, (want + page - 1) // page
    gone = (i >= new[:, None]) & (i < old[:, None])
    flat = pages.clamp(min=0).long().reshape(-1)
    refs.index_add_(0, flat, -gone.reshape(-1).to(torch.int32))
    pages.masked_fill_(gone, -1)
    tail = (lens // page).clamp(max=width - 1).long()
    last = pages.gather(1, tail[:, None])[:, 0]
    grows = want > lens
    swap = grows & (lens % page > 0) & (refs[last.clamp(min=0).long()] > 1)
    need = (new - old).clamp(min=0) + swap
    upto = need.cumsum(0)
    rank = torch.where(refs <= 0, 1, 0).cumsum(0)                    # of free pages, 1 for the lowest
    fits = (need == 0) | (upto <= rank[-1])
    first = upto - need
    # page `rank` r of the free ones, as an array
    order = torch.full((refs.numel() + 1,), -1, dtype=torch.int32, device=refs.device)
    order.scatter_(0, torch.where(refs <= 0, rank - 1, refs.numel()).long(),
                   torch.arange(refs.numel(), dtype=torch.int32, device=refs.device))
    swap = swap & fits
    put = fits[:, None] & grows[:, None] & (i >= old[:, None]) & (i < new[:, None])
    put |= swap[:, None] & (i == tail[:, None])
    place = first[:, None] + i - old[:, None] + swap[:, None]
    place = torch.where(swap[:, None] & (i == tail[:, None]), first[:, None], place)
    fresh = order[place.clamp(0, refs.numel()).long()]
    one = torch.where(put, 1, 0).to(torch.int32).reshape(-1)
    refs.index_add_(0, torch.where(put, fresh, 0).long().reshape(-1), one)
    refs.index_add_(0, last.clamp(min=0).long(), -swap.to(torch.int32))
    to = fresh.gather(1, tail[:, None])[:, 0]
    copies.copy_(torch.where(swap[:, None], torch.stack([last, to], 1), -1))
    pages.copy_(torch.where(put, fresh, pages))
    lens.copy_(torch.where(fits, want, lens))
    s["status"].copy_((~fits.all()).to(torch.int32)[None])


def _plain_tables(s, c):
    _resize(s, c, s["less"], s["none"])
    src, dst = s["src"].long(), s["dst"].long()
    i = torch.arange(s["pages"].shape[1], device=src.device)
    shared = i < ((s["lens"] + c["page"] - 1) // c["page"])[src][:, None]
    s["pages"][dst] = torch.where(shared, s["pages"][src], s["pages"][dst])
    s["refs"].index_add_(0, s["pages"][src].clamp(min=0).long().reshape(-1), shared.reshape(-1).to(torch.int32))
    s["lens"][dst] = s["lens"][src]
    _resize(s, c, s["more"], s["copies"])
    return [s["pages"], s["lens"], s["refs"], s["copies"], s["status"]]


def _bits(pool):
    return pool.view(torch.int16 if pool.element_size() == 2 else torch.uint8)


def _plain_copy(s, c):
    pool, pairs = _bits(s["pool"]), s["pairs"].long()
    # a pair that is none is done as the last one
    pairs = torch.where(pairs[:, :1] >= 0, pairs, pairs[-1])
    pool[:, :, pairs[:, 1]] = pool[:, :, pairs[:, 0]]
    return s["pool"]


def _plain_compact(s, c):
    pool, page = _bits(s["pool"]), c["page"]
    token = torch.arange(s["keep"].numel(), device=pool.device)
    seq = torch.searchsorted(s["start"].long(), token, right=True) - 1
    to, at = token - s["start"][seq].long(), s["keep"].long()
    rows = pool[:, :, s["src"][seq, at // page].long(), :, at % page]
    pool[:, :, s["dst"][seq, to // page].long(), :, to % page] = rows
    return s["pool"]


def _plain_product(s, c):
    w = _values(s["w"], c["out"], c["inn"])
    x = s["x"].float()
    if c["op"] == "mx4q":
        codes, scale = _quantized(x)
        x = _values(_packed(codes, scale), c["t"], c["inn"])
    s["y"].copy_(torch.matmul(x, w.t()))
    return s["y"]


def _plain_pack(s, c):
    codes, scale = _quantized(s["x"].float())
    s["out"].copy_(_values(_packed(codes, scale), c["out"], c["inn"]))
    return s["out"]


# ------------------------------------------------------------------ exact
def exact(c, seed):
    if c["op"] == "tables":
        return None
    s = prepare(c, seed)
    return {"verify": _exact_verify, "copy": _exact_copy, "compact": _exact_compact, "mx4": _exact_product,
            "mx4q": _exact_product, "pack": lambda s, c: _nearest(s["x"].double())}[c["op"]](s, c)


def _exact_verify(s, c):
    starts, tokens = s["q_start"].tolist(), s["tokens"].tolist()
    out, count, prob = [-1] * s["n"], [], torch.zeros(s["n"], dtype=torch.float64, device=DEV)
    for b in range(c["b"]):
        t = float(s["temperature"][b])
        got = []
        for r in range(starts[b], starts[b + 1]):
            x = s["target"][r].double()
            p = (x == x.max()).double() if t <= 0 else torch.softmax(x / t, 0)
            if t <= 0:
                p = torch.zeros_like(p).index_fill_(0, p.nonzero()[0], 1.0)
            d = tokens[r + 1] if r + 1 < starts[b + 1] else -1
            q = torch.zeros_like(p)
            if d >= 0 and s["draft"] is not None and t > 0:
                q = torch.softmax(s["draft"][r].double() / t, 0)
            elif d >= 0:
                q[d] = 1.0
            if d >= 0 and float(s["accept"][r]) * float(q[d]) < float(p[d]):
                got.append(d)
                prob[r] = p[d]
                continue
            w = (p - q).clamp(min=0)
            w = w if float(w.sum()) > 0 else p
            sums = torch.cumsum(w, 0)
            got.append(int((sums <= float(s["pick"][b]) * sums[-1]).sum()))
            prob[r] = p[got[-1]]
            break
        out[starts[b]:starts[b] + len(got)] = got
        count.append(len(got))
    return [_i32(out), _i32(count), prob]


def _exact_copy(s, c):
    pool = s["pool"].double()
    for a, b in s["pairs"].tolist():
        if a >= 0:
            pool[:, :, b] = pool[:, :, a]
    return pool


def _exact_compact(s, c):
    pool, page = s["pool"].double(), c["page"]
    starts = s["start"].tolist()
    for b in range(c["b"]):
        keep = s["keep"][starts[b]:starts[b + 1]].long()
        rows = pool[:, :, s["src"][b].long()].transpose(2, 3).flatten(3, 4)[:, :, :, keep]
        for i in range(0, len(keep), page):
            part = rows[:, :, :, i:i + page]
            pool[:, :, int(s["dst"][b, i // page]), :, :part.shape[3]] = part
    return pool


_POINTS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(x):
    """The values that a 64-bit tensor's blocks of 32 columns take in the format: the nearest point of the block's grid,
    of two equally near ones the one with the even code."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -125)
    scale = top / torch.frexp(top).mantissa / 8    # top = mantissa 2^n with the mantissa in [1/2, 1): floor(log2) = n - 1
    v = b.abs() / scale
    y = torch.zeros_like(v)
    for k in range(1, 8):
        half = (_POINTS[k - 1] + _POINTS[k]) / 2
        y = torch.where(v >= half if k % 2 == 0 else v > half, _POINTS[k], y)
    return (torch.copysign(y, b) * scale).view(x.shape)


def _exact_product(s, c):
    if 2 * c["t"] * c["out"] * c["inn"] > 5e14:
        return None
    w = _values(s["w"], c["out"], c["inn"], torch.float64)
    x = s["x"].double()
    if c["op"] == "mx4q":
        x = _nearest(x)
    return x @ w.t()
