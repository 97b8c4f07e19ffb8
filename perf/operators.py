"""Cases of the decoder-layer operators around the delta products: appending rotated keys and values to a paged
cache, attention over the cache for a batch whose sequences share prefixes, and products with a 4-bit backbone.

own = False computes the plain forms (elementary torch operations in 32 bits); own = True calls the library.
Lengths are a function of the case (not of the seed), so that work(case) can count them.  `lens` of a case spreads
its sequences' lengths between half of the bound and the bound; "with_empty" gives one sequence no key at all.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one chat joins the cache of a 7B layer (32 heads): the smallest call, where latency counts
        dict(name="append_1_7b", op="append", n=1, hq=32, hkv=32, d=128, page=16, kv="bf16", rot=128, inter=False,
             far=4096),
        # a decode step of 64 chats of a grouped-query layer, e4m3 cache, far positions, fused qkv rows
        dict(name="append_64_gqa_e4m3", op="append", n=64, hq=32, hkv=8, d=128, page=64, kv="e4m3", rot=128,
             inter=False, far=120000),
        # the prompts of 8 tenants x 2048 tokens of a 13B layer (40 heads)
        dict(name="append_16384_13b", op="append", n=16384, hq=40, hkv=40, d=128, page=64, kv="bf16", rot=128,
             inter=False, far=16384),
        # one chat of about a thousand tokens, 7B layer, no shared prefix: the smallest attention call
        dict(name="attn_1x1000_7b", op="attn", b=1, g=0, nq=1, prefix=0, own_kv=1000, hq=32, hkv=32, d=128, page=16,
             kv="bf16", with_empty=False),
        # 64 chats over 16 tenants, each tenant's system prompt shared by its chats
        dict(name="attn_64x16pre2048_gqa", op="attn", b=64, g=16, nq=1, prefix=2048, own_kv=700, hq=32, hkv=8, d=128,
             page=64, kv="bf16", with_empty=False),
        # 48 chats of one tenant over one long document, e4m3 cache
        dict(name="attn_48x1pre30000_e4m3", op="attn", b=48, g=1, nq=1, prefix=30000, own_kv=333, hq=32, hkv=8, d=128,
             page=32, kv="e4m3", with_empty=True),
        # 4 long chats without a shared prefix: few rows, a long axis
        dict(name="attn_4x131072_gqa", op="attn", b=4, g=0, nq=1, prefix=0, own_kv=131072, hq=32, hkv=8, d=128, page=64,
             kv="bf16", with_empty=False),
        # 20 chats check 5 drafted tokens each; 13B layer, 3 tenants' prompts of an odd length
        dict(name="attn_20x5_3pre1111_13b", op="attn", b=20, g=3, nq=5, prefix=1111, own_kv=413, hq=40, hkv=40, d=128,
             page=16, kv="bf16", with_empty=True),
        # the prompts of 8 tenants x 2048 tokens, grouped-query layer, causal
        dict(name="attn_prompt_8x2048_gqa", op="attn", b=8, g=0, nq=2048, prefix=0, own_kv=2048, hq=32, hkv=8, d=128,
             page=64, kv="bf16", with_empty=False),
        # one token through the q, k, v or o matrix of a 7B layer
        dict(name="w4_1_4096x4096", op="w4", t=1, out=4096, inn=4096),
        # one token through the down matrix of a grouped-query model's layer, 7 tokens of drafted text
        dict(name="w4_7_4096x14336", op="w4", t=7, out=4096, inn=14336),
        # a step of 64 chats through the gate or up matrix of a 7B layer
        dict(name="w4_64_11008x4096", op="w4", t=64, out=11008, inn=4096),
    ]


HEADS = [(32, 32), (40, 40), (32, 8), (16, 4), (8, 8), (24, 4)]
SHAPES = [(4096, 4096), (1024, 4096), (5120, 5120), (11008, 4096), (4096, 11008), (14336, 4096), (4096, 14336),
          (13824, 5120), (5120, 13824), (512, 1152), (1920, 640)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "w4"])
    if op == "w4":
        out, inn = rng.choice(SHAPES)
        return dict(op="w4", t=_log(rng, 1, 64), out=out, inn=inn)
    hq, hkv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "append":
        return dict(op="append", n=_log(rng, 1, 8192), hq=hq, hkv=hkv, d=d, page=page, kv=kv,
                    rot=rng.choice([d, d, d // 2]), inter=rng.random() < 0.3, far=_log(rng, 100, 200000))
    g = rng.choice([0, 0, 1, 3, 8])
    b = max(g, _log(rng, 1, 64))
    prefix = _log(rng, 1, 16384) if g else 0
    long = rng.random() < 0.3   # prompts; otherwise a few tokens a sequence
    if long:
        b, prefix = min(b, 8), min(prefix, 2048)
        g = min(g, b)
        own_kv = _log(rng, 64, 2048)
        nq = max(1, int(own_kv * rng.uniform(0.3, 1.0)))
        b = max(1, min(b, 600000000 // (nq * hq * (prefix + own_kv))))
        g = min(g, b)
        prefix = prefix if g else 0
    else:
        nq = rng.choice([1, 1, 1, 2, 5, 8])
        own_kv = max(nq, _log(rng, 1, 32768))
        own_kv = max(nq, min(own_kv, 900000 // (b * hkv)))   # the plain form holds every key in 32 bits
        prefix = min(prefix, 6000000 // (b * hkv))
    return dict(op="attn", b=b, g=g, nq=nq, prefix=prefix, own_kv=own_kv, hq=hq, hkv=hkv, d=d, page=page, kv=kv,
                with_empty=rng.random() < 0.3)


# ---------------------------------------------------------------- lengths
def _spread(i, lo, hi):
    """A length between lo and hi for item i."""
    return lo + (i * 40503 + 11 * i * i + 7) % 65521 % (hi - lo + 1)


def _lengths(c):
    """Host lists of an attention case: query tokens and own keys of each sequence, the sequences of each group (as
    starts) and the prefix length of each group.  The last sequence takes the bounds themselves."""
    b, g = c["b"], c["g"]
    nq = [c["nq"] if i == b - 1 or c["nq"] <= 8 else _spread(i, (c["nq"] + 1) // 2, c["nq"]) for i in range(b)]
    kv = [c["own_kv"] if i == b - 1 else max(nq[i], _spread(i, (c["own_kv"] + 1) // 2, c["own_kv"])) for i in range(b)]
    if c["with_empty"]:   # a sequence that has no key of its own yet (and, without a prefix, none at all)
        kv[0] = 0
    start = [int(math.ceil(b * (k / g) ** 1.5)) for k in range(g)] + [b] if g else [0]
    pre = [c["prefix"] if k == g - 1 else _spread(k + 5, (c["prefix"] + 1) // 2, c["prefix"]) for k in range(g)]
    return nq, kv, start, pre


def _pages(n, page):
    return (n + page - 1) // page


def work(c):
    if c["op"] == "append":
        e = 2 if c["kv"] == "bf16" else 1
        el = c["n"] * c["d"]
        return {"bytes": el * (c["hq"] * 4 + 2 * c["hkv"] * (2 + e)) + 12 * c["n"], "flops": 3 * el * (c["hq"] + c["hkv"])}
    if c["op"] == "w4":
        t, out, inn = c["t"], c["out"], c["inn"]
        return {"bytes": out * inn // 2 + 4 * out * (inn // 128) + 2 * t * (inn + out), "flops": 2 * t * out * inn}
    nq, kv, start, pre = _lengths(c)
    e = 2 if c["kv"] == "bf16" else 1
    keys = sum(kv) + sum(p for k, p in enumerate(pre) if start[k + 1] > start[k])
    pairs = 0
    for k in range(max(1, c["g"])):
        lo, hi = (start[k], start[k + 1]) if c["g"] else (0, c["b"])
        for i in range(lo, hi):
            first = kv[i] - nq[i]
            pairs += nq[i] * (pre[k] if c["g"] else 0) + sum(max(0, first + j + 1) for j in range(nq[i]))
    return {"bytes": 2 * keys * c["hkv"] * c["d"] * e + 4 * sum(nq) * c["hq"] * c["d"],
            "flops": 4 * pairs * c["hq"] * c["d"]}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _bf16(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _cache(c, pages, g, std):
    """A page pool [pages][heads][page][d] in use, and its scales."""
    shape = (pages, c["hkv"], c["page"], c["d"])
    if c["kv"] == "bf16":
        return _bf16(shape, g, std), None
    scale = torch.rand(c["hkv"], generator=g, device=DEV) * 0.02 + 0.01
    x = torch.randn(shape, generator=g, device=DEV) * std / scale[None, :, None, None]
    return x.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] == "w4":
        return _prepare_w4(c, g)
    if c["op"] == "append":
        return _prepare_append(c, g)
    return _prepare_attn(c, g)


def _prepare_append(c, g):
    n, d, page = c["n"], c["d"], c["page"]
    pages = _pages(n, page) + 8
    k, ks = _cache(c, pages, g, 1.0)
    v, vs = _cache(c, pages, g, 1.0)
    qkv = _bf16((n, (c["hq"] + 2 * c["hkv"]) * d), g)   # the rows of a fused projection
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int64)
    if n > 8:
        slots[n // 3] = -1   # a padded row: not stored
    pos = torch.randint(0, c["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
    s = dict(c=c, k=k, v=v, ks=ks, vs=vs, qkv=qkv, slots=slots, pos=pos, freq=freq,
             q_out=torch.empty((n, c["hq"] * d), dtype=torch.bfloat16, device=DEV))
    if own:   # the views that a serving loop keeps
        import tenant_rank_serving_amd as trs
        s["cache"] = trs.KvCache(k, v, ks, vs)
        s["rope"] = trs.Rope(freq, interleaved=c["inter"])
    return s


def _tables(lens, page, first, perm, width):
    """Page tables [len(lens)][width]: sequence i takes the next pages of the shuffled pool; the rest is -1."""
    t = torch.full((max(1, len(lens)), max(1, width)), -1, dtype=torch.int32)
    for i, n in enumerate(lens):
        m = _pages(n, page)
        t[i, :m] = perm[first:first + m]
        first += m
    return t.to(DEV), first


def _prepare_attn(c, g):
    nq, kv, start, pre = _lengths(c)
    page = c["page"]
    total = sum(_pages(n, page) for n in kv) + sum(_pages(n, page) for n in pre) + 3
    k, ks = _cache(c, total, g, 1.5)
    v, vs = _cache(c, total, g, 1.0)
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
    own_pages, used = _tables(kv, page, 0, perm, _pages(c["own_kv"], page))
    pre_pages, used = _tables(pre, page, used, perm, _pages(c["prefix"], page))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    q_start = i32([sum(nq[:i]) for i in range(c["b"] + 1)])
    n = sum(nq)
    s = dict(c=c, n=n, k=k, v=v, ks=ks, vs=vs, q=_bf16((n, c["hq"] * c["d"]), g, 1.5), q_start=q_start, kv_len=i32(kv),
             pages=own_pages, group_start=i32(start), prefix_len=i32(pre), prefix_pages=pre_pages,
             y=torch.zeros((n, c["hq"] * c["d"]), dtype=torch.bfloat16, device=DEV))
    if own:   # the views and the plan that a serving loop keeps; they hold the tensors' addresses and the bounds only
        import tenant_rank_serving_amd as trs
        s["cache"] = trs.KvCache(k, v, ks, vs)
        groups = dict(group_start=s["group_start"], prefix_len=s["prefix_len"], prefix_pages=pre_pages,
                      max_prefix=c["prefix"],
                      max_group_q=max(sum(nq[start[j]:start[j + 1]]) for j in range(c["g"]))) if c["g"] else {}
        s["batch"] = trs.AttnBatch(q_start, s["kv_len"], own_pages, max_q=c["nq"], max_kv=c["own_kv"], **groups)
        s["ws"] = torch.empty(trs.dc_attention_workspace_bytes(s["cache"], s["batch"], c["hq"], n), dtype=torch.uint8,
                              device=DEV)
    return s


def _prepare_w4(c, g):
    t, out, inn = c["t"], c["out"], c["inn"]
    codes = torch.randint(0, 16, (out, inn), generator=g, device=DEV, dtype=torch.int32)
    scale = torch.exp(torch.randn((inn // 128, out), generator=g, device=DEV) * 0.5 - 5.0).to(torch.float16)
    zero = torch.randint(4, 12, (inn // 128, out), generator=g, device=DEV).to(torch.float16)
    w4 = _pack_w4(codes, scale, zero)
    s = dict(c=c, w4=w4, x=_bf16((t, inn), g), y=torch.empty((t, out), dtype=torch.bfloat16, device=DEV))
    if own:
        import tenant_rank_serving_amd as trs
        s["view"] = trs.W4View(out, inn, w4)
    return s


# The 4-bit format: codes [out/16][in/128][4][16][4] words, word (T, g, c, i, j) holding the codes of row 16T + i,
# columns 128g + 32c + 8j + e, code e at bit 4(e/2) + 16(e%2); then scale | zero << 16 as words [in/128][out].
def _pack_w4(codes, scale, zero):
    out, inn = codes.shape
    w = codes.view(out // 16, 16, inn // 128, 4, 4, 8).permute(0, 2, 3, 1, 4, 5).to(torch.int64)
    e = torch.arange(8, device=DEV)
    words = (w << (4 * (e // 2) + 16 * (e % 2))).sum(-1).reshape(-1)
    sz = (scale.view(torch.int16).to(torch.int64) & 0xFFFF) | ((zero.view(torch.int16).to(torch.int64) & 0xFFFF) << 16)
    both = torch.cat([words, sz.reshape(-1)])
    return torch.where(both >= 1 << 31, both - (1 << 32), both).to(torch.int32)


def _unpack_w4(w4, out, inn):
    """(codes [out][in], scale [in/128][out], zero [in/128][out]) of a 4-bit buffer, as int32 and fp16."""
    nc = out * inn // 8
    e = torch.arange(8, device=w4.device, dtype=torch.int32)
    codes = (w4[:nc, None] >> (4 * (e // 2) + 16 * (e % 2))) & 15
    codes = codes.view(out // 16, inn // 128, 4, 16, 4, 8).permute(0, 3, 1, 2, 4, 5).reshape(out, inn)
    sz = w4[nc:nc + out * (inn // 128)].view(torch.float16).view(inn // 128, out, 2)
    return codes, sz[..., 0], sz[..., 1]


# ------------------------------------------------------------------- runs
def run(s):
    c = s["c"]
    if own:
        return _own(s, c)
    if c["op"] == "append":
        return _plain_append(s, c)
    if c["op"] == "w4":
        return _plain_w4(s, c)
    return _plain_attn(s, c)


def _own(s, c):
    import tenant_rank_serving_amd as trs
    if c["op"] == "append":
        d, hq, hkv = c["d"], c["hq"], c["hkv"]
        q, k, v = s["qkv"].split([hq * d, hkv * d, hkv * d], dim=1)
        trs.dc_kv_append(s["cache"], q, k, v, s["pos"], s["slots"], s["rope"], s["q_out"])
        return [s["q_out"], s["k"], s["v"]]
    if c["op"] == "w4":
        trs.dc_apply_w4(s["view"], s["x"], s["y"])
        return s["y"]
    trs.dc_attention(s["cache"], s["q"], s["batch"], c["d"] ** -0.5, s["y"], s["ws"])
    return s["y"]


def _rotated(x, cos, sin, rot, inter):
    """x fp32 [n][h][d] with its first rot elements rotated by the angles whose cos and sin are [n][1][rot/2]."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_append(s, c):
    n, d, hq, hkv, page = c["n"], c["d"], c["hq"], c["hkv"], c["page"]
    x = s["qkv"].float().view(n, hq + 2 * hkv, d)
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    qk = _rotated(x[:, :hq + hkv], cos, sin, c["rot"], c["inter"])
    s["q_out"].copy_(qk[:, :hq].reshape(n, hq * d))
    # rows that are not stored: written back as they are, by the row of another slot's own value
    keep = s["slots"] >= 0
    at = torch.where(keep, s["slots"], s["slots"].max())
    src = torch.where(keep, torch.arange(n, device=x.device), s["slots"].argmax())
    pg, sl = at // page, at % page
    for cache, scale, new in ((s["k"], s["ks"], qk[:, hq:]), (s["v"], s["vs"], x[:, hq + hkv:])):
        new = new if scale is None else (new / scale[:, None]).clamp(-448, 448)
        new = new.to(cache.dtype)[src]
        if scale is None:
            cache[pg, :, sl] = new
        else:
            cache.view(torch.uint8)[pg, :, sl] = new.view(torch.uint8)
    return [s["q_out"], s["k"], s["v"]]


def _keys(cache, scale, page, tables, lens, width):
    """The first `width` rows of each table's sequence as fp32 [rows][width][heads][d], zero past its length."""
    i = torch.arange(width, device=cache.device)
    pg = tables[:, i // page].long().clamp(min=0)
    x = cache[pg, :, (i % page)[None, :]].float() if scale is None else \
        cache.view(torch.uint8)[pg, :, (i % page)[None, :]].view(torch.float8_e4m3fn).float() * scale[:, None]
    return torch.where((i < lens[:, None])[..., None, None], x, 0.0)


def _plain_attn(s, c):
    b, hq, hkv, d, page, nq = c["b"], c["hq"], c["hkv"], c["d"], c["page"], c["nq"]
    dev = s["q"].device
    seq = torch.arange(b, device=dev)
    count = s["q_start"][1:] - s["q_start"][:-1]
    lens = s["kv_len"]
    # each sequence's keys: its own, behind those of its group's prefix
    parts, vis = [], []
    j = torch.arange(nq, device=dev)
    if c["g"]:
        grp = torch.searchsorted(s["group_start"], seq.to(torch.int32), right=True) - 1
        plen = s["prefix_len"][grp]
        parts.append((s["prefix_pages"][grp], plen, c["prefix"]))
        vis.append((torch.arange(c["prefix"], device=dev) < plen[:, None])[:, None, :].expand(b, nq, c["prefix"]))
    parts.append((s["pages"], lens, c["own_kv"]))
    last = (lens - count)[:, None] + j                     # the newest own key that query j sees
    vis.append(torch.arange(c["own_kv"], device=dev) <= last[..., None])
    k = torch.cat([_keys(s["k"], s["ks"], page, t, n, w) for t, n, w in parts], 1).permute(0, 2, 3, 1).contiguous()
    v = torch.cat([_keys(s["v"], s["vs"], page, t, n, w) for t, n, w in parts], 1).permute(0, 2, 1, 3).contiguous()
    vis = torch.cat(vis, 2)                                # [b][nq][keys]
    # query rows of each sequence, padded to nq: [b][kv head][nq * heads of it][d]
    rows = (s["q_start"][:-1, None] + j).clamp(max=s["n"] - 1).long()
    q = s["q"].float().view(s["n"], hkv, hq // hkv, d)[rows].permute(0, 2, 1, 3, 4).reshape(b, hkv, nq * (hq // hkv), d)
    sc = torch.matmul(q, k).mul_(d ** -0.5).view(b, hkv, nq, hq // hkv, -1)
    seen = vis[:, None, :, None, :]
    sc = torch.where(seen, sc, -math.inf)
    top = sc.amax(-1, keepdim=True).clamp(min=-3e38)       # a row that sees no key has no weight
    sc = sc.sub_(top).exp_()
    total = sc.sum(-1, keepdim=True)
    y = torch.matmul(sc.view(b, hkv, nq * (hq // hkv), -1), v).view(b, hkv, nq, hq // hkv, d)
    y = (y / torch.where(total > 0, total, 1.0)).permute(0, 2, 1, 3, 4).reshape(b, nq, hq * d)
    token = torch.arange(s["n"], device=dev)
    of = torch.searchsorted(s["q_start"], token.to(torch.int32), right=True) - 1
    s["y"].copy_(y[of, token - s["q_start"][of]])
    return s["y"]


def _plain_w4(s, c):
    codes, scale, zero = _unpack_w4(s["w4"], c["out"], c["inn"])
    w = codes.view(c["out"], -1, 128).float() - zero.t().float()[..., None]
    w = (w * scale.t().float()[..., None]).view(c["out"], c["inn"])
    s["y"].copy_(torch.matmul(s["x"].float(), w.t()))
    return s["y"]


# ------------------------------------------------------------------ exact
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(s, c)
    if c["op"] == "w4":
        codes, scale, zero = _unpack_w4(s["w4"], c["out"], c["inn"])
        y = torch.zeros((c["t"], c["out"]), dtype=torch.float64, device=DEV)
        for i in range(c["inn"] // 128):
            x = s["x"][:, 128 * i:128 * i + 128].double()
            y += (x @ codes[:, 128 * i:128 * i + 128].double().t() - x.sum(1, keepdim=True) * zero[i].double()) * scale[i].double()
        return y
    return _exact_attn(s, c)


def _exact_append(s, c):
    d, hq, hkv, rot = c["d"], c["hq"], c["hkv"], c["rot"]
    x = s["qkv"].double().view(c["n"], -1, d)
    z = torch.polar(torch.ones((c["n"], rot // 2), dtype=torch.float64, device=DEV), s["pos"].double()[:, None] * s["freq"])
    i = torch.arange(rot // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rot // 2)
    w = torch.complex(x[:, :hq + hkv][..., first], x[:, :hq + hkv][..., second]) * z[:, None]
    qk = x[:, :hq + hkv].clone()
    qk[..., first], qk[..., second] = w.real, w.imag
    flat = lambda t: t.double().permute(0, 2, 1, 3).reshape(-1, hkv, d).clone()  # noqa: E731
    sel = s["slots"] >= 0
    out = []
    for cache, scale, new in ((s["k"], s["ks"], qk[:, hq:]), (s["v"], s["vs"], x[:, hq + hkv:])):
        rows = flat(cache)
        if scale is not None:   # an e4m3 cache holds codes: what they would be without their rounding
            new = (new / scale.double()[:, None]).clamp(-448, 448)
        rows[s["slots"][sel]] = new[sel]
        out.append(rows.view(-1, c["page"], hkv, d).permute(0, 2, 1, 3).contiguous())
    return [qk[:, :hq].reshape(c["n"], hq * d), out[0], out[1]]


def _exact_attn(s, c):
    nq, kv, start, pre = _lengths(c)
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    y = torch.zeros((s["n"], hq, d), dtype=torch.float64, device=DEV)

    def rows(cache, scale, table, n, h):
        t = table[:_pages(n, page)].long()
        r = cache[t, h].double() if scale is None else \
            cache.view(torch.uint8)[t, h].view(torch.float8_e4m3fn).double() * scale[h].double()
        return r.reshape(-1, d)[:n]

    if sum(n * (c["prefix"] + m) for n, m in zip(nq, kv)) * hq > 4e9:
        return None
    at = 0
    for i in range(c["b"]):
        k = max([j for j in range(c["g"]) if start[j] <= i], default=None)
        # of several groups that start at the same sequence, the last one holds it
        q = s["q"].view(s["n"], hq, d)[at:at + nq[i]].double()
        see = torch.arange(kv[i], device=DEV)[None] <= torch.arange(nq[i], device=DEV)[:, None] + kv[i] - nq[i]
        if k is not None:
            see = torch.cat([torch.ones((nq[i], pre[k]), dtype=torch.bool, device=DEV), see], 1)
        for h in range(hkv):
            K, V = rows(s["k"], s["ks"], s["pages"][i], kv[i], h), rows(s["v"], s["vs"], s["pages"][i], kv[i], h)
            if k is not None:
                K = torch.cat([rows(s["k"], s["ks"], s["prefix_pages"][k], pre[k], h), K])
                V = torch.cat([rows(s["v"], s["vs"], s["prefix_pages"][k], pre[k], h), V])
            if not K.shape[0]:
                continue
            r = hq // hkv
            sc = torch.einsum("nhd,kd->nhk", q[:, h * r:h * r + r], K) / math.sqrt(d)
            sc = sc.masked_fill(~see[:, None], -math.inf)
            p = torch.softmax(sc, -1).nan_to_num(0.0)
            y[at:at + nq[i], h * r:h * r + r] = torch.einsum("nhk,kd->nhd", p, V)
        at += nq[i]
    return y.view(s["n"], hq * d)
