"""Cases, plain forms and exact values of the paged 8-bit KV cache operators.

Three operators, as a serving or training program of this library uses them:
  rope    rotary positions of q, k or the indexer's heads, and their gradient
  append  new keys and values into a paged 8-bit cache, keys rotated on the way
  attn    attention over that cache: every cached key, or the keys that top-k selected
"""
import math
import random

import torch

own = False

D = 128          # head dimension of K and V
E_MIN = -64      # least scale exponent of a cache block
FMT = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's queries of 16 sequences at 128K: latency counts
        dict(name="rope_decode_16", op="rope", T=16, H=32, D=128, R=128, off=0, inter=False, dtype="bf16",
             inverse=False, fused=False, far=131072, yarn=0.0),
        # queries of a 128K prefill, rotated out of the fused qkv projection
        dict(name="rope_prefill_128k", op="rope", T=131072, H=32, D=128, R=128, off=0, inter=False, dtype="bf16",
             inverse=False, fused=True, far=0, yarn=0.0),
        # gradient of the indexer's queries in training: half of each 64-wide head rotated, pairs interleaved
        dict(name="rope_bwd_indexer_32k", op="rope", T=32768, H=32, D=64, R=32, off=32, inter=True, dtype="bf16",
             inverse=True, fused=False, far=0, yarn=8.0),
        # gradient of K's heads kept in fp32, an odd token count, long-context scaling
        dict(name="rope_bwd_fp32_4095", op="rope", T=4095, H=4, D=128, R=64, off=0, inter=False, dtype="fp32",
             inverse=True, fused=False, far=1000000, yarn=32.0),
        # one decode step: 16 sequences near 128K, one token each
        dict(name="append_decode_16", op="append", B=16, Hkv=4, page=64, fmt="e4m3", ctx=131072, new=1, ragged=0,
             R=128, inter=False),
        # prefill of eight sequences, 64K tokens in all, into empty and partly filled pages
        dict(name="append_prefill_64k", op="append", B=8, Hkv=4, page=64, fmt="e4m3", ctx=500, new=8192, ragged=1,
             R=128, inter=False),
        # short ragged chunks of many sequences, position-free keys in 8-bit integers
        dict(name="append_int8_ragged", op="append", B=61, Hkv=2, page=16, fmt="int8", ctx=1000, new=37, ragged=1,
             R=0, inter=False),
        # one short sequence: a chat's first tokens
        dict(name="attn_short_1", op="attn", B=1, rows=1, Hq=32, Hkv=4, page=64, fmt="e4m3", n=777, ragged=0, topk=0),
        # the decode workload: 16 sequences of 128K keys, each read whole
        dict(name="attn_decode_16x128k", op="attn", B=16, rows=1, Hq=32, Hkv=4, page=64, fmt="e4m3", n=131328,
             ragged=0, topk=0),
        # a serving batch of uneven lengths, 8-bit integers, 16 heads a KV head, two rows a sequence
        dict(name="attn_ragged_61_int8", op="attn", B=61, rows=2, Hq=32, Hkv=2, page=16, fmt="int8", n=16000,
             ragged=1, topk=0),
        # the decode workload's sparse step: the 2048 selected keys of 128K, 16 sequences
        dict(name="attn_sparse_16x128k", op="attn", B=16, rows=1, Hq=32, Hkv=4, page=64, fmt="e4m3", n=131328,
             ragged=0, topk=2048),
        # a chunk of a sparse prefill over a 32K sequence
        dict(name="attn_sparse_prefill", op="attn", B=1, rows=1024, Hq=32, Hkv=4, page=64, fmt="e4m3", n=32768,
             ragged=0, topk=2048),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    if op == "rope":
        d = rng.choice([64, 128])
        r = rng.choice([16, 32, 48, 64, d])
        h = rng.choice([1, 2, 4, 8, 16, 32])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, T=_between(rng, 1, (1 << 22) // h // (2 if dtype == "fp32" else 1) // 2), H=h, D=d, R=r,
                    off=rng.choice([0, d - r]), inter=rng.random() < 0.5, dtype=dtype,
                    inverse=rng.random() < 0.5, fused=rng.random() < 0.5, far=rng.choice([0, 131072, 1000000]),
                    yarn=rng.choice([0.0, 8.0, 32.0]))
    hkv = rng.choice([1, 2, 4])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["e4m3", "e4m3", "int8"])
    if op == "append":
        b = _between(rng, 1, 128)
        new = rng.choice([1, _between(rng, 1, 65536 // b)])
        return dict(op=op, B=b, Hkv=hkv, page=page, fmt=fmt, ctx=_between(rng, 1, (1 << 20) // b), new=new,
                    ragged=0 if new == 1 else 1, R=0 if fmt == "int8" else rng.choice([0, 32, 64, 128]),
                    inter=rng.random() < 0.5)
    g = rng.choice([1, 4, 7, 8, 16])
    b = _between(rng, 1, 128)
    rows = rng.choice([1, 1, _between(rng, 1, max(1, 512 // b))])
    topk = rng.choice([0, 0, _between(rng, 1, 2048)])
    most = (1 << 20) // (b * rows) if topk == 0 else 131072 // b
    return dict(op=op, B=b, rows=rows, Hq=g * hkv, Hkv=hkv, page=page, fmt=fmt, n=_between(rng, 1, max(2, most)),
                ragged=rng.choice([0, 1]), topk=topk)


def _lens(case, key):
    """Per-sequence lengths of a case: all near case[key], or anything from none to it (ragged)."""
    r = random.Random("%s %s" % (key, sorted((k, v) for k, v in case.items() if k != "name")))
    most = case[key]
    if case["ragged"]:
        lens = [int(most * r.random() ** 2) for _ in range(case["B"])]
        lens[r.randrange(case["B"])] = most
        return lens
    if key == "new":
        return [most] * case["B"]
    return [max(1, most - r.randrange(1 + most // 100)) for _ in range(case["B"])]


def work(case):
    if case["op"] == "rope":
        n, es = case["T"] * case["H"] * case["D"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * es, "flops": 3 * case["T"] * case["H"] * case["R"]}
    if case["op"] == "append":
        n, hkv = sum(_lens(case, "new")), case["Hkv"]
        return {"bytes": 2 * n * hkv * D * 3, "flops": 2 * n * hkv * D * 2 + 3 * n * hkv * case["R"]}
    n, rows, hkv = _lens(case, "n"), case["rows"], case["Hkv"]
    if case["topk"]:
        pairs = sum(rows * min(x, case["topk"]) for x in n)
        read = sum(min(x, rows * min(x, case["topk"])) for x in n)
    else:
        pairs = sum(sum(max(0, x - r) for r in range(rows)) for x in n)
        read = sum(n)
    t = case["B"] * rows
    return {"bytes": read * hkv * D * 2 + 4 * t * case["Hq"] * D + 4 * t * case["topk"],
            "flops": 4 * pairs * case["Hq"] * D}


# ------------------------------------------------------------------ inputs
def _inv_freq(r, yarn):
    """theta^(-2i/r); with yarn > 1 the slow half of them divided by that factor, a ramp between."""
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    f = 1e6 ** (-2 * i / r)
    if yarn:
        ramp = ((i / max(1, r // 2 - 1) - 0.25) * 2).clamp(0, 1)
        f = f * (1 - ramp) + f / yarn * ramp
    return f


def _seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _pages(case, lens, g):
    """A page pool, and a table that deals its pages to the sequences in any order."""
    page = case["page"]
    per = max(1, max(-(-x // page) for x in lens))
    count = sum(-(-x // page) for x in lens) + 3
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["B"], per), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, x in enumerate(lens):
        k = -(-x // page)
        table[b, :k] = order[at:at + k]
        at += k
    return count, table


def _filled(case, count, g):
    """A pool of `count` pages as earlier steps left it: values of a magnitude of their own in each page
    and head, rounded to 8 bits with the block's power-of-two scale."""
    dtype, top = FMT[case["fmt"]]
    x = _normal(g, count, case["page"], case["Hkv"], D)
    x *= torch.exp(0.5 * _normal(g, count, 1, case["Hkv"], 1))
    amax = x.abs().amax((1, 3)).float()
    m, e = torch.frexp(amax / top)
    scale = torch.exp2((e - (m == 0.5).int()).clamp(min=E_MIN).float())
    x = x / scale[:, None, :, None].to(torch.bfloat16)
    return (x.round() if dtype == torch.int8 else x).to(dtype), scale


def prepare(case, seed):
    g = _seeded(seed)
    s = dict(case)
    if case["op"] == "rope":
        t, h, d = case["T"], case["H"], case["D"]
        wide = h + 2 * max(1, h // 8) if case["fused"] else h
        x = _normal(g, t, wide * d)
        s["x"] = (x if case["dtype"] == "bf16" else x.float())[:, :h * d].unflatten(1, (h, d))
        s["inv_freq"] = _inv_freq(case["R"], case["yarn"])
        s["mscale"] = 0.1 * math.log(case["yarn"]) + 1.0 if case["yarn"] else 1.0
        s["pos"] = torch.randint(case["far"], (t,), generator=g, device="cuda", dtype=torch.int32) if case["far"] else None
        s["out"] = torch.empty((t, h, d), dtype=s["x"].dtype, device="cuda")
        return s
    if case["op"] == "append":
        ctx, new = _lens(case, "ctx"), _lens(case, "new")
        count, s["table"] = _pages(case, [a + b for a, b in zip(ctx, new)], g)
        s["k_pages"], s["k_scale"] = _filled(case, count, g)
        s["v_pages"], s["v_scale"] = _filled(case, count, g)
        n = sum(new)
        kv = _normal(g, n, 2 * case["Hkv"], D)
        kv *= torch.exp(0.7 * _normal(g, n, 1, 1))
        s["k_new"], s["v_new"] = kv[:, :case["Hkv"]], kv[:, case["Hkv"]:]
        s["ctx_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["cu_new"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32) if case["ragged"] else None
        s["inv_freq"] = _inv_freq(case["R"], 0.0) if case["R"] else None
        return s
    lens, rows = _lens(case, "n"), case["rows"]
    count, s["table"] = _pages(case, lens, g)
    s["k_pages"], s["k_scale"] = _filled(case, count, g)
    s["v_pages"], s["v_scale"] = _filled(case, count, g)
    s["q"] = _normal(g, case["B"] * rows, case["Hq"], D)
    s["scale"] = D ** -0.5
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["seq"] = torch.arange(case["B"], dtype=torch.int32, device="cuda").repeat_interleave(rows) if rows > 1 else None
    # the last of a sequence's rows sees all of it, each row before it one key less; sparse rows see all
    back = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    s["n_keys"] = (n[:, None] - (back if not case["topk"] else 0 * back)).clamp(min=0).flatten()
    s["most"] = max(lens)
    s["idx"] = None
    if case["topk"]:
        # scores with a part that a sequence's rows share, so that their selections overlap
        k = case["topk"]
        far = max(k, s["most"])
        at = torch.arange(far, device="cuda")
        some = torch.randn((case["B"], far // 64 + 1), generator=g, device="cuda")
        sc = torch.rand((case["B"] * rows, far), generator=g, device="cuda")
        sc += some.repeat_interleave(rows, 0)[:, at // 64]
        sc.masked_fill_(at >= s["n_keys"][:, None], -1e9)
        top, idx = sc.topk(k, dim=1)
        # in top-k's order: by (key / 32) mod 4, ascending, then the -1 padding
        order = torch.where(top < -1e8, 1 << 40, (idx // 32 % 4 << 32) + idx).argsort(1)
        s["idx"] = idx.masked_fill(top < -1e8, -1).gather(1, order).to(torch.int32)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"rope": _rope, "append": _append, "attn": _attn}[s["op"]](s)


def _own(s):
    import dsa_lightning_indexer_02_b200 as dsa
    if s["op"] == "rope":
        dsa.dsa_rope(s["x"], s["out"], s["inv_freq"], pos=s["pos"], rot_offset=s["off"], interleaved=s["inter"],
                     mscale=s["mscale"], inverse=s["inverse"])
        return s["out"]
    if s["op"] == "append":
        dsa.dsa_kv_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"],
                          s["ctx_len"], cu_new=s["cu_new"], inv_freq=s["inv_freq"], interleaved=s["inter"])
        return {"k": s["k_pages"], "v": s["v_pages"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    dsa.dsa_paged_attn(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["n_keys"],
                       s["scale"], s["out"], seq=s["seq"], idx=s["idx"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _turned(x, pos, inv_freq, off, inter, mscale, inverse):
    """x [T, H, D] in fp32 with the dims off .. off + 2 * len(inv_freq) rotated; angles in 64 bits."""
    r = 2 * inv_freq.shape[0]
    a = pos.double()[:, None] * inv_freq
    c, s = (mscale * a.cos()).float()[:, None], (mscale * a.sin()).float()[:, None]
    if inverse:
        s = -s
    y = x.float().clone()
    p = y[..., off:off + r]
    u, v = (p[..., 0::2], p[..., 1::2]) if inter else (p[..., :r // 2], p[..., r // 2:])
    nu, nv = u * c - v * s, u * s + v * c
    u.copy_(nu)
    v.copy_(nv)
    return y


def _rope(s):
    pos = torch.arange(s["T"], device="cuda") if s["pos"] is None else s["pos"]
    return _turned(s["x"], pos, s["inv_freq"], s["off"], s["inter"], s["mscale"], s["inverse"]).to(s["x"].dtype)


def _append(s):
    page, b, dev = s["page"], s["B"], "cuda"
    n = s["k_new"].shape[0]
    cu = torch.arange(b + 1, device=dev) if s["cu_new"] is None else s["cu_new"].long()
    tok = torch.arange(n, device=dev)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    ctx = s["ctx_len"].long()
    pos = ctx[seq] + tok - cu[seq]
    pid, slot = s["table"][seq, pos // page].long(), pos % page
    some = cu[1:] > cu[:-1]                              # sequences with new tokens
    first = s["table"].gather(1, (ctx // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    held = torch.where(some, ctx % page, 0)              # tokens that its first page holds already
    first = torch.where(held > 0, first, s["k_pages"].shape[0] - 1).clamp(min=0)
    k = s["k_new"].float() if s["inv_freq"] is None else _turned(s["k_new"], pos, s["inv_freq"], 0, s["inter"], 1.0, False)
    _store(s["k_pages"], s["k_scale"], k, pid, slot, first, held, s["fmt"])
    _store(s["v_pages"], s["v_scale"], s["v_new"].float(), pid, slot, first, held, s["fmt"])
    return {"k": s["k_pages"], "v": s["v_pages"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _round8(x, fmt):
    return (x.round() if fmt == "int8" else x).to(FMT[fmt][0]).view(torch.uint8)


def _store(pages, scale, x, pid, slot, first, held, fmt):
    """Rounds the tokens x to 8 bits and writes them at (pid, slot); a page's scale starts anew with its
    slot 0 and grows otherwise, the `held` tokens of the pages `first` being rounded again."""
    top = FMT[fmt][1]
    amax = torch.zeros_like(scale).scatter_reduce(0, pid[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax / top)                       # m in [0.5, 1): 2^(e-1) suffices where m is 0.5
    need = torch.exp2((e - (m == 0.5).int()).clamp(min=E_MIN).float())
    kept = torch.zeros(scale.shape[0], dtype=torch.int64, device="cuda").scatter_reduce(0, first, held, "amax") > 0
    hit = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill(0, pid, True)
    new = torch.where(hit[:, None], torch.where(kept[:, None], torch.maximum(scale, need), need), scale)
    raw = pages.view(torch.uint8)
    old = raw[first]
    again = _round8(pages[first].float() * (scale[first] / new[first])[:, None, :, None], fmt)
    mine = torch.arange(pages.shape[1], device="cuda") < held[:, None]
    at, where = mine.nonzero(as_tuple=True)
    raw[first[at], where] = torch.where(mine[..., None, None], again, old)[at, where]
    raw[pid, slot] = _round8(x / new[pid][..., None], fmt)
    scale.copy_(new)


def _attn(s):
    page, hkv = s["page"], s["Hkv"]
    t, hq, d = s["q"].shape
    n = s["n_keys"].long()
    if s["idx"] is None:
        pos = torch.arange(max(1, s["most"]), device="cuda").expand(t, -1)
        ok = pos < n[:, None]
    else:
        pos = s["idx"].long()
        ok = (pos >= 0) & (pos < n[:, None])
    pos = torch.where(ok, pos, 0)
    seq = torch.arange(t, device="cuda") if s["seq"] is None else s["seq"].long()
    pid = s["table"][seq[:, None], pos // page].clamp(min=0).long()
    row = pid * page + pos % page
    q = s["q"].float().unflatten(1, (hkv, hq // hkv))
    k = s["k_pages"].view(torch.uint8).flatten(0, 1)[row].view(FMT[s["fmt"]][0]).float() * s["k_scale"][pid][..., None]
    z = torch.einsum("thgd,tnhd->thgn", q, k) * s["scale"]
    del k
    z = z.masked_fill(~ok[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    v = s["v_pages"].view(torch.uint8).flatten(0, 1)[row].view(FMT[s["fmt"]][0]).float() * s["v_scale"][pid][..., None]
    o = torch.einsum("thgn,tnhd->thgd", p, v) / torch.where(l > 0, l, 1.0)
    return {"out": o.reshape(t, hq, d).to(torch.bfloat16), "lse": (m + l.log()).reshape(t, hq)}


# ------------------------------------------------------------------ values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)


def _exact_turn(x, pos, f, off, inter, m, sign):
    """Each rotated pair as a complex number times m * exp(sign * i * pos * f)."""
    n = f.shape[0]
    one = off + torch.arange(n, device=x.device) * (2 if inter else 1)
    two = one + (1 if inter else n)
    turn = torch.polar(torch.full_like(f, m).expand(len(pos), n), sign * pos.double()[:, None] * f)
    z = torch.complex(x[..., one], x[..., two]) * turn[:, None]
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_rope(s):
    pos = s["pos"] if s["pos"] is not None else torch.arange(s["T"], device="cuda")
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    for a in range(0, s["T"], 16384):
        y[a:a + 16384] = _exact_turn(s["x"][a:a + 16384].double(), pos[a:a + 16384], s["inv_freq"], s["off"],
                                     s["inter"], s["mscale"], -1.0 if s["inverse"] else 1.0)
    return y


def _exact_round(x, fmt):
    """The nearest value that 8 bits hold, ties to even, in 64 bits."""
    if fmt == "int8":
        return torch.round(x)
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    page, fmt = s["page"], s["fmt"]
    ctx = s["ctx_len"].tolist()
    cu = list(range(s["B"] + 1)) if s["cu_new"] is None else s["cu_new"].tolist()
    table = s["table"].tolist()
    powers = torch.tensor([2.0 ** e for e in range(E_MIN, 128)], dtype=torch.float64, device="cuda")
    got = {}
    for name in ("k", "v"):
        pages, scale = s[name + "_pages"].double(), s[name + "_scale"].double()
        x = s[name + "_new"].double()
        at = [(b, c) for b in range(s["B"]) for c in range(ctx[b], ctx[b] + cu[b + 1] - cu[b])]
        if name == "k" and s["inv_freq"] is not None:
            x = _exact_turn(x, torch.tensor([c for _, c in at], device="cuda"), s["inv_freq"], 0, s["inter"], 1.0, 1.0)
        pieces = []                                      # (page, its first new slot, first token, last token)
        for b in range(s["B"]):
            c, i, end = ctx[b], cu[b], cu[b + 1]
            while i < end:
                k = min(end - i, page - c % page)
                pieces.append((table[b][c // page], c % page, i, i + k))
                i, c = i + k, c + k
        big = x.abs().amax(-1)
        for p, slot, i, j in pieces:
            most = big[i:j].amax(0)
            new = powers[(most[:, None] > FMT[fmt][1] * powers).sum(1)]
            if slot:
                new = torch.maximum(new, scale[p])
                pages[p, :slot] = _exact_round(pages[p, :slot] * (scale[p] / new)[:, None], fmt)
            scale[p] = new
            pages[p, slot:slot + j - i] = _exact_round(x[i:j] / new[:, None], fmt)
        got[name], got[name + "_scale"] = (pages if fmt == "e4m3" else pages.to(torch.int8)), scale
    return got


def _exact_attn(s):
    t, hq, d = s["q"].shape
    page, g = s["page"], hq // s["Hkv"]
    out = torch.zeros((t, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64, device="cuda")
    n = s["n_keys"].tolist()
    raw = [s[x + "_pages"].view(torch.uint8) for x in "kv"]
    for r in range(t):
        b = r if s["seq"] is None else r // s["rows"]
        pos = torch.arange(n[r], device="cuda")
        if s["idx"] is not None:
            pos = s["idx"][r][s["idx"][r] >= 0].long()
        if not len(pos):
            continue
        p = s["table"][b].long()[pos // page]
        k, v = (x[p, pos % page].view(s["k_pages"].dtype).double() * y[p].double()[..., None]
                for x, y in zip(raw, (s["k_scale"], s["v_scale"])))
        q = s["q"][r].double().reshape(-1, g, d)
        z = torch.matmul(q, k.permute(1, 2, 0)) * s["scale"]
        lse[r] = torch.logsumexp(z, -1).flatten()
        out[r] = torch.matmul(torch.softmax(z, -1), v.transpose(0, 1)).reshape(hq, d)
    return {"out": out, "lse": lse}
