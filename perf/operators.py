"""The operators of the 8-bit paged KV cache: what is measured, their plain forms and their values in 64 bits.

The cache holds K and V as E4M3 codes in pages [n_pages, Hkv, page, 128] with one FP32 scale per (page, KV head):

* write: new BF16 rows go into the pages.  A value is rounded to 4 significant bits (q4); the scale of a (page, head)
  is 2^e, e = max(-120, floor(log2 max |q4|) - 7) over the page's tokens so far; the code is q4 / 2^e, or 0 where that
  is under 2^-6.  When the scale of a partly filled page grows, its earlier codes are brought to the new scale.
* read: ranges of tokens come back as packed BF16 rows.
* decode: one query token a sequence attends to its cached tokens.
"""
import math

import torch

own = False

D = 128
THETA = 1.0e6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch appends one token a sequence, mostly into partly filled pages
        dict(name="write step 64", op="write", seqs=64, lo=500, hi=4000, new_lo=1, new_hi=1, hq=32, hkv=8, page=16, rope=False),
        # chunks of several prompts over caches that end inside a page, the keys rotated on the way
        dict(name="write chunks rope", op="write", seqs=5, lo=0, hi=3001, new_lo=333, new_hi=2048, hq=32, hkv=8, page=16, rope=True),
        # whole long prompts of the tensor-parallel half of the heads
        dict(name="write prompts", op="write", seqs=4, lo=0, hi=0, new_lo=30011, new_hi=32768, hq=16, hkv=4, page=64, rope=False),
        # a few tokens of one sequence come back
        dict(name="read 77", op="read", seqs=1, lo=900, hi=900, new_lo=77, new_hi=77, hq=32, hkv=8, page=16, rope=False),
        # the caches that the next chunks of a chunked prefill attend to
        dict(name="read prompts", op="read", seqs=4, lo=0, hi=0, new_lo=20000, new_hi=32768, hq=32, hkv=8, page=16, rope=False),
        # one short conversation: latency
        dict(name="decode 1 x 700", op="decode", seqs=1, lo=700, hi=700, hq=32, hkv=8, page=16, rope=False),
        # a serving batch, contexts over the whole range
        dict(name="decode 64 mixed", op="decode", seqs=64, lo=512, hi=32768, hq=32, hkv=8, page=16, rope=False),
        # few long sequences: the cache of each is split over many SMs
        dict(name="decode 4 x 32768", op="decode", seqs=4, lo=32768, hi=32768, hq=32, hkv=8, page=16, rope=False),
        # a small batch of the tensor-parallel half of the heads, the query rotated in the call
        dict(name="decode 8 rope", op="decode", seqs=8, lo=1, hi=9001, hq=16, hkv=4, page=64, rope=True),
        # more sequences than one launch's tables hold, groups of five, large pages
        dict(name="decode 200 short", op="decode", seqs=200, lo=33, hi=2500, hq=40, hkv=8, page=128, rope=False),
    ]


HEADS = [(32, 8), (16, 4), (8, 8), (32, 4), (24, 8), (40, 8), (4, 1), (8, 1)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    hq, hkv = rng.choice(HEADS)
    c = dict(op=rng.choice(["write", "read", "decode", "decode"]), hq=hq, hkv=hkv, page=rng.choice([8, 16, 32, 64, 128]),
             rope=rng.random() < 0.4)
    c["seqs"] = _log(rng, 1, 200)
    if c["op"] == "decode":
        most = max(1, min(32768, 64 * 16640 * 8 // (c["seqs"] * hkv)))
        c["hi"] = _log(rng, 1, most)
        c["lo"] = rng.randint(1, c["hi"])
    else:
        most = max(1, min(32768, 4 * 26000 * 8 // (c["seqs"] * hkv)))
        c["new_hi"] = _log(rng, 1, most)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["hi"] = rng.randint(0, max(0, min(4000, 300000 // c["seqs"])))
        c["lo"] = rng.randint(0, c["hi"])
        c["rope"] = c["rope"] and c["op"] == "write"
    return c


def _spread(lo, hi, n):
    """n lengths over [lo, hi], both ends among them, in a mixed order."""
    step = next(s for s in (7, 11, 13, 17) if math.gcd(s, n) == 1)
    return [hi - (hi - lo) * ((i * step) % n) // max(n - 1, 1) for i in range(n)]


def _lengths(case):
    """(tokens before, tokens of the call) of each sequence; decode: (0, context)."""
    n = case["seqs"]
    ctx = _spread(case["lo"], case["hi"], n)
    if case["op"] == "decode":
        return [0] * n, ctx
    return ctx, _spread(case["new_lo"], case["new_hi"], n)


def work(case):
    pos, new = _lengths(case)
    hq, hkv, ps, n = case["hq"], case["hkv"], case["page"], case["seqs"]
    t = sum(new)
    pages = sum(-(-(p + m) // ps) - p // ps for p, m in zip(pos, new))
    codes = 2 * t * hkv * D + 2 * pages * hkv * 4 + pages * 4
    table = D * 4 * (max(p + m for p, m in zip(pos, new)) if case["op"] == "write" else n) if case["rope"] else 0
    if case["op"] == "decode":
        return {"bytes": codes + table + n * hq * (D * (2 + 4 + 2) + 4), "flops": 4 * hq * D * t}
    return {"bytes": codes + table + 2 * t * hkv * D * 2, "flops": 2 * t * hkv * D * 8}


# ------------------------------------------------------------------ inputs

def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 16 + k)


def _two(e):
    """2^e for whole numbers e of -126 .. 127, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _rows(shape, seed, k, gain):
    """Normal rows whose channels differ in size, a few of them large, as keys and queries have them."""
    x = torch.randn(shape, generator=_gen(seed, k), device="cuda", dtype=torch.float32)
    if gain:
        g = torch.rand(shape[-2:], generator=_gen(7, k), device="cuda") * 0.7 + 0.3
        g = torch.where(torch.rand(shape[-2:], generator=_gen(8, k), device="cuda") < 0.03, g * 6, g)
        x = x * g
    return x.to(torch.bfloat16)


def _pool(shape, seed, k, valid, gain):
    """Pages as write leaves them: codes (NaN in the slots no token has, as a buffer that was used before can have) and scales."""
    n_pages, hkv = shape[:2]
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty((n_pages, hkv), dtype=torch.float32, device="cuda")
    some = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    g = _gen(seed, k)
    ch = torch.rand((hkv, 1, D), generator=_gen(9, k), device="cuda") * 0.7 + 0.3
    if gain:
        ch = torch.where(torch.rand(ch.shape, generator=_gen(10, k), device="cuda") < 0.03, ch * 6, ch)
    slot = torch.arange(shape[2], device="cuda")
    for a in range(0, n_pages, some):
        b = min(n_pages, a + some)
        x = torch.randn((b - a,) + tuple(shape[1:]), generator=g, device="cuda") * ch
        fill = slot[None, None, :, None] >= valid[a:b, None, None, None]
        x.masked_fill_(fill, 0.0)
        top = x.abs().amax((2, 3)).clamp_min(1e-30)
        s = _two(torch.frexp(top)[1] - 8)
        c = x / s[:, :, None, None]
        c = torch.where(c.abs() < 2.0 ** -6, torch.zeros_like(c), c).clamp_(-240, 240).to(torch.float8_e4m3fn)
        codes[a:b] = c.view(torch.uint8).masked_fill_(fill, 0x7F)
        scales[a:b] = s
    return codes, scales


def _table(n):
    i = torch.arange(64, dtype=torch.float64)
    a = torch.arange(n, dtype=torch.float64)[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64), -2.0 * i / D)[None, :]
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32).cuda()


def prepare(case, seed):
    pos, new = _lengths(case)
    n, hkv, hq, ps = case["seqs"], case["hkv"], case["hq"], case["page"]
    pages = [-(-(p + m) // ps) for p, m in zip(pos, new)]
    n_pages, max_pages = sum(pages) + 3, max(pages)
    cpu = torch.Generator().manual_seed(int(seed))
    perm = torch.randperm(n_pages, generator=cpu, dtype=torch.int32)
    first = torch.tensor([0] + pages).cumsum(0)[:-1]
    count = torch.tensor(pages)
    col = torch.arange(max_pages)
    table = torch.where(col[None, :] < count[:, None], perm[(first[:, None] + col[None, :]).clamp_max(n_pages - 1)], torch.tensor(-1, dtype=torch.int32))
    held = torch.tensor(pos if case["op"] == "write" else [p + m for p, m in zip(pos, new)])
    valid = torch.zeros(n_pages, dtype=torch.int64)
    inside = col[None, :] < count[:, None]
    valid[table[inside].long()] = (held[:, None] - col[None, :] * ps).clamp(0, ps)[inside]
    s = {"case": dict(case), "pos": pos, "new": new, "n_pages": n_pages, "max_pages": max_pages, "table": table.cuda(), "ps": ps, "hq": hq, "hkv": hkv, "n": n}
    valid = valid.cuda()
    s["k"], s["ks"] = _pool((n_pages, hkv, ps, D), seed, 1, valid, True)
    s["v"], s["vs"] = _pool((n_pages, hkv, ps, D), seed, 2, valid, False)
    s["rope"] = _table(max(p + m for p, m in zip(pos, new))) if case["rope"] else None
    total = sum(new)
    if case["op"] == "decode":
        s["q"] = _rows((n, hq, D), seed, 3, True)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty((n, hq, D), dtype=torch.float32, device="cuda")
        s["out_bf16"] = torch.empty((n, hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((n, hq), dtype=torch.float32, device="cuda")
        blocks = sum(-(-c // 128) for c in new)
        s["workspace"] = torch.empty(blocks * hq * 516 + 256 + n * hkv * 512, dtype=torch.uint8, device="cuda")
    elif case["op"] == "write":
        s["new_k"], s["new_v"] = _rows((total, hkv, D), seed, 4, True), _rows((total, hkv, D), seed, 5, False)
    else:
        s["out_k"], s["out_v"] = (torch.empty((total, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s["cu"] = [0]
    for m in new:
        s["cu"].append(s["cu"][-1] + m)
    return s


# ------------------------------------------------------------------ the operators, plainly

def _tokens(s):
    """(sequence, position) of every token of the call."""
    new = torch.tensor(s["new"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), new)
    start = torch.tensor(s["cu"][:-1], device="cuda")
    return seq, torch.arange(s["cu"][-1], device="cuda") - start[seq] + torch.tensor(s["pos"], device="cuda")[seq]


def _rotated(x, rope, at):
    """Rows turned by the angles of their positions: products rounded to FP32, sums in 64 bits, the row rounded to BF16."""
    c, z = rope[at, None, :64], rope[at, None, 64:]
    a, b = x[..., :64].float(), x[..., 64:].float()
    return torch.cat([a.double() * c.double() - (b * z).double(), b.double() * c.double() + (a * z).double()], -1).float().to(torch.bfloat16)


def _q4(x):
    """Rounded to 4 significant bits, ties to even; under the smallest normal number it is 0."""
    m, e = torch.frexp(x.float())
    return torch.where(x.abs() < 2.0 ** -126, torch.zeros_like(m), torch.round(m * 16) * 0.125 * _two(e - 1))


def _into(s, new, codes, scales, page, slot, before):
    """The rows `new` into their pages, of which the first `before` slots were filled: each touched page as a whole."""
    touched, which = torch.unique(page, return_inverse=True)
    before = torch.zeros(touched.numel(), dtype=torch.int64, device="cuda").index_put_((which,), before)
    old = torch.arange(s["ps"], device="cuda")[None, :] < before[:, None]
    fresh = torch.zeros_like(old).index_put_((which, slot), torch.ones_like(old[0, 0]))
    had = codes[touched].view(torch.float8_e4m3fn).float() * scales[touched][:, :, None, None]
    vals = torch.where(old[:, None, :, None], had, torch.zeros_like(had))
    vals = vals.transpose(1, 2).index_put_((which, slot), _q4(new)).transpose(1, 2)
    top = vals.abs().amax((2, 3))
    scale = _two(torch.where(top > 0, torch.frexp(top)[1] - 8, -120).clamp_min(-120))
    scale = torch.where(before[:, None] > 0, torch.maximum(scale, scales[touched]), scale)
    code = vals / scale[:, :, None, None]
    code = torch.where(code.abs() < 2.0 ** -6, torch.zeros_like(code), code).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[touched] = torch.where((old | fresh)[:, None, :, None], code, codes[touched])
    scales[touched] = scale


def _write(s):
    seq, at = _tokens(s)
    page, slot = s["table"][seq, at // s["ps"]].long(), at % s["ps"]
    before = (torch.tensor(s["pos"], device="cuda")[seq] - (at - slot)).clamp(0, s["ps"])
    _into(s, s["new_k"] if s["rope"] is None else _rotated(s["new_k"], s["rope"], at), s["k"], s["ks"], page, slot, before)
    _into(s, s["new_v"], s["v"], s["vs"], page, slot, before)
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_scale": s["ks"], "v_scale": s["vs"]}


def _read(s):
    seq, at = _tokens(s)
    page, slot = s["table"][seq, at // s["ps"]].long(), at % s["ps"]

    def rows(codes, scales):
        return (codes[page, :, slot].view(torch.float8_e4m3fn).float() * scales[page][:, :, None]).to(torch.bfloat16)

    return {"k": rows(s["k"], s["ks"]), "v": rows(s["v"], s["vs"])}


def _decode(s):
    n, hkv, ps = s["n"], s["hkv"], s["ps"]
    ctx = torch.tensor(s["new"], device="cuda")
    q = s["q"] if s["rope"] is None else _rotated(s["q"], s["rope"], ctx - 1)
    q = q.float().view(n, hkv, s["hq"] // hkv, D)
    page = s["table"].long().clamp_min(0)
    hidden = (torch.arange(s["max_pages"] * ps, device="cuda")[None, :] >= ctx[:, None])[:, None, :, None]

    def cached(codes, scales):
        x = codes[page].view(torch.float8_e4m3fn).float() * scales[page][..., None, None]
        return x.transpose(1, 2).reshape(n, hkv, -1, D).masked_fill_(hidden, 0.0)

    x = (q @ cached(s["k"], s["ks"]).transpose(2, 3) * s["scale"]).masked_fill_(hidden.transpose(2, 3), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    out = ((p @ cached(s["v"], s["vs"])) / l).reshape(n, s["hq"], D)
    return {"out": out, "out_bf16": out.to(torch.bfloat16), "lse": (m + torch.log(l)).reshape(n, s["hq"])}


def _own(s):
    import deterministic_context_attention_gb300 as rlk

    params = rlk.make_params(s["n"], s["hq"], s["hkv"], 128)
    pool = (s["k"], s["v"], s["ks"], s["vs"], s["n_pages"], s["ps"], s["table"], s["max_pages"])
    top = 0 if s["rope"] is None else s["rope"].shape[0]
    if s["case"]["op"] == "write":
        rlk.rlk_attn_qcache_write(params, s["new_k"], s["new_v"], s["cu"], s["pos"], s["rope"], top, *pool)
        return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_scale": s["ks"], "v_scale": s["vs"]}
    if s["case"]["op"] == "read":
        rlk.rlk_attn_qcache_read(params, *pool, s["cu"], s["pos"], s["out_k"], s["out_v"])
        return {"k": s["out_k"], "v": s["out_v"]}
    rlk.rlk_attn_decode_qcache(params, s["q"], *pool, s["new"], 0, s["rope"], top, s["out"], s["out_bf16"], s["lse"], s["workspace"])
    return {"out": s["out"], "out_bf16": s["out_bf16"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"write": _write, "read": _read, "decode": _decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------ their values in 64 bits

def _exact_rows(x, rope, at):
    if rope is None:
        return x.double()
    x, t = x.double(), rope.double()[at]
    out = torch.empty_like(x)
    for i in range(64):
        c, z = t[:, None, i], t[:, None, 64 + i]
        out[..., i] = x[..., i] * c - (x[..., 64 + i] * z).float().double()
        out[..., 64 + i] = x[..., 64 + i] * c + (x[..., i] * z).float().double()
    return out.float().to(torch.bfloat16).double()


def exact(case, seed):
    s = prepare(case, seed)
    ps, ks = s["ps"], (("k", s["k"], s["ks"]), ("v", s["v"], s["vs"]))
    worth = torch.arange(256, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn).double()
    if case["op"] == "write":
        got = {}
        for name, codes, scales in ks:
            value, scale = worth[codes.long()] if codes.numel() < 1 << 30 else None, scales.double()
            if value is None:
                return None
            for b in range(s["n"]):
                p0, m, c0 = s["pos"][b], s["new"][b], s["cu"][b]
                x = s["new_" + name][c0:c0 + m]
                x = _exact_rows(x, s["rope"] if name == "k" else None, torch.arange(p0, p0 + m, device="cuda"))
                # 4 significant bits: a whole number of steps of 2^(floor(log2 |x|) - 3)
                step = ((torch.frexp(x.abs().clamp_min(2.0 ** -126))[1].long() - 4 + 1023) << 52).view(torch.float64)
                x = torch.round(x / step) * step
                # the first page, partly filled before, and then whole pages
                a = 0
                head = min(m, (ps - p0 % ps) % ps)
                spans = ([(0, head)] if head else []) + ([(head, m)] if m > head else [])
                for a, z in spans:
                    first, used = (p0 + a) // ps, (p0 + a) % ps
                    count = -(-(used + z - a) // ps)
                    page = s["table"][b, first:first + count].long()
                    block = torch.zeros((count * ps, s["hkv"], D), dtype=torch.float64, device="cuda")
                    if used:
                        block[:used] = (value[page[0], :, :used] * scale[page[0]][:, None, None]).transpose(0, 1)
                    block[used:used + z - a] = x[a:z]
                    block = block.view(count, ps, s["hkv"], D).transpose(1, 2)
                    top = block.abs().amax((2, 3))
                    sc = ((torch.frexp(top.clamp_min(2.0 ** -140))[1].long() - 8 + 1023) << 52).view(torch.float64).clamp_min(2.0 ** -120)
                    if used:
                        sc = torch.maximum(sc, scale[page])
                    code = block / sc[:, :, None, None]
                    code[code.abs() < 2.0 ** -6] = 0.0
                    held = (torch.arange(count * ps, device="cuda") < used + z - a).view(count, 1, ps, 1)
                    value[page] = torch.where(held, code, value[page])
                    scale[page] = sc
            got[name], got[name + "_scale"] = value, scale
        return got
    if case["op"] == "read":
        got = {}
        for name, codes, scales in ks:
            rows = []
            for b in range(s["n"]):
                at = torch.arange(s["pos"][b], s["pos"][b] + s["new"][b], device="cuda")
                page = s["table"][b].long()[at // ps]
                rows.append(worth[codes[page, :, at % ps].long()] * scales[page].double()[:, :, None])
            got[name] = torch.cat(rows)
        return got
    out, lse, g = [], [], s["hq"] // s["hkv"]
    for b in range(s["n"]):
        c = s["new"][b]
        page = s["table"][b, : -(-c // ps)].long()
        k, v = ((worth[codes[page].long()] * scales[page].double()[:, :, None, None]).transpose(0, 1).reshape(s["hkv"], -1, D)[:, :c] for _, codes, scales in ks)
        q = _exact_rows(s["q"][b:b + 1], s["rope"], torch.tensor([c - 1], device="cuda"))[0].view(s["hkv"], g, D)
        x = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
        z = torch.logsumexp(x, -1)
        lse.append(z.reshape(-1))
        out.append(torch.matmul(torch.exp(x - z[..., None]), v).reshape(-1, D))
    out = torch.stack(out)
    return {"out": out, "out_bf16": out, "lse": torch.stack(lse)}
