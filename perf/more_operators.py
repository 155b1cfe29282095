"""Differential attention and the paged BF16 cache it reads: what is measured, the plain forms and the values in 64 bits.

* append: new K and V rows go into the pages, K rotated by its positions on the way; the queries of the same tokens and a
  packed copy of the rotated keys come along where asked. The rotation's pairs are (i, i + 64) of the 128 elements, or
  (i, i + 32) of each half (width 64).
* prefill: out = softmax(s q1 k1^T) v - lam softmax(s q2 k2^T) v, causal, where q1 and k1 are the first 64 elements of a
  head, q2 and k2 the others, and lam is learned, one weight a query head.
* backward: the gradients of q, k, v and lam.
* decode: one query token a sequence over the pages.
"""
import math

import torch

own = False

D = 128
M = 64  # width of a map
SCALE = 1.0 / 8.0
THETA = 1.0e6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: a token a sequence into its partly filled page, its query rotated beside it
        dict(name="append step 64", op="append", seqs=64, lo=500, hi=4000, new_lo=1, new_hi=1, hq=32, hkv=8, page=16, width=128, queries=True),
        # chunks of prompts on their way to the differential prefill, which wants the rotated keys packed too
        dict(name="append chunks maps", op="append", seqs=5, lo=0, hi=3001, new_lo=333, new_hi=2048, hq=32, hkv=8, page=16, width=64, queries=True),
        # whole long prompts whose keys were rotated before: K and V alone
        dict(name="append prompts", op="append", seqs=4, lo=0, hi=0, new_lo=20011, new_hi=32768, hq=32, hkv=8, page=64, width=0, queries=False),
        # the shortest prompt: latency
        dict(name="prefill 1 x 77", op="prefill", seqs=1, lo=77, hi=77, new_lo=77, new_hi=77, hq=32, hkv=8, train=False),
        # a varlen training batch, which keeps what the backward pass reads
        dict(name="prefill varlen", op="prefill", seqs=4, lo=777, hi=4096, new_lo=777, new_hi=4096, hq=32, hkv=8, train=True),
        # a chunk of 512 queries against the growing cache, the tensor-parallel half of the heads
        dict(name="prefill chunk", op="prefill", seqs=2, lo=7000, hi=8192, new_lo=512, new_hi=512, hq=16, hkv=4, train=False),
        # a training batch
        dict(name="backward 2 x 4096", op="backward", seqs=2, lo=4096, hi=4096, hq=32, hkv=8),
        # short ragged sequences, five query heads a KV head
        dict(name="backward ragged", op="backward", seqs=7, lo=5, hi=1201, hq=40, hkv=8),
        # one short conversation: latency
        dict(name="decode 1 x 700", op="decode", seqs=1, lo=700, hi=700, hq=32, hkv=8, page=16),
        # a serving batch, contexts over the whole range
        dict(name="decode 64 mixed", op="decode", seqs=64, lo=512, hi=32768, hq=32, hkv=8, page=16),
        # few long sequences: the cache of each is split over many SMs
        dict(name="decode 4 x 32768", op="decode", seqs=4, lo=32768, hi=32768, hq=32, hkv=8, page=16),
        # many short ones in large pages, groups of eight
        dict(name="decode 150 short", op="decode", seqs=150, lo=33, hi=2500, hq=32, hkv=4, page=64),
    ]


HEADS = [(32, 8), (16, 4), (8, 8), (32, 4), (24, 8), (40, 8), (4, 1), (8, 1)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    hq, hkv = rng.choice(HEADS)
    c = dict(op=rng.choice(["append", "prefill", "backward", "decode"]), hq=hq, hkv=hkv)
    if c["op"] == "append":
        c["page"], c["width"] = rng.choice([8, 16, 32, 64, 128]), rng.choice([0, 64, 128])
        c["seqs"] = _log(rng, 1, 200)
        c["queries"] = c["width"] > 0 and rng.random() < 0.6
        rows = 2 * hkv + (hq + hkv if c["queries"] else 0)
        c["new_hi"] = _log(rng, 1, max(1, min(32768, 4 * 26000 * 16 // (c["seqs"] * rows))))
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["hi"] = rng.randint(0, max(0, min(4000, 300000 // c["seqs"])))
        c["lo"] = rng.randint(0, c["hi"])
    elif c["op"] == "decode":
        c["page"] = rng.choice([8, 16, 32, 64, 128])
        c["seqs"] = _log(rng, 1, 200)
        c["hi"] = _log(rng, 1, max(1, min(32768, 64 * 16640 * 8 // (c["seqs"] * hkv))))
        c["lo"] = rng.randint(1, c["hi"])
    else:
        c["seqs"] = _log(rng, 1, 12)
        area = (32 * 24_000_000 if c["op"] == "prefill" else 32 * 30_000_000) // (hq * c["seqs"])
        # (the gradients of q and k of sequences of one token are zero: rounding alone is no value to compare)
        c["hi"] = _log(rng, 2 if c["op"] == "backward" else 1, min(8192, math.isqrt(area)))
        c["lo"] = rng.randint(1, c["hi"])
        if c["op"] == "prefill":
            c["train"] = rng.random() < 0.5
            # whole sequences, or their last tokens
            c["new_hi"] = c["hi"] if rng.random() < 0.5 else rng.randint(1, c["lo"])
            c["new_lo"] = c["lo"] if c["new_hi"] == c["hi"] else rng.randint(1, c["new_hi"])
    return c


def _spread(lo, hi, n):
    """n lengths over [lo, hi], both ends among them, in a mixed order."""
    step = next(s for s in (7, 11, 13, 17) if math.gcd(s, n) == 1)
    return [hi - (hi - lo) * ((i * step) % n) // max(n - 1, 1) for i in range(n)]


def _lengths(case):
    """append: (tokens before, tokens of the call) of each sequence; otherwise (queries, keys)."""
    n = case["seqs"]
    keys = _spread(case["lo"], case["hi"], n)
    if case["op"] == "append":
        return keys, _spread(case["new_lo"], case["new_hi"], n)
    if case["op"] == "prefill":
        return _spread(case["new_lo"], case["new_hi"], n), keys
    return ([1] * n if case["op"] == "decode" else keys), keys


def work(case):
    a, b = _lengths(case)
    hq, hkv, n = case["hq"], case["hkv"], case["seqs"]
    if case["op"] == "append":
        t, ps = sum(b), case["page"]
        rows = 4 * hkv + (2 * hq + hkv if case["queries"] else 0)
        ids = sum(-(-(p + m) // ps) - p // ps for p, m in zip(a, b))
        table = max(p + m for p, m in zip(a, b)) if n * 4 < t else t
        return {"bytes": t * rows * D * 2 + ids * 4 + (table * (D if case["width"] == 128 else M) * 4 if case["width"] else 0),
                "flops": t * (hkv + (hq if case["queries"] else 0)) * D * 3 if case["width"] else t}
    if case["op"] == "decode":
        ps = case["page"]
        return {"bytes": sum(b) * hkv * 2 * D * 2 + sum(-(-c // ps) for c in b) * 4 + n * hq * (D * (2 + 4 + 2) + 8),
                "flops": sum(b) * hq * 6 * D}
    seen = sum(q * k - q * (q - 1) // 2 for q, k in zip(a, b))  # (query, key) pairs under the mask
    tq, tk = sum(a), sum(b)
    if case["op"] == "prefill":
        out = tq * hq * (2 * D * 4 + 8) if case["train"] else tq * hq * D * 2
        return {"bytes": tq * hq * D * 2 + 2 * tk * hkv * D * 2 + out, "flops": seen * hq * 6 * D}
    return {"bytes": tq * hq * (2 * D * 2 + 2 * D * 4 + 8) + 2 * tk * hkv * D * 2 + (tq * hq + 2 * tk * hkv) * D * 4,
            "flops": seen * hq * 10 * D}


# ------------------------------------------------------------------ inputs

def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 16 + k)


def _rows(shape, seed, k, gain):
    """Normal rows whose channels differ in size, a few of them large, as keys and queries have them."""
    x = torch.randn(shape, generator=_gen(seed, k), device="cuda", dtype=torch.float32)
    if gain:
        g = torch.rand(shape[-2:], generator=_gen(7, k), device="cuda") * 0.7 + 0.3
        g = torch.where(torch.rand(shape[-2:], generator=_gen(8, k), device="cuda") < 0.03, g * 6, g)
        x = x * g
    return x.to(torch.bfloat16)


def _table(n):
    i = torch.arange(64, dtype=torch.float64)
    a = torch.arange(n, dtype=torch.float64)[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64), -2.0 * i / D)[None, :]
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32).cuda()


def _cu(lengths):
    c = [0]
    for m in lengths:
        c.append(c[-1] + m)
    return c


def _pages(s, tokens, seed, gain_k):
    """Pages in a scattered order, their unused slots NaN as in a buffer that was used before."""
    case, ps, hkv, n = s["case"], s["case"]["page"], s["case"]["hkv"], s["case"]["seqs"]
    pages = [-(-t // ps) for t in tokens]
    s["n_pages"], s["max_pages"] = sum(pages) + 3, max(pages)
    perm = torch.randperm(s["n_pages"], generator=torch.Generator().manual_seed(int(seed)), dtype=torch.int32)
    first, count, col = torch.tensor([0] + pages).cumsum(0)[:-1], torch.tensor(pages), torch.arange(s["max_pages"])
    inside = col[None, :] < count[:, None]
    table = torch.where(inside, perm[(first[:, None] + col[None, :]).clamp_max(s["n_pages"] - 1)], torch.tensor(-1, dtype=torch.int32))
    held = torch.zeros(s["n_pages"], dtype=torch.int64)
    held[table[inside].long()] = (torch.tensor(s["held"])[:, None] - col[None, :] * ps).clamp(0, ps)[inside]
    s["table"] = table.cuda()
    unused = (torch.arange(ps)[None, :] >= held[:, None]).cuda()[:, :, None, None]
    for name, k, gain in (("k_pool", 1, gain_k), ("v_pool", 2, False)):
        s[name] = _rows((s["n_pages"], ps, hkv, D), seed, k, gain).masked_fill_(unused, math.nan)


def prepare(case, seed):
    a, b = _lengths(case)
    n, hq, hkv = case["seqs"], case["hq"], case["hkv"]
    s = {"case": dict(case), "n": n, "a": a, "b": b, "scale": SCALE}
    f32, bf16 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
    if case["op"] == "append":
        s["held"], s["cu"] = a, _cu(b)
        t = s["cu"][-1]
        _pages(s, [p + m for p, m in zip(a, b)], seed, True)
        s["k"], s["v"] = _rows((t, hkv, D), seed, 4, True), _rows((t, hkv, D), seed, 5, False)
        s["rope"] = _table(max(p + m for p, m in zip(a, b))) if case["width"] else None
        s["q"] = _rows((t, hq, D), seed, 3, True) if case["queries"] else None
        s["q_out"] = torch.empty((t, hq, D), **bf16) if case["queries"] else None
        s["k_out"] = torch.empty((t, hkv, D), **bf16) if case["queries"] else None
        return s
    s["lam"] = 0.5 + 0.3 * torch.randn(hq, generator=_gen(seed, 6), device="cuda", dtype=torch.float32)
    if case["op"] == "decode":
        s["held"] = b
        _pages(s, b, seed, True)
        s["q"] = _rows((n, hq, D), seed, 3, True)
        s["out"], s["out_bf16"], s["lse"] = torch.empty((n, hq, D), **f32), torch.empty((n, hq, D), **bf16), torch.empty((n, hq, 2), **f32)
        blocks = sum(-(-c // 128) for c in b)
        s["workspace"] = torch.empty(blocks * hq * 2 * 516 + 256 + n * hkv * 512, dtype=torch.uint8, device="cuda")
        return s
    s["cu_q"], s["cu_k"] = _cu(a), _cu(b)
    tq, tk = s["cu_q"][-1], s["cu_k"][-1]
    s["q"], s["k"], s["v"] = _rows((tq, hq, D), seed, 3, True), _rows((tk, hkv, D), seed, 4, True), _rows((tk, hkv, D), seed, 5, False)
    if case["op"] == "prefill":
        s["out"] = torch.empty((tq, hq, D), **f32) if case["train"] else None
        s["out2"] = torch.empty((tq, hq, D), **f32) if case["train"] else None
        s["lse"] = torch.empty((tq, hq, 2), **f32) if case["train"] else None
        s["out_bf16"] = None if case["train"] else torch.empty((tq, hq, D), **bf16)
        return s
    # what the forward pass of the same batch left
    parts = [_sequence(s, i) for i in range(n)]
    s["out"], s["out2"], s["lse"] = (torch.cat([p[j] for p in parts]) for j in range(3))
    s["dout"] = _rows((tq, hq, D), seed, 9, False)
    s["dq"], s["dk"], s["dv"] = torch.empty((tq, hq, D), **f32), torch.empty((tk, hkv, D), **f32), torch.empty((tk, hkv, D), **f32)
    s["dlam"] = torch.empty(hq, **f32)
    s["workspace"] = torch.empty((tq + 128) * hq * 16 + 256, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the operators, plainly

def _rotated(x, rope, at, width):
    """Rows turned by the angles of their positions: products rounded to FP32, sums in 64 bits, the row rounded to BF16."""
    step, h = D // width, width // 2
    c, z = rope[at, None, None, :64:step], rope[at, None, None, 64::step]
    x = x.view(x.shape[0], x.shape[1], step, width)
    a, b = x[..., :h].float(), x[..., h:].float()
    y = torch.cat([a.double() * c.double() - (b * z).double(), b.double() * c.double() + (a * z).double()], -1)
    return y.float().to(torch.bfloat16).view(x.shape[0], -1, D)


def _append(s):
    ps, width = s["case"]["page"], s["case"]["width"]
    new = torch.tensor(s["b"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), new)
    start, before = torch.tensor(s["cu"][:-1], device="cuda"), torch.tensor(s["a"], device="cuda")
    at = torch.arange(s["cu"][-1], device="cuda") - start[seq] + before[seq]
    page, slot = s["table"][seq, at // ps].long(), at % ps
    k = _rotated(s["k"], s["rope"], at, width) if width else s["k"]
    s["k_pool"][page, slot] = k
    s["v_pool"][page, slot] = s["v"]
    got = {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    return got | {"q_out": _rotated(s["q"], s["rope"], at, width), "k_out": k} if s["case"]["queries"] else got


def _maps(q, k, scale):
    """Weights under the causal mask and their log sums of one sequence: q [ql, Hq, 128], k [kl, Hkv, 128] -> two [Hkv, G, ql, kl], two [Hkv, G, ql, 1]."""
    ql, kl, hkv = q.shape[0], k.shape[0], k.shape[1]
    q = q.float().view(ql, hkv, -1, 2, M).permute(3, 1, 2, 0, 4)
    k = k.float().view(kl, hkv, 2, M).permute(2, 1, 3, 0)
    hidden = torch.arange(kl, device=q.device)[None, :] > torch.arange(kl - ql, kl, device=q.device)[:, None]

    def one(m):
        x = torch.matmul(q[m], k[m][:, None]).mul_(scale).masked_fill_(hidden, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        return p.div_(total), top + torch.log(total)

    return one(0), one(1)


def _sequence(s, i):
    """out, the second map's output and both log sums of sequence i, in 32 bits."""
    q, k, v = s["q"][s["cu_q"][i]:s["cu_q"][i + 1]], s["k"][s["cu_k"][i]:s["cu_k"][i + 1]], s["v"][s["cu_k"][i]:s["cu_k"][i + 1]]
    (p1, l1), (p2, l2) = _maps(q, k, s["scale"])
    v = v.float().permute(1, 0, 2)[:, None]
    back = lambda x: x.permute(2, 0, 1, 3).reshape(q.shape[0], q.shape[1], -1)  # noqa: E731
    o2 = back(torch.matmul(p2, v))
    return back(torch.matmul(p1, v)) - s["lam"][:, None] * o2, o2, back(torch.cat([l1, l2], -1))


def _prefill(s):
    parts = [_sequence(s, i) for i in range(s["n"])]
    out, out2, lse = (torch.cat([p[j] for p in parts]) for j in range(3))
    return {"out": out, "out2": out2, "lse": lse} if s["case"]["train"] else {"out_bf16": out.to(torch.bfloat16)}


def _sequence_backward(s, i):
    rows = slice(s["cu_q"][i], s["cu_q"][i + 1])
    n, hkv, hq = rows.stop - rows.start, s["case"]["hkv"], s["case"]["hq"]
    (p1, _), (p2, _) = _maps(s["q"][rows], s["k"][rows], s["scale"])
    heads = lambda x: x.float().view(n, hkv, hq // hkv, D).permute(1, 2, 0, 3)  # noqa: E731
    q, do = heads(s["q"][rows]), heads(s["dout"][rows])
    k, v = (s[x][rows].float().permute(1, 0, 2)[:, None] for x in ("k", "v"))
    lam = s["lam"].view(hkv, -1, 1, 1)
    d2 = (do * heads(s["out2"][rows])).sum(-1, keepdim=True)
    d1 = (do * heads(s["out"][rows])).sum(-1, keepdim=True) + lam * d2
    dv = torch.matmul((p1 - lam * p2).transpose(2, 3), do).sum(1)
    dp = torch.matmul(do, v.transpose(2, 3))
    s1 = p1.mul_(dp - d1)
    s2 = p2.mul_(dp - d2).mul_(-lam)
    dq = torch.cat([torch.matmul(s1, k[..., :M]), torch.matmul(s2, k[..., M:])], -1) * s["scale"]
    dk = torch.cat([torch.matmul(s1.transpose(2, 3), q[..., :M]).sum(1), torch.matmul(s2.transpose(2, 3), q[..., M:]).sum(1)], -1) * s["scale"]
    return dq.permute(2, 0, 1, 3).reshape(n, hq, D), dk.permute(1, 0, 2), dv.permute(1, 0, 2), -d2.double().sum((2, 3)).reshape(hq)


def _backward(s):
    parts = [_sequence_backward(s, i) for i in range(s["n"])]
    dq, dk, dv = (torch.cat([p[j] for p in parts]) for j in range(3))
    return {"dq": dq, "dk": dk, "dv": dv, "dlam": torch.stack([p[3] for p in parts]).sum(0).float()}


def _decode(s):
    n, hkv, hq, ps = s["n"], s["case"]["hkv"], s["case"]["hq"], s["case"]["page"]
    page = s["table"].long().clamp_min(0)
    hidden = (torch.arange(s["max_pages"] * ps, device="cuda")[None, :] >= torch.tensor(s["b"], device="cuda")[:, None])[:, None, None, :]
    cached = lambda x: x[page].reshape(n, -1, hkv, D).permute(0, 2, 1, 3).float().masked_fill_(hidden.transpose(2, 3), 0.0)  # noqa: E731
    k, v = cached(s["k_pool"]), cached(s["v_pool"])
    q = s["q"].float().view(n, hkv, hq // hkv, D)

    def one(m):
        at = slice(m * M, m * M + M)
        x = torch.matmul(q[..., at], k[..., at].transpose(2, 3)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        return (torch.matmul(p, v) / total).view(n, hq, D), (top + torch.log(total)).view(n, hq, 1)

    (o1, l1), (o2, l2) = one(0), one(1)
    out = o1 - s["lam"][:, None] * o2
    return {"out": out, "out_bf16": out.to(torch.bfloat16), "lse": torch.cat([l1, l2], -1)}


def _own(s):
    import deterministic_context_attention_gb300 as rlk

    c = s["case"]
    params = rlk.make_params(s["n"], c["hq"], c["hkv"], 128, softmax_scale=s["scale"])
    if c["op"] == "append":
        rlk.rlk_attn_cache_append(params, s["q"], s["q_out"], s["k"], s["k_out"], s["v"], s["cu"], s["a"], s["rope"],
                                  0 if s["rope"] is None else s["rope"].shape[0], c["width"] or 128, s["k_pool"], s["v_pool"],
                                  s["n_pages"], c["page"], s["table"], s["max_pages"])
        got = {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
        return got | {"q_out": s["q_out"], "k_out": s["k_out"]} if c["queries"] else got
    if c["op"] == "prefill":
        rlk.rlk_attn_diff_prefill(params, s["q"], s["k"], s["v"], s["lam"], s["cu_q"], s["cu_k"], -1, s["out"], s["out_bf16"], s["out2"], s["lse"])
        return {"out": s["out"], "out2": s["out2"], "lse": s["lse"]} if c["train"] else {"out_bf16": s["out_bf16"]}
    if c["op"] == "backward":
        rlk.rlk_attn_diff_backward(params, s["q"], s["k"], s["v"], s["lam"], s["out"], s["out2"], s["dout"], s["lse"], s["cu_q"], -1,
                                   s["dq"], s["dk"], s["dv"], s["dlam"], s["workspace"])
        return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"], "dlam": s["dlam"]}
    rlk.rlk_attn_diff_decode(params, s["q"], s["lam"], s["k_pool"], s["v_pool"], s["n_pages"], c["page"], s["table"], s["max_pages"],
                             s["b"], 0, s["out"], s["out_bf16"], s["lse"], s["workspace"])
    return {"out": s["out"], "out_bf16": s["out_bf16"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "prefill": _prefill, "backward": _backward, "decode": _decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------ their values in 64 bits

def _exact_append(s):
    ps, width = s["case"]["page"], s["case"]["width"]

    def turned(x, p0):
        y, n = x.double(), x.shape[0]
        if not width:
            return y
        out = y.clone()
        pos = torch.arange(p0, p0 + n, device="cuda")
        for i in range(width // 2):
            col = i * (D // width)
            c, z = s["rope"].double()[pos, col][:, None], s["rope"].double()[pos, 64 + col][:, None]
            for g in range(0, D, width):
                u, w = y[:, :, g + i], y[:, :, g + i + width // 2]
                out[:, :, g + i], out[:, :, g + i + width // 2] = u * c - w * z, w * c + u * z
        return out

    got = {"k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
    rows = {"q": [], "k": []}
    for b in range(s["n"]):
        p0, m, c0 = s["a"][b], s["b"][b], s["cu"][b]
        rows["k"].append(turned(s["k"][c0:c0 + m], p0))
        if s["case"]["queries"]:
            rows["q"].append(turned(s["q"][c0:c0 + m], p0))
        pos = torch.arange(p0, p0 + m, device="cuda")
        flat = s["table"][b].long()[pos // ps] * ps + pos % ps
        got["k_pool"].view(-1, s["case"]["hkv"], D)[flat] = rows["k"][-1]
        got["v_pool"].view(-1, s["case"]["hkv"], D)[flat] = s["v"][c0:c0 + m].double()
    if s["case"]["queries"]:
        got["q_out"], got["k_out"] = torch.cat(rows["q"]), torch.cat(rows["k"])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    hq, hkv = case["hq"], case["hkv"]
    g = hq // hkv
    names = {"prefill": ("out", "out2", "lse"), "decode": ("out", "out2", "lse"), "backward": ("dq", "dk", "dv")}[case["op"]]
    parts = {x: [] for x in names}
    dlam = torch.zeros(hq, dtype=torch.float64, device="cuda")
    for b in range(s["n"]):
        nq, nk = s["a"][b], s["b"][b]
        if case["op"] == "decode":
            pages = s["table"][b, : -(-nk // case["page"])].long()
            k, v = (s[x][pages].reshape(-1, hkv, D)[:nk].double() for x in ("k_pool", "v_pool"))
            q = s["q"][b:b + 1].double()
        else:
            q = s["q"][s["cu_q"][b]:s["cu_q"][b + 1]].double()
            k, v = (s[x][s["cu_k"][b]:s["cu_k"][b + 1]].double() for x in ("k", "v"))
        row = {x: torch.zeros((nq, hq, D) if x in ("out", "out2", "dq") else (nq, hq, 2) if x == "lse" else (nk, hkv, D), dtype=torch.float64, device="cuda") for x in names}
        seen = torch.ones((nq, nk), dtype=torch.bool, device="cuda").tril(nk - nq)
        for h in range(hq):
            weights = []
            for m in range(2):
                x = (q[:, h, m * M:m * M + M] @ k[:, h // g, m * M:m * M + M].T * s["scale"]).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, 1)
                weights.append(torch.exp(x - z[:, None]))
                if "lse" in row:
                    row["lse"][:, h, m] = z
            lam = s["lam"][h].double()
            if case["op"] != "backward":
                second = weights[1] @ v[:, h // g]
                row["out"][:, h], row["out2"][:, h] = weights[0] @ v[:, h // g] - lam * second, second
                continue
            do = s["dout"][s["cu_q"][b]:s["cu_q"][b + 1], h].double()
            dp = do @ v[:, h // g].T
            row["dv"][:, h // g] += (weights[0] - lam * weights[1]).T @ do
            for m, sign in ((0, 1.0), (1, -lam)):
                mean = (weights[m] * dp).sum(1, keepdim=True)
                ds = weights[m] * (dp - mean) * sign * s["scale"]
                row["dq"][:, h, m * M:m * M + M] = ds @ k[:, h // g, m * M:m * M + M]
                row["dk"][:, h // g, m * M:m * M + M] += ds.T @ q[:, h, m * M:m * M + M]
            dlam[h] -= mean.sum()
        for x in names:
            parts[x].append(row[x])
    got = {x: torch.cat(parts[x]) for x in names}
    if case["op"] == "backward":
        return got | {"dlam": dlam}
    if case["op"] == "decode":
        return {"out": got["out"], "out_bf16": got["out"], "lse": got["lse"]}
    return got if case["train"] else {"out_bf16": got["out"]}
