"""Problems and runs of the 8-bit paged KV cache for the tests."""
from __future__ import annotations

import dataclasses

import numpy as np

import oracle.qcache as oq
from deterministic_context_attention_gb300 import synth

STALE = 0xA7  # what the slots no token has hold before a test


@dataclasses.dataclass
class Cache:
    """Host image of an 8-bit cache: pools, scales, page table."""
    k: np.ndarray
    v: np.ndarray
    ks: np.ndarray
    vs: np.ndarray
    table: np.ndarray
    page: int

    @property
    def n_pages(self):
        return self.k.shape[0]

    def copy(self):
        return Cache(self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy(), self.table.copy(), self.page)

    def device(self):
        import torch
        return [torch.from_numpy(a.copy()).cuda() for a in (self.k, self.v, self.ks, self.vs, self.table)]


def empty_cache(lens, hkv, page, seed=0, spare=3, stale=STALE):
    """Pages for sequences of ``lens`` tokens, scattered over the pool."""
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + spare
    perm = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), max(max(per), 1)), -1, np.int32)
    at = 0
    for s, c in enumerate(per):
        table[s, :c] = perm[at:at + c]
        at += c
    k = np.full((n_pages, hkv, page, 128), stale, np.uint8)
    ks = np.full((n_pages, hkv), 3.0e9, np.float32)
    return Cache(k, k.copy(), ks, ks.copy(), table, page)


def tokens(lens, hkv, seed, spread=True):
    """K and V rows of every sequence; with ``spread`` their size varies by
    head, channel and token, so that scales differ and grow inside a page."""
    g = np.random.default_rng([seed, 99])
    out = []
    for s, n in enumerate(lens):
        kv = []
        for _ in range(2):
            x = g.standard_normal((n, hkv, 128), dtype=np.float32)
            if spread:
                x *= np.exp2(g.integers(-6, 7, (n, 1, 1))) * np.exp2(g.integers(-3, 4, (1, hkv, 128)))
                x[g.random((n, hkv, 128)) < 0.02] = 0.0
            kv.append(synth.bf16_round(x))
        out.append(kv)
    return out


def filled(lens, hkv, page, seed, spread=True, stale=0x7F):
    """A cache that holds ``lens`` tokens of every sequence, by definition."""
    c = empty_cache(lens, hkv, page, seed, stale=stale)
    for s, (k, v) in enumerate(tokens(lens, hkv, seed, spread)):
        oq.write_tokens(c.k, c.ks, c.table[s], k)
        oq.write_tokens(c.v, c.vs, c.table[s], v)
    return c


def bf16_pools(c):
    """The cache's values as BF16 pools [n_pages, page, hkv, 128] (float32,
    exact), NaN codes included."""
    return tuple(np.ascontiguousarray(oq.values(p, s).transpose(0, 2, 1, 3)).astype(np.float32)
                 for p, s in ((c.k, c.ks), (c.v, c.vs)))


def run_write(rlk, torch, dev, params, k, v, cu, pos, n_pages, page, rope=None, max_pos=0):
    kd, vd, ksd, vsd, td = dev
    rlk.rlk_attn_qcache_write(params, k, v, cu, pos, rope, max_pos, kd, vd, ksd, vsd, n_pages, page, td, td.shape[1])


def to_bf16(torch, x):
    return torch.from_numpy(np.ascontiguousarray(synth.bf16_bits(x)).view(np.int16)).cuda().view(torch.bfloat16)


def decode(rlk, torch, c, q, ctx, hq, split_k=1, seqs=None, rope=None, max_pos=0, table=None, dev=None, scale=None,
           check=True):
    """rlk_attn_decode_qcache of the given sequences; numpy outputs."""
    seqs = list(range(len(ctx))) if seqs is None else list(seqs)
    ctx = np.asarray(ctx, np.int32)[seqs]
    kd, vd, ksd, vsd, td = c.device() if dev is None else dev
    td = torch.from_numpy(np.ascontiguousarray((c.table if table is None else table)[seqs])).cuda()
    n, hkv = len(seqs), c.k.shape[1]
    out = torch.full((n, hq, 128), float("nan"), device="cuda")
    outb = torch.full((n, hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, hq), float("nan"), device="cuda")
    p = rlk.make_params(n, hq, hkv, 128, softmax_scale=scale)
    ws = None
    if split_k != 1:
        ws = torch.empty(rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DECODE_QCACHE, None, ctx), dtype=torch.uint8,
                         device="cuda")
    rlk.rlk_attn_decode_qcache(p, to_bf16(torch, q[seqs]), kd, vd, ksd, vsd, c.n_pages, c.page, td, td.shape[1], ctx,
                               split_k, rope, max_pos, out, outb, lse, ws)
    if check:
        rlk.rlk_attn_check_device_error()
    return out.cpu().numpy(), outb.float().cpu().numpy(), lse.cpu().numpy()
