"""rlk_attn_cache_append on the GPU, bit for bit against the definition.

The rotation's products are rounded to FP32 on their own, the sum of such a
product and an exact one (48 bits) is exact in 64 bits up to the rounding that
the fused multiply-add makes, so NumPy in float64 rounded to float32 and then
to BF16 gives the same bits; unrotated rows are copies.
"""
import numpy as np
import pytest

import deterministic_context_attention_gb300 as rlk
from deterministic_context_attention_gb300 import synth

pytestmark = pytest.mark.gpu

STALE = 0x7FC1  # a NaN that no arithmetic here makes: what untouched places hold


def _bits(x):
    return (synth.bf16_round(np.asarray(x, np.float32)).view(np.uint32) >> 16).astype(np.uint16)


def _rotated(x, table, pos, width):
    """x [T, H, 128] float32 (BF16 values), positions [T] -> bits."""
    h, step = width // 2, 128 // width
    c, s = table[pos][:, None, None, :64:step], table[pos][:, None, None, 64::step]
    y = x.reshape(x.shape[0], x.shape[1], step, width)
    a, b = y[..., :h], y[..., h:]
    f64 = np.float64
    lo = (a.astype(f64) * c - (b * s).astype(f64)).astype(np.float32)
    hi = (b.astype(f64) * c + (a * s).astype(f64)).astype(np.float32)
    return _bits(np.concatenate([lo, hi], -1).reshape(x.shape))


def _table_of(lens, page, spare, seed):
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + spare
    perm = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    table, at = np.full((len(lens), max(max(per), 1)), -1, np.int32), 0
    for i, c in enumerate(per):
        table[i, :c] = perm[at:at + c]
        at += c
    return table, n_pages


class Problem:
    def __init__(self, pos, new, hq, hkv, page, width, seed=0):
        torch = pytest.importorskip("torch")
        g = np.random.default_rng([seed, 5])
        self.pos, self.new, self.hq, self.hkv, self.page, self.width = list(pos), list(new), hq, hkv, page, width
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        t = int(self.cu[-1])
        self.q, self.k, self.v = (synth.bf16_round(g.standard_normal((t, h, 128), dtype=np.float32)) for h in (hq, hkv, hkv))
        self.table, self.n_pages = _table_of([a + b for a, b in zip(pos, new)], page, 3, seed)
        self.at = np.concatenate([np.arange(a, a + b) for a, b in zip(pos, new)]).astype(np.int64)
        self.seq = np.repeat(np.arange(len(new)), new)
        self.max_pos = max(int(self.at.max()) + 1 if t else 1, 1)
        self.rope = rlk.rlk_attn_rope_table(1.0e6, self.max_pos) if width else None
        self.dev = lambda bits: torch.from_numpy(bits.view(np.int16).copy()).cuda().view(torch.bfloat16)
        self.params = rlk.make_params(len(new), hq, hkv)

    def expected(self):
        k = _rotated(self.k, self.rope, self.at, self.width) if self.width else _bits(self.k)
        pools = []
        for rows in (k, _bits(self.v)):
            pool = np.full((self.n_pages, self.page, self.hkv, 128), STALE, np.uint16)
            pool[self.table[self.seq, self.at // self.page], self.at % self.page] = rows
            pools.append(pool)
        q = _rotated(self.q, self.rope, self.at, self.width) if self.width else None
        return pools[0], pools[1], q, k

    def device(self):
        import torch
        stale = lambda *shape: self.dev(np.full(shape, STALE, np.uint16))  # noqa: E731
        t = int(self.cu[-1])
        pool = (self.n_pages, self.page, self.hkv, 128)
        return dict(q=self.dev(_bits(self.q)), k=self.dev(_bits(self.k)), v=self.dev(_bits(self.v)), q_out=stale(t, self.hq, 128),
                    k_out=stale(t, self.hkv, 128), kp=stale(*pool), vp=stale(*pool), table=torch.from_numpy(self.table).cuda(),
                    rope=None if self.rope is None else torch.from_numpy(self.rope).cuda())

    def call(self, d, queries=True, stream=None):
        rlk.rlk_attn_cache_append(self.params, d["q"] if queries else None, d["q_out"] if queries else None, d["k"],
                                  d["k_out"] if queries else None, d["v"], self.cu, self.pos, d["rope"],
                                  self.max_pos if self.width else 0, self.width or 128, d["kp"], d["vp"], self.n_pages,
                                  self.page, d["table"], self.table.shape[1], stream=stream)


def _back(x):
    import torch
    return x.view(torch.int16).cpu().numpy().view(np.uint16)


def _check(p, d, queries):
    import torch
    torch.cuda.synchronize()
    rlk.rlk_attn_check_device_error()
    kp, vp, q, k = p.expected()
    assert np.array_equal(_back(d["kp"]), kp)
    assert np.array_equal(_back(d["vp"]), vp)
    if queries:
        assert np.array_equal(_back(d["q_out"]), q)
        assert np.array_equal(_back(d["k_out"]), k)
    else:
        assert np.all(_back(d["q_out"]) == STALE) and np.all(_back(d["k_out"]) == STALE)
    assert np.array_equal(_back(d["v"]), _bits(p.v))


@pytest.mark.parametrize("width,queries", [(0, False), (64, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("pos,new,hq,hkv,page", [
    ([0], [1], 32, 8, 16), ([15], [1], 32, 8, 16), ([700], [1], 4, 1, 8), ([0], [129], 8, 8, 32),
    ([13, 0, 64, 5], [3, 0, 65, 1], 24, 8, 16), ([0, 127, 128], [128, 1, 300], 40, 8, 128),
    ([3, 1000, 77, 0, 5], [333, 17, 0, 64, 1], 16, 4, 64), ([9, 2], [31, 40], 7, 7, 8)])
def test_rows_are_the_definition_s(pos, new, hq, hkv, page, width, queries):
    p = Problem(pos, new, hq, hkv, page, width, seed=hq + page)
    d = p.device()
    p.call(d, queries)
    _check(p, d, queries)


def test_width_128_has_the_bits_of_the_rope_pass():
    import torch
    p = Problem([3, 50], [200, 61], 32, 8, 16, 128, seed=3)
    d = p.device()
    p.call(d)
    q, k = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    rlk.rlk_attn_rope_qk(p.params, d["q"], q, d["k"], k, p.cu, p.pos, d["rope"], p.max_pos)
    assert np.array_equal(_back(q), _back(d["q_out"])) and np.array_equal(_back(k), _back(d["k_out"]))


@pytest.mark.parametrize("width", [64, 128])
def test_in_place(width):
    p = Problem([3, 50, 0], [200, 61, 5], 32, 8, 16, width, seed=4)
    d = p.device()
    d["q_out"], d["k_out"] = d["q"], d["k"]
    p.call(d)
    _check(p, d, True)


def test_token_by_token_in_chunks_and_at_once():
    whole = Problem([0], [77], 16, 4, 16, 64, seed=5)
    want = whole.expected()
    for step in (1, 7, 40):
        d = whole.device()
        for a in range(0, 77, step):
            n = min(step, 77 - a)
            q, k, v, qo, ko = (d[x][a:a + n] for x in ("q", "k", "v", "q_out", "k_out"))
            rlk.rlk_attn_cache_append(rlk.make_params(1, 16, 4), q, qo, k, ko, v, [0, n], [a], d["rope"], whole.max_pos, 64,
                                      d["kp"], d["vp"], whole.n_pages, 16, d["table"], whole.table.shape[1])
        for got, w in zip((d["kp"], d["vp"], d["q_out"], d["k_out"]), want):
            assert np.array_equal(_back(got), w), step


def test_more_sequences_than_one_launch_takes():
    g = np.random.default_rng(6)
    pos, new = g.integers(0, 40, 600), g.integers(0, 4, 600)
    p = Problem(pos.tolist(), new.tolist(), 8, 2, 8, 128, seed=6)
    d = p.device()
    p.call(d)
    _check(p, d, True)


def test_bad_pages_are_reported_and_their_rows_left_out():
    p = Problem([0, 0], [40, 20], 8, 2, 16, 64, seed=7)
    want = p.expected()
    for bad in (-1, p.n_pages, 2 ** 31 - 1, -2 ** 31):
        d = p.device()
        d["table"][0, 1] = bad
        p.call(d)
        with pytest.raises(rlk.RlkError) as e:
            rlk.rlk_attn_check_device_error()
        assert e.value.status == 8
        rlk.rlk_attn_check_device_error()  # and reported once
        kp, vp = want[0].copy(), want[1].copy()
        kp[p.table[0, 1]] = vp[p.table[0, 1]] = STALE
        assert np.array_equal(_back(d["kp"]), kp) and np.array_equal(_back(d["vp"]), vp)
        assert np.array_equal(_back(d["q_out"]), want[2]) and np.array_equal(_back(d["k_out"]), want[3])


def test_another_stream_and_a_captured_call():
    import torch
    p = Problem([3, 50], [20, 61], 32, 8, 16, 64, seed=8)
    d = p.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.call(d, stream=side)
    side.synchronize()
    _check(p, d, True)
    d = p.device()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call(d)
    assert np.all(_back(d["kp"]) == STALE)
    for _ in range(2):
        graph.replay()
        _check(p, d, True)
    # other rows at the captured addresses
    p.k = p.k[::-1].copy()
    d["k"].copy_(p.dev(_bits(p.k)))
    graph.replay()
    _check(p, d, True)


def test_pool_past_32_bit_offsets():
    # 2.2 G elements a pool: the last page's rows lie past 2^31 elements
    import torch
    hkv, page, n_pages = 8, 128, 17000
    kp = torch.zeros((n_pages, page, hkv, 128), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k, v = (torch.randn((130, hkv, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[n_pages - 1, 3]], dtype=torch.int32, device="cuda")
    rlk.rlk_attn_cache_append(rlk.make_params(1, 8, hkv), None, None, k, None, v, [0, 130], None, None, 0, 128, kp, vp,
                              n_pages, page, table, 2)
    rlk.rlk_attn_check_device_error()
    for pool, rows in ((kp, k), (vp, v)):
        assert torch.equal(pool[n_pages - 1], rows[:128]) and torch.equal(pool[3, :2], rows[128:])
        assert int(torch.count_nonzero(pool[3, 2:])) == 0 and int(torch.count_nonzero(pool[:3])) == 0


def test_decode_reads_what_append_wrote():
    """The plain paged decode over appended pages has the bits of the prefill over the same packed rows."""
    import torch
    p = Problem([0, 0, 0], [200, 1, 333], 32, 8, 16, 128, seed=9)
    d = p.device()
    p.call(d)
    out, ref = (torch.empty((3, 32, 128), dtype=torch.float32, device="cuda") for _ in range(2))
    lens = np.array(p.new, np.int32)
    rlk.rlk_attn_decode_paged(p.params, d["q_out"][torch.tensor(p.cu[1:] - 1).long().cuda()].contiguous(), d["kp"], d["vp"],
                              p.n_pages, 16, d["table"], p.table.shape[1], lens, out, None, None)
    full = torch.empty((int(p.cu[-1]), 32, 128), dtype=torch.float32, device="cuda")
    rlk.rlk_attn_prefill(p.params, d["q_out"], d["k_out"], d["v"], p.cu, p.cu, -1, full, None, None)
    ref = full[torch.tensor(p.cu[1:] - 1).long().cuda()]
    assert torch.equal(out.view(torch.int32), ref.view(torch.int32))
