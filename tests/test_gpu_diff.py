"""Differential attention on the GPU: against the FP64 definition, within the
bounds that its FP32 evaluation can reach (oracle/diff.py), and bit for bit
against itself over chunks, ranks, batches, pages, splits and repeats."""
import numpy as np
import pytest

import deterministic_context_attention_gb300 as rlk
import oracle.diff as od
from deterministic_context_attention_gb300 import synth

pytestmark = pytest.mark.gpu

SCALE = 0.125
GRAD_REL_L2 = 1e-4  # the backward's gate, as for the plain one


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Problem:
    """Packed rows of a batch: queries are the last tokens of each sequence."""

    def __init__(self, q_lens, k_lens, hq, hkv, seed=0, gain=1.0, scale=SCALE):
        g = np.random.default_rng([seed, 7])
        self.q_lens, self.k_lens, self.hq, self.hkv, self.scale = list(q_lens), list(k_lens), hq, hkv, scale
        self.cq, self.ck = _cu(q_lens), _cu(k_lens)
        tq, tk = int(self.cq[-1]), int(self.ck[-1])
        rows = lambda t, h, s=1.0: synth.bf16_round(np.float32(s) * g.standard_normal((t, h, 128), dtype=np.float32))  # noqa: E731
        self.q, self.k, self.v, self.dout = rows(tq, hq, gain), rows(tk, hkv), rows(tk, hkv), rows(tq, hq)
        self.lam = (0.5 + 0.5 * g.standard_normal(hq)).astype(np.float32)

    @property
    def params(self):
        return self.params_of()

    def params_of(self, cp=1, layout=1):
        return rlk.make_params(len(self.q_lens), self.hq, self.hkv, 128, cp, layout, self.scale)

    def device(self):
        import torch
        bf = lambda x: torch.from_numpy(x).cuda().to(torch.bfloat16)  # noqa: E731
        return bf(self.q), bf(self.k), bf(self.v), torch.from_numpy(self.lam).cuda()

    def forward(self, dev=None, ranks=(-1,), cp=1, layout=1, stream=None):
        """out, out_bf16, out2, lse on the device (NaN where nothing was written)."""
        import torch
        q, k, v, lam = dev or self.device()
        t = int(self.cq[-1])
        full = lambda *s, **kw: torch.full(s, float("nan"), device="cuda", **kw)  # noqa: E731
        out, out2, lse = full(t, self.hq, 128), full(t, self.hq, 128), full(t, self.hq, 2)
        outb = full(t, self.hq, 128, dtype=torch.bfloat16)
        for r in ranks:
            rlk.rlk_attn_diff_prefill(self.params_of(cp, layout), q, k, v, lam, self.cq, self.ck, r, out, outb, out2, lse, stream=stream)
        rlk.rlk_attn_check_device_error()
        return out, outb, out2, lse

    def backward(self, dev=None, fwd=None, ranks=(-1,), cp=1, layout=1):
        """dq, dk, dv, dlam on the device."""
        import torch
        q, k, v, lam = dev or self.device()
        out, _, out2, lse = fwd or self.forward((q, k, v, lam))
        dout = torch.from_numpy(self.dout).cuda().to(torch.bfloat16)
        p = self.params_of(cp, layout)
        ws = torch.full((rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DIFF_BACKWARD, self.cq),), 0xFF, dtype=torch.uint8, device="cuda")
        got = [torch.full(x.shape, float("nan"), dtype=torch.float32, device="cuda") for x in (q, k, v, lam)]
        for r in ranks:
            rlk.rlk_attn_diff_backward(p, q, k, v, lam, out, out2, dout, lse, self.cq, r, *got, ws)
        rlk.rlk_attn_check_device_error()
        return got

    def sequence(self, s):
        a, b = slice(self.cq[s], self.cq[s + 1]), slice(self.ck[s], self.ck[s + 1])
        return self.q[a], self.k[b], self.v[b], a, b


def _np(x):
    return x.float().cpu().numpy().astype(np.float64)


def _same(a, b, what=""):
    import torch
    for i, (x, y) in enumerate(zip(a, b)):
        kind = torch.int16 if x.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(x.contiguous().view(kind), y.contiguous().view(kind)), (what, i)


def _within(got, want, tol, what):
    off = np.abs(got - want)
    assert np.isfinite(got).all(), what
    assert np.all(off <= tol), (what, float((off / np.maximum(tol, 1e-300)).max()), float(off.max()))


SHAPES = [([1], [1], 32, 8), ([77], [77], 32, 8), ([128, 1, 129], [128, 1, 129], 8, 8), ([1, 1], [300, 513], 4, 1),
          ([64, 200, 0, 3], [700, 200, 0, 3], 40, 8), ([257], [385], 8, 1), ([130], [130], 16, 1)]


@pytest.mark.parametrize("q_lens,k_lens,hq,hkv", SHAPES)
def test_prefill_is_the_definition(q_lens, k_lens, hq, hkv):
    import torch
    p = Problem(q_lens, k_lens, hq, hkv, seed=len(q_lens) + hq)
    out, outb, out2, lse = p.forward()
    for s in range(len(q_lens)):
        q, k, v, a, _ = p.sequence(s)
        if q.shape[0] == 0:
            continue
        w, w2, wl, t, t2, tl = od.forward(q, k, v, p.lam, p.scale)
        _within(_np(out[a]), w, t, "out")
        _within(_np(out2[a]), w2, t2, "out2")
        _within(_np(lse[a]), wl, tl, "lse")
    _same([outb], [out.to(torch.bfloat16)], "one rounding at the end")


@pytest.mark.parametrize("gain", [12.0, 0.01])
def test_prefill_with_large_and_small_scores(gain):
    p = Problem([150], [290], 8, 2, seed=3, gain=gain)
    out, _, out2, lse = p.forward()
    w, w2, wl, t, t2, tl = od.forward(p.q, p.k, p.v, p.lam, p.scale)
    _within(_np(out), w, t, "out")
    _within(_np(out2), w2, t2, "out2")
    _within(_np(lse), wl, tl, "lse")


@pytest.mark.parametrize("q_lens,k_lens,hq,hkv", SHAPES + [([1000, 300, 90], [1000, 2300, 90], 32, 8)])
def test_prefill_agrees_with_plain_prefills_over_one_map(q_lens, k_lens, hq, hkv):
    # each side's O_m is within the plain prefill's gate (TOL_OUT, TOL_LSE) of the definition
    import torch
    from tests.gpu_helpers import TOL_LSE, TOL_OUT
    p = Problem(q_lens, k_lens, hq, hkv, seed=5)
    dev = p.device()
    out, _, out2, lse = p.forward(dev)
    q, k, v, lam = dev
    o, l = [], []
    for m in range(2):
        one = torch.zeros_like(q)
        one[..., 64 * m:64 * m + 64] = q[..., 64 * m:64 * m + 64]
        o.append(torch.empty_like(out))
        l.append(torch.empty(out.shape[:2], device="cuda"))
        rlk.rlk_attn_prefill(p.params, one, k, v, p.cq, p.ck, -1, o[m], None, l[m])
    want = o[0].double() - lam.double()[:, None] * o[1].double()
    assert bool(((out - want).abs() <= 2 * TOL_OUT * (1 + lam.abs()[:, None])).all())
    assert float((out2 - o[1]).abs().max()) <= 2 * TOL_OUT and float((lse - torch.stack(l, -1)).abs().max()) <= 2 * TOL_LSE


def _uneven(x, hq, seed):
    """Channels of different size, a few large, as queries and keys have them."""
    g = np.random.default_rng([seed, 11])
    gain = g.uniform(0.3, 1.0, x.shape[-2:]) * np.where(g.random(x.shape[-2:]) < 0.03, 6.0, 1.0)
    return synth.bf16_round((x * gain).astype(np.float32))


def _fp64_rows(p, rows):
    """out and lse of some query rows of a one-sequence problem, in FP64 on the device."""
    import torch
    q, k, v, lam = (x.double() for x in p.device())
    g, nk, nq = p.hq // p.hkv, k.shape[0], q.shape[0]
    out = torch.empty((len(rows), p.hq, 128), dtype=torch.float64, device="cuda")
    lse = torch.empty((len(rows), p.hq, 2), dtype=torch.float64, device="cuda")
    seen = torch.arange(nk, device="cuda")[None] <= torch.tensor(rows, device="cuda")[:, None] + nk - nq
    for h in range(p.hq):
        o = []
        for m in range(2):
            at = slice(64 * m, 64 * m + 64)
            x = (q[rows, h, at] @ k[:, h // g, at].T * p.scale).masked_fill(~seen, -np.inf)
            lse[:, h, m] = torch.logsumexp(x, 1)
            o.append(torch.exp(x - lse[:, h, m, None]) @ v[:, h // g])
        out[:, h] = o[0] - lam[h] * o[1]
    return out, lse


# relative 2-norm over long contexts: P's two pieces leave 2^-18 of a weight at
# the most, in random directions; a log-sum-exp fold is 1e-4 off here
LONG_REL_L2 = 2.0 ** -17


def test_long_contexts_with_uneven_channels():
    p = Problem([64], [20000], 8, 2, seed=18)
    p.q, p.k = _uneven(p.q, 8, 1), _uneven(p.k, 2, 2)
    out, _, _, lse = p.forward()
    rows = [0, 17, 63]
    want, wl = _fp64_rows(p, rows)
    assert float(wl.abs().min()) > 8  # log sums of a size at which FP32 holds 2^-21
    assert float((out[rows] - want).norm() / want.norm()) <= LONG_REL_L2
    assert float((lse[rows] - wl).abs().max()) <= 2.0 ** -17
    c = Paged([20000, 9000], 8, 2, 16, seed=18)
    c.p.q, c.p.k = _uneven(c.p.q, 8, 1), _uneven(c.p.k, 2, 2)
    c = Paged.of(c.p, c.ctx, 16, 18)
    got, _, gl = c.decode(0)
    for s in range(2):
        one = Problem([1], [int(c.ctx[s])], 8, 2)
        one.q, one.k, one.v, a, _ = c.p.sequence(s)
        one.lam = c.p.lam
        want, wl = _fp64_rows(one, [0])
        assert float((got[a] - want).norm() / want.norm()) <= LONG_REL_L2
        assert float((gl[a] - wl).abs().max()) <= 2.0 ** -17


def test_equal_maps_cancel():
    p = Problem([200], [200], 8, 2, seed=6)
    p.q[..., 64:], p.k[..., 64:] = p.q[..., :64], p.k[..., :64]
    p.lam[:] = 1.0
    out, _, out2, lse = p.forward()
    assert np.all(_np(out) == 0) and np.all(_np(lse)[..., 0] == _np(lse)[..., 1])
    p.lam[:4] = 0.0  # and a weight of zero leaves the first map
    out, _, out2, _ = p.forward()
    assert np.all(_np(out)[:, :4] == _np(out2)[:, :4]) and np.all(_np(out)[:, 4:] == 0)


@pytest.mark.parametrize("chunk", [1, 100, 128, 333])
def test_chunks_have_the_bits_of_the_whole(chunk):
    import torch
    p = Problem([700], [700], 16, 4, seed=8)
    dev = p.device()
    whole = p.forward(dev)
    q, k, v, lam = dev
    starts = range(0, 700, chunk) if chunk > 1 else (0, 1, 127, 128, 500, 699)
    for a in starts:
        b = min(700, a + chunk)
        part = Problem([b - a], [b], 16, 4)
        got = part.forward((q[a:b].contiguous(), k[:b].contiguous(), v[:b].contiguous(), lam))
        _same(got, [x[a:b] for x in whole], a)


@pytest.mark.parametrize("cp,layout", [(2, 0), (4, 1), (8, 1)])
def test_ranks_repeats_and_batch_order(cp, layout):
    import torch
    lens = [300, 1, 513, 128]
    p = Problem(lens, lens, 8, 2, seed=9)
    dev = p.device()
    fwd, bwd = p.forward(dev), p.backward(dev)
    _same(p.forward(dev), fwd, "repeat")
    _same(p.forward(dev, ranks=range(cp), cp=cp, layout=layout), fwd, "ranks")
    _same(p.backward(dev, fwd), bwd, "repeat")
    _same(p.backward(dev, fwd, ranks=reversed(range(cp)), cp=cp, layout=layout), bwd, "ranks")
    order = [2, 0, 3]  # another order, without the second sequence
    rows = torch.from_numpy(np.concatenate([np.arange(p.cq[s], p.cq[s + 1]) for s in order])).cuda()
    part = Problem([lens[s] for s in order], [lens[s] for s in order], 8, 2)
    part.dout = p.dout[rows.cpu().numpy()]
    sub = (dev[0][rows].contiguous(), dev[1][rows].contiguous(), dev[2][rows].contiguous(), dev[3])
    got = part.forward(sub)
    _same(got, [x[rows] for x in fwd], "subset")
    _same(part.backward(sub, got)[:3], [x[rows] for x in bwd[:3]], "subset")


def test_rows_behind_the_batch_stay():
    import torch
    p = Problem([100, 3], [100, 3], 8, 2, seed=10)
    q, k, v, lam = p.device()
    pad = lambda x: torch.cat([x, torch.full_like(x[:40], float("nan"))])  # noqa: E731
    big = [pad(x) for x in (q, k, v)]
    outs = [torch.full((143, 8, n), 7.0, device="cuda") for n in (128, 128, 2)]
    rlk.rlk_attn_diff_prefill(p.params, *big, lam, p.cq, p.ck, -1, outs[0], None, outs[1], outs[2])
    ref = p.forward()
    _same([x[:103] for x in outs], [ref[0], ref[2], ref[3]])
    assert all(bool((x[103:] == 7.0).all()) for x in outs)
    ws = torch.empty(rlk.rlk_attn_workspace_size(p.params, rlk.RLK_OP_DIFF_BACKWARD, p.cq), dtype=torch.uint8, device="cuda")
    grads = [torch.full(x.shape, 7.0, device="cuda") for x in (*big, lam)]
    dout = pad(torch.from_numpy(p.dout).cuda().to(torch.bfloat16))
    rlk.rlk_attn_diff_backward(p.params, *big, lam, outs[0], outs[1], dout, outs[2], p.cq, -1, *grads, ws)
    rlk.rlk_attn_check_device_error()
    _same([x[:103] for x in grads[:3]] + grads[3:], p.backward())
    assert all(bool((x[103:] == 7.0).all()) for x in grads[:3])


# ---------------------------------------------------------------- backward

def _check_backward(p):
    got = [_np(x) for x in p.backward()]
    want, tol = [np.zeros_like(x) for x in got], [np.zeros_like(x) for x in got]
    for s in range(len(p.q_lens)):
        q, k, v, a, b = p.sequence(s)
        if q.shape[0] == 0:
            continue
        r = od.backward(q, k, v, p.lam, p.dout[a], p.scale)
        for i, at in enumerate((a, b, b)):
            want[i][at], tol[i][at] = r[i], r[4 + i]
        want[3] += r[3]
        tol[3] += r[7] + 2.0 ** -23 * np.abs(want[3])
    for x, w, t, name in zip(got, want, tol, ("dq", "dk", "dv", "dlam")):
        _within(x, w, t, name)
    if max(p.q_lens) > 1:  # (of one token alone the gradients of q and k are zero)
        for x, w, name in zip(got, want, ("dq", "dk", "dv", "dlam")):
            assert np.linalg.norm(x - w) <= GRAD_REL_L2 * np.linalg.norm(w), name


@pytest.mark.parametrize("lens,hq,hkv", [([1], 8, 2), ([2], 4, 4), ([77], 32, 8), ([128, 1, 129], 8, 8), ([257, 0, 64], 10, 2),
                                         ([385], 8, 1), ([130, 300], 40, 8)])
def test_backward_is_the_definition(lens, hq, hkv):
    _check_backward(Problem(lens, lens, hq, hkv, seed=len(lens) + hq))


@pytest.mark.parametrize("lam", [0.0, 1.0, -3.0])
def test_backward_at_other_weights(lam):
    p = Problem([200], [200], 8, 2, seed=12)
    p.lam[:] = lam
    _check_backward(p)


def test_backward_with_large_scores():
    _check_backward(Problem([150], [150], 8, 2, seed=13, gain=6.0))


def test_backward_without_the_second_map_is_the_plain_one():
    # lambda = 0: out = O_1, dv and the first halves are those of the plain backward over map 1 alone
    import torch
    p = Problem([300, 130], [300, 130], 8, 2, seed=14)
    p.lam[:] = 0.0
    dev = p.device()
    fwd = p.forward(dev)
    dq, dk, dv, dlam = p.backward(dev, fwd)
    q, k, v, _ = dev
    one = torch.zeros_like(q)
    one[..., :64] = q[..., :64]
    dout = torch.from_numpy(p.dout).cuda().to(torch.bfloat16)
    ws = torch.empty(rlk.rlk_attn_workspace_size(p.params, rlk.RLK_OP_BACKWARD, p.cq), dtype=torch.uint8, device="cuda")
    ref = [torch.empty(x.shape, device="cuda") for x in (q, k, v)]
    rlk.rlk_attn_backward(p.params, one, k, v, fwd[0], dout, fwd[3][..., 0].contiguous(), p.cq, -1, *ref, ws)
    for x, y in ((dq[..., :64], ref[0][..., :64]), (dk[..., :64], ref[1][..., :64]), (dv, ref[2])):
        # each side is within GRAD_REL_L2 of the definition (the sums' cuts differ,
        # and the tensor core truncates: 2^-24 of the sum a product)
        assert float((x - y).norm()) <= 2 * GRAD_REL_L2 * float(y.norm())
    assert not bool(dq[..., 64:].any()) and not bool(dk[..., 64:].any()) and bool(dlam.any())


def test_more_sequences_than_one_launch_takes():
    g = np.random.default_rng(15)
    lens = g.integers(0, 40, 300).tolist()
    p = Problem(lens, lens, 4, 2, seed=15)
    dev = p.device()
    fwd, grads = p.forward(dev), p.backward(dev)
    total = np.zeros(4)
    for s in (0, 127, 128, 255, 256, 299):
        a = slice(int(p.cq[s]), int(p.cq[s + 1]))
        if a.start == a.stop:
            continue
        part = Problem([lens[s]], [lens[s]], 4, 2)
        part.dout = p.dout[a]
        sub = (*(x[a].contiguous() for x in dev[:3]), dev[3])
        one = part.forward(sub)
        _same(one, [x[a] for x in fwd], s)
        _same(part.backward(sub, one)[:3], [x[a] for x in grads[:3]], s)
    want, tol = np.zeros(4), np.zeros(4)
    for s in range(300):
        q, k, v, a, _ = p.sequence(s)
        if q.shape[0]:
            r = od.backward(q, k, v, p.lam, p.dout[a], p.scale)
            want += r[3]
            tol += r[7]
    _within(_np(grads[3]), want, tol + 3 * 2.0 ** -23 * np.abs(want), "dlam")


def test_more_tiles_than_one_launch_takes():
    # 118 sequences of 16 tiles: both directions need a second launch, whose
    # results are those of each sequence alone
    import torch
    n, each, hq = 118, 2001, 2
    p = Problem([1], [1], hq, 1)
    p.q_lens = p.k_lens = [each] * n
    p.cq = p.ck = _cu(p.q_lens)
    g = torch.Generator(device="cuda").manual_seed(23)
    rows = lambda h: torch.randn((n * each, h, 128), device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    dev = (rows(hq), rows(1), rows(1), torch.tensor([0.3, 0.7], device="cuda"))
    p.dout = rows(hq).float().cpu().numpy()
    fwd = p.forward(dev)
    grads = p.backward(dev, fwd)
    for s in (0, 57, 117):
        a = slice(s * each, (s + 1) * each)
        one = Problem([1], [1], hq, 1)
        one.q_lens = one.k_lens = [each]
        one.cq = one.ck = _cu([each])
        one.dout = p.dout[a]
        sub = (*(x[a].contiguous() for x in dev[:3]), dev[3])
        alone = one.forward(sub)
        _same(alone, [x[a] for x in fwd], s)
        _same(one.backward(sub, alone)[:3], [x[a] for x in grads[:3]], s)


@pytest.mark.parametrize("layout", [0, 1])
def test_every_rank_has_the_whole_dlambda(layout):
    # ranks without a row of their own among them
    p = Problem([1, 70], [1, 70], 12, 4, seed=25)
    dev = p.device()
    fwd = p.forward(dev)
    want = p.backward(dev, fwd)[3]
    for r in range(8):
        _same([p.backward(dev, fwd, ranks=[r], cp=8, layout=layout)[3]], [want], r)


def test_two_backward_calls_at_once():
    # on two streams, each with its own workspace and outputs
    import torch
    p = Problem([700, 33], [700, 33], 8, 2, seed=24)
    dev = p.device()
    fwd = p.forward(dev)
    want = p.backward(dev, fwd)
    out, _, out2, lse = fwd
    dout = torch.from_numpy(p.dout).cuda().to(torch.bfloat16)
    need = rlk.rlk_attn_workspace_size(p.params, rlk.RLK_OP_DIFF_BACKWARD, p.cq)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.full_like(x, float("nan")) for x in want] for _ in streams]
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, g, w in zip(streams, got, ws):
            rlk.rlk_attn_diff_backward(p.params, *dev, out, out2, dout, lse, p.cq, -1, *g, w, stream=st)
    torch.cuda.synchronize()
    rlk.rlk_attn_check_device_error()
    for g in got:
        _same(g, want)


def test_empty_batches():
    import torch
    p = Problem([0, 0], [0, 0], 8, 2)
    dlam = torch.full((8,), float("nan"), device="cuda")
    lam = torch.ones(8, device="cuda")
    rlk.rlk_attn_diff_backward(p.params, None, None, None, lam, None, None, None, None, p.cq, -1, None, None, None, dlam, None)
    rlk.rlk_attn_check_device_error()
    assert not bool(dlam.any())
    many = rlk.make_params(300, 8, 2)
    dlam.fill_(float("nan"))
    rlk.rlk_attn_diff_backward(many, None, None, None, lam, None, None, None, None, [0] * 301, -1, None, None, None, dlam, None)
    assert not bool(dlam.any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_do_not_leak(bad):
    # a sequence of NaN or Inf beside ones whose last tiles it shares
    import torch
    lens = [130, 70, 5, 300]
    p = Problem(lens, lens, 8, 2, seed=21)
    fwd, bwd = p.forward(), p.backward()
    at = slice(int(p.cq[1]), int(p.cq[2]))
    for x in (p.q, p.k, p.v, p.dout):
        x[at] = bad
    keep = torch.ones(int(p.cq[-1]), dtype=torch.bool)
    keep[at] = False
    got = p.forward()
    _same([x[keep] for x in got], [x[keep] for x in fwd], "forward")
    assert not bool(torch.isfinite(got[0][at]).any())
    _same([x[keep] for x in p.backward(fwd=got)[:3]], [x[keep] for x in bwd[:3]], "backward")


# ---------------------------------------------------------------- decode

class Paged:
    """A cache of random rows, the unused slots NaN, and one query a sequence."""

    def __init__(self, ctx, hq, hkv, page, seed=0):
        self._set(Problem([1] * len(ctx), ctx, hq, hkv, seed=seed), ctx, page, seed)

    @classmethod
    def of(cls, p, ctx, page, seed):
        c = cls.__new__(cls)
        c._set(p, ctx, page, seed)
        return c

    def _set(self, p, ctx, page, seed, spare=2):
        import torch
        self.p, hkv = p, p.hkv
        self.ctx, self.page = np.asarray(ctx, np.int32), page
        self.dev = self.p.device()
        per = [-(-c // page) for c in ctx]
        self.n_pages, self.max_pages = sum(per) + spare, max(per) + 1
        perm = np.random.default_rng(seed).permutation(self.n_pages).astype(np.int32)
        table, at = np.full((len(ctx), self.max_pages), -1, np.int32), 0
        for i, c in enumerate(per):
            table[i, :c] = perm[at:at + c]
            at += c
        self.table = torch.from_numpy(table).cuda()
        self.kp = torch.full((self.n_pages, page, hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vp = self.kp.clone()
        _, k, v, _ = self.dev
        rlk.rlk_attn_cache_append(self.p.params, None, None, k, None, v, self.p.ck, None, None, 0, 128, self.kp, self.vp,
                                  self.n_pages, page, self.table, self.max_pages)
        need = rlk.rlk_attn_workspace_size(self.p.params, rlk.RLK_OP_DIFF_DECODE, None, self.ctx)
        self.ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")

    def outputs(self):
        import torch
        n, hq = len(self.ctx), self.p.hq
        out = torch.full((n, hq, 128), float("nan"), device="cuda")
        return out, out.to(torch.bfloat16), torch.full((n, hq, 2), float("nan"), device="cuda")

    def call(self, split, outs, ws=True, stream=None):
        q, _, _, lam = self.dev
        rlk.rlk_attn_diff_decode(self.p.params, q, lam, self.kp, self.vp, self.n_pages, self.page, self.table, self.max_pages,
                                 self.ctx, split, *outs, self.ws if ws else None, stream=stream)

    def decode(self, split, ws=True):
        outs = self.outputs()
        self.call(split, outs, ws)
        rlk.rlk_attn_check_device_error()
        return outs

    def prefill(self):
        out, outb, _, lse = self.p.forward(self.dev)
        return out, outb, lse


def _near_prefill(c, got):
    """The decode's fold has two levels, the prefill's one: within twice what
    either may be off the definition (their bounds, with values of size 4)."""
    from tests.gpu_helpers import TOL_LSE, TOL_OUT
    out, outb, lse = c.prefill()
    size = 1 + c.dev[3].abs()[:, None]
    assert bool(((got[0] - out).abs() <= 2 * TOL_OUT * size).all())
    assert float((got[2] - lse).abs().max()) <= 2 * TOL_LSE
    import torch
    _same([got[1]], [got[0].to(torch.bfloat16)], "one rounding at the end")


def test_decode_does_not_depend_on_batch_pages_or_order():
    import torch
    ctx = [700, 1, 513, 2049, 128]
    c = Paged(ctx, 16, 4, 16, seed=20)
    want = c.decode(0)
    for order, page, seed in (([3, 0], 16, 21), ([4, 2, 1, 0, 3], 64, 22), ([2], 8, 23)):
        part = Problem([1] * len(order), [ctx[s] for s in order], 16, 4)
        part.q, part.lam = c.p.q[order], c.p.lam
        rows = np.concatenate([np.arange(c.p.ck[s], c.p.ck[s + 1]) for s in order])
        part.k, part.v = c.p.k[rows], c.p.v[rows]
        d = Paged.of(part, [ctx[s] for s in order], page, seed)
        for split in (0, 1, 3):
            _same(d.decode(split), [x[order] for x in want], (order, split))


@pytest.mark.parametrize("ctx,hq,hkv,page", [
    ([1], 32, 8, 16), ([127, 128, 129], 8, 8, 32), ([700, 1, 300], 40, 8, 64), ([3000, 5], 4, 1, 8), ([513], 8, 1, 16),
    ([260, 1025], 14, 2, 128), ([90, 2000, 16], 6, 2, 16), ([600] * 20, 16, 2, 16)])
def test_decode_has_the_same_bits_for_every_split(ctx, hq, hkv, page):
    c = Paged(ctx, hq, hkv, page, seed=hq + page)
    want = c.decode(1, ws=False)
    _near_prefill(c, want)
    for split in (0, 2, 3, 7, 64):
        _same(c.decode(split), want, split)
        _same(c.decode(split), want, (split, "again"))


@pytest.mark.parametrize("ctx,hq,hkv,page", [([1, 300, 129], 32, 8, 16), ([700], 8, 1, 64)])
def test_decode_is_the_definition(ctx, hq, hkv, page):
    c = Paged(ctx, hq, hkv, page, seed=2)
    out, _, lse = c.decode(0)
    for s in range(len(ctx)):
        q, k, v, a, _ = c.p.sequence(s)
        w, _, wl, t, _, tl = od.forward(q, k, v, c.p.lam, c.p.scale)
        _within(_np(out[a]), w, t, "out")
        _within(_np(lse[a]), wl, tl, "lse")


def test_long_sequences_spread_over_the_device():
    c = Paged([20000, 32768], 32, 8, 16, seed=3)
    want = c.decode(1)
    _near_prefill(c, want)
    for split in (0, 4, 9):
        _same(c.decode(split), want, split)


def test_decode_of_large_batches():
    g = np.random.default_rng(4)
    c = Paged(g.integers(1, 1400, 300).tolist(), 8, 2, 16, seed=4)
    want = c.decode(1)
    _near_prefill(c, want)
    for split in (0, 3):
        _same(c.decode(split), want, split)


def test_only_the_asked_outputs_are_written():
    import torch
    c = Paged([300, 40], 8, 2, 16, seed=5)
    ref = c.decode(0)
    for split in (0, 1, 3):
        out = torch.empty_like(ref[0])
        c.call(split, (out, None, None))
        outb = torch.empty_like(ref[1])
        c.call(split, (None, outb, None))
        rlk.rlk_attn_check_device_error()
        _same([out, outb], ref[:2], split)


def test_bad_pages_are_reported():
    c = Paged([300, 40], 8, 2, 16, seed=6)
    good = c.decode(0)
    table = c.table.clone()
    for bad in (-1, c.n_pages, 2 ** 31 - 1):
        c.table = table.clone()
        c.table[0, 3] = bad
        for split in (1, 0, 3):
            outs = c.outputs()
            c.call(split, outs)
            with pytest.raises(rlk.RlkError) as e:
                rlk.rlk_attn_check_device_error()
            assert e.value.status == 8
            _same([x[1:] for x in outs], [x[1:] for x in good], "the other sequence")
    c.table = table
    _same(c.decode(0), good)


def test_two_graphs_share_a_workspace():
    import torch
    c = Paged([3000, 40, 777], 32, 8, 16, seed=7)
    want = c.decode(1)
    runs = []
    for split in (0, 5):
        outs = c.outputs()
        c.call(split, outs)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.call(split, outs)
        runs.append((graph, outs))
    for turn in range(3):
        for graph, outs in (runs if turn % 2 else reversed(runs)):
            for x in outs:
                x.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            _same(outs, want, turn)
        _same(c.decode(0), want, "eager between")
    c.dev[0].copy_(-c.dev[0])  # another query at the captured address
    want = c.decode(1)
    for graph, outs in runs:
        graph.replay()
        torch.cuda.synchronize()
        _same(outs, want, "new query")


def test_other_streams_and_captured_training_steps():
    import torch
    p = Problem([300, 1, 129], [300, 1, 129], 8, 2, seed=16)
    dev = p.device()
    fwd, grads = p.forward(dev), p.backward(dev)
    dout = torch.from_numpy(p.dout).cuda().to(torch.bfloat16)
    ws = torch.empty(rlk.rlk_attn_workspace_size(p.params, rlk.RLK_OP_DIFF_BACKWARD, p.cq), dtype=torch.uint8, device="cuda")
    outs, got = [torch.empty_like(x) for x in fwd], [torch.empty_like(x) for x in grads]

    def step(stream=None):
        rlk.rlk_attn_diff_prefill(p.params, *dev, p.cq, p.ck, -1, *outs, stream=stream)
        rlk.rlk_attn_diff_backward(p.params, *dev, outs[0], outs[2], dout, outs[3], p.cq, -1, *got, ws, stream=stream)

    def clear():
        for x in (*outs, *got):
            x.fill_(float("nan"))
        torch.cuda.synchronize()

    clear()
    side = torch.cuda.Stream()
    step(side)
    side.synchronize()
    _same(outs, fwd, "stream")
    _same(got, grads, "stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        clear()
        graph.replay()
        torch.cuda.synchronize()
        _same(outs, fwd, "graph")
        _same(got, grads, "graph")


# ---------------------------------------------------------------- together

def test_a_conversation_from_prompt_to_token():
    """A prompt in two chunks and three tokens more: append (rotated maps) and
    prefill for the chunks, append and decode for the tokens.  The chunks' rows
    and the cache have the bits of one append and prefill over the whole, the
    tokens' rows agree with it."""
    import torch
    n, hq, hkv, page = 203, 16, 4, 16
    p = Problem([n], [n], hq, hkv, seed=17)
    q, k, v, lam = p.device()
    max_pages, n_pages = 16, 20
    rope = torch.from_numpy(rlk.rlk_attn_rope_table(1.0e6, 256)).cuda()
    table = torch.from_numpy(np.random.default_rng(17).permutation(n_pages)[:max_pages].astype(np.int32)).cuda()[None]

    def pools():
        x = torch.full((n_pages, page, hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        return x, x.clone()

    one = rlk.make_params(1, hq, hkv, softmax_scale=SCALE)

    def append(a, b, pool):
        qo, ko = torch.empty_like(q[a:b]), torch.empty_like(k[a:b])
        rlk.rlk_attn_cache_append(one, q[a:b], qo, k[a:b], ko, v[a:b], [0, b - a], [a], rope, 256, 64, *pool, n_pages, page,
                                  table, max_pages)
        return qo, ko

    whole = pools()
    qr, kr = append(0, n, whole)
    ref, ref_lse = torch.empty((n, hq, 128), device="cuda"), torch.empty((n, hq, 2), device="cuda")
    rlk.rlk_attn_diff_prefill(one, qr, kr, v, lam, [0, n], [0, n], -1, ref, None, None, ref_lse)

    pool, keys = pools(), []
    got, lse = torch.empty_like(ref), torch.empty_like(ref_lse)
    for a, b in ((0, 130), (130, 200)):
        qo, ko = append(a, b, pool)
        keys.append(ko)
        rlk.rlk_attn_diff_prefill(one, qo, torch.cat(keys), v[:b], lam, [0, b - a], [0, b], -1, got[a:b], None, None, lse[a:b])
    ws = torch.empty(rlk.rlk_attn_workspace_size(one, rlk.RLK_OP_DIFF_DECODE, None, [n]), dtype=torch.uint8, device="cuda")
    for t in range(200, n):
        qo, _ = append(t, t + 1, pool)
        rlk.rlk_attn_diff_decode(one, qo, lam, *pool, n_pages, page, table, max_pages, [t + 1], 0, got[t:t + 1], None,
                                 lse[t:t + 1], ws)
    rlk.rlk_attn_check_device_error()
    _same([got[:200], lse[:200], *pool], [ref[:200], ref_lse[:200], *whole])
    from tests.gpu_helpers import TOL_LSE, TOL_OUT
    assert bool(((got - ref).abs() <= 2 * TOL_OUT * (1 + lam.abs()[:, None])).all())
    assert float((lse - ref_lse).abs().max()) <= 2 * TOL_LSE
