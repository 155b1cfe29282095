"""Differential attention where values are extreme (scores that are NaN, infinite or large)
and where sequences are long enough that accumulators leave more than once;
groups of every size in the decode."""
import numpy as np
import pytest

import oracle.diff as od
from tests.test_gpu_diff import Paged, Problem, _near_prefill, _np, _same, _within

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _map_slice(which):
    return slice(0, 128) if which == "both" else slice(64 * which, 64 * which + 64)


def _check_nan_rows(got, clean, first, which, what):
    """Rows from `first` on are NaN in the maps that see a NaN key (and only there),
    the rows before them have the bits of the run without it."""
    out, outb, out2, lse = got
    _same([x[:first] for x in got], [x[:first] for x in clean], what)
    maps = (0, 1) if which == "both" else (which,)
    assert not np.isfinite(_np(out[first:])).any() and not np.isfinite(_np(outb[first:])).any(), what
    for m in range(2):
        if m in maps:
            assert not np.isfinite(_np(lse[first:, :, m])).any(), (what, m)
        else:
            _same([lse[first:, :, m]], [clean[3][first:, :, m]], (what, m))
    if 1 in maps:
        assert not np.isfinite(_np(out2[first:])).any(), what
    else:
        _same([out2[first:]], [clean[2][first:]], what)


@pytest.mark.parametrize("which", [0, 1, "both"])
@pytest.mark.parametrize("first,last", [(0, 1), (5, 6), (127, 128), (128, 129), (200, 202), (256, 257), (128, 256), (384, 385)])
def test_a_nan_key_reaches_every_row_that_sees_it(first, last, which):
    # keys first .. last - 1 are NaN: a row may see one key of a block alone
    # (first a multiple of 128), or a whole block of NaN
    p = Problem([400], [400], 8, 2, seed=31)
    clean = p.forward()
    p.k[first:last, :, _map_slice(which)] = NAN
    _check_nan_rows(p.forward(), clean, first, which, (first, last, which))


@pytest.mark.parametrize("which", [0, "both"])
def test_a_nan_key_reaches_the_rows_of_a_chunk(which):
    p = Problem([90, 3], [400, 130], 8, 1, seed=32)  # rows 310 .. 399 and 127 .. 129
    clean = p.forward()
    p.k[128:256, :, _map_slice(which)] = NAN  # whole block, long past
    p.k[400 + 128, :, _map_slice(which)] = NAN
    got = p.forward()
    _check_nan_rows([x[:90] for x in got], [x[:90] for x in clean], 0, which, "first")
    _check_nan_rows([x[90:] for x in got], [x[90:] for x in clean], 1, which, "second")


def test_a_nan_query_is_its_own_rows_alone():
    import torch
    p = Problem([300], [300], 8, 2, seed=33)
    clean = p.forward()
    p.q[[0, 128, 255], 3] = NAN
    got = p.forward()
    keep = torch.ones(300, 8, dtype=torch.bool)
    keep[[0, 128, 255], 3] = False
    _same([x[keep] for x in got], [x[keep] for x in clean])
    assert not any(np.isfinite(_np(x[~keep])).any() for x in got)


@pytest.mark.parametrize("ctx,at", [([400, 129], (128, 129)), ([400, 300], (128, 256)), ([1100, 513], (512, 513)), ([129, 70], (0, 1))])
def test_a_nan_key_reaches_the_decoded_row(ctx, at):
    p = Problem([1] * 2, ctx, 8, 2, seed=34)
    clean = Paged.of(p, ctx, 16, 34).decode(0)
    p.k[at[0]:at[1]] = NAN  # of the first sequence
    c = Paged.of(p, ctx, 16, 34)
    for split in (0, 1, 3):
        got = c.decode(split)
        assert not any(np.isfinite(_np(x[0])).any() for x in got), split
        _same([x[1:] for x in got], [x[1:] for x in clean], split)


def test_a_nan_key_reaches_the_gradients():
    # every row from key 200 on is NaN, and with it every key's gradient; the
    # queries of the tiles before it see nothing of it
    p = Problem([400], [400], 8, 2, seed=35)
    clean = p.backward()
    p.k[200] = NAN
    fwd = p.forward()
    dq, dk, dv, dlam = p.backward(fwd=fwd)
    _same([dq[:128]], [clean[0][:128]])
    assert not any(np.isfinite(_np(x)).any() for x in (dq[200:], dk, dv, dlam))


def test_scores_of_minus_infinity_weigh_nothing():
    # as scores of -1e7 do, bit for bit, in some keys or in all of a block
    p = Problem([500], [500], 8, 2, seed=36)
    p.q[..., 0] = np.abs(p.q[..., 0]) + 1.0
    p.q[..., 64] = np.abs(p.q[..., 64]) + 1.0
    rows = slice(400, 500)
    keys = [3, 127, 300, *range(128, 256)]
    runs = []
    for low in (-1e8, -np.inf):
        p.k[keys, :, 0] = p.k[keys, :, 64] = low
        runs.append([x[rows] for x in p.forward()])
    _same(runs[1], runs[0])
    p.k[:128, :, 0] = p.k[:128, :, 64] = -np.inf  # the first block, and the first row of all
    got = p.forward()
    assert not np.isfinite(_np(got[0][:128])).any()
    p.k[:128, :, 0] = p.k[:128, :, 64] = -1e8
    p.k[128:256, :, 0] = p.k[128:256, :, 64] = -1e8
    _same([x[rows] for x in got], [x[rows] for x in p.forward()])


def _large_scores(n, hq, hkv, seed, size):
    """Scores of one product a map: a small integer times size / 8, exact in FP32.
    Key j's integers of either map come back beside the problem."""
    p = Problem([n], [n], hq, hkv, seed=seed)
    g = np.random.default_rng([seed, 3])
    p.q[:], p.k[:] = 0.0, 0.0
    p.q[..., 5] = p.q[..., 70] = 2.0 ** 20
    level = g.integers(-60, 61, (n, hkv, 2))
    p.k[..., 5], p.k[..., 70] = level[..., 0] * (size / 2.0 ** 20), level[..., 1] * (size / 2.0 ** 20)
    return p, level


def _check_one_hot(p, level, rows, out, out2, lse, size):
    """The softmax of scores that far apart: the mean of V over the keys that have the
    largest (2^-15 of the values' sizes, the sums' roundings; lse three roundings)."""
    g = p.hq // p.hkv
    v = p.v.astype(np.float64)
    for i, row in enumerate(rows):
        for h in range(p.hq):
            o, t = [], []
            for m in range(2):
                lv = level[:row + 1, h // g, m]
                top = np.flatnonzero(lv == lv.max())
                o.append(v[top, h // g].mean(0))
                t.append(2.0 ** -15 * np.abs(v[top, h // g]).mean(0))
                s = float(lv.max()) * size * p.scale
                _within(lse[i, h, m], s + np.log(len(top)), 2.0 ** -22 * (abs(s) + 8), ("lse", row, h, m))
            _within(out2[i, h], o[1], t[1], ("out2", row, h))
            lam = float(p.lam[h])
            _within(out[i, h], o[0] - lam * o[1], t[0] + abs(lam) * t[1] + 2.0 ** -23 * np.abs(o[0] - lam * o[1]), ("out", row, h))


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 25])
def test_large_scores(size):
    # up to 160 / 8 of size, 2^29.3: the prefill takes sizes below 2^30
    p, level = _large_scores(700, 4, 2, 37, size)
    out, _, out2, lse = (_np(x) for x in p.forward())
    rows = [0, 1, 127, 128, 300, 511, 699]
    _check_one_hot(p, level, rows, out[rows], out2[rows], lse[rows], size)
    level[:] = level - 100  # below zero throughout
    p.k[..., 5], p.k[..., 70] = level[..., 0] * (size / 2.0 ** 20), level[..., 1] * (size / 2.0 ** 20)
    out, _, out2, lse = (_np(x) for x in p.forward())
    _check_one_hot(p, level, rows, out[rows], out2[rows], lse[rows], size)


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 29, 2.0 ** 33, 2.0 ** 100])
def test_decode_of_large_scores(size):
    p, level = _large_scores(1300, 4, 2, 38, size)
    one = Problem([1], [1300], 4, 2, seed=38)
    one.q, one.k, one.v, one.lam = p.q[-1:], p.k, p.v, p.lam
    for split in (0, 1):
        out, _, lse = (_np(x) for x in Paged.of(one, [1300], 16, 38).decode(split))
        g, v = 2, p.v.astype(np.float64)
        for h in range(4):
            o, t = [], []
            for m in range(2):
                lv = level[:, h // g, m]
                top = np.flatnonzero(lv == lv.max())
                o.append(v[top, h // g].mean(0))
                t.append(2.0 ** -15 * np.abs(v[top, h // g]).mean(0))
                s = float(lv.max()) * size * p.scale
                _within(lse[0, h, m], s + np.log(len(top)), 2.0 ** -22 * (abs(s) + 8), ("lse", h, m))
            lam = float(p.lam[h])
            _within(out[0, h], o[0] - lam * o[1], t[0] + abs(lam) * t[1] + 2.0 ** -23 * np.abs(o[0] - lam * o[1]), ("out", h))


# ---------------------------------------------------------------- long sequences

def _definition(p):
    """Gradients of whole sequences in FP64 on the device, and for dlambda the sums
    of |dO| |O_2| over a head's rows."""
    import torch
    q, k, v, lam = (x.double() for x in p.device())
    do = torch.from_numpy(p.dout).cuda().double()
    g = p.hq // p.hkv
    dq, dk, dv, dlam, size = (torch.zeros_like(x) for x in (q, k, v, lam, lam))
    for s in range(len(p.q_lens)):
        a = slice(int(p.cq[s]), int(p.cq[s + 1]))
        hidden = torch.ones((a.stop - a.start,) * 2, dtype=torch.bool, device="cuda").triu(1)
        for h in range(p.hq):
            kv = h // g
            dp = do[a, h] @ v[a, kv].T
            for m, c in ((0, 1.0), (1, -float(lam[h]))):
                at = slice(64 * m, 64 * m + 64)
                w = torch.softmax((q[a, h, at] @ k[a, kv, at].T * p.scale).masked_fill(hidden, -np.inf), 1)
                delta = (w * dp).sum(1, keepdim=True)
                ds = c * w * (dp - delta)
                dq[a, h, at] = p.scale * (ds @ k[a, kv, at])
                dk[a, kv, at] += p.scale * (ds.T @ q[a, h, at])
                dv[a, kv] += c * (w.T @ do[a, h])
                if m:
                    dlam[h] -= delta.sum()
                    size[h] += (do[a, h].norm(dim=1) * (w @ v[a, kv]).norm(dim=1)).sum()
    return dq, dk, dv, dlam, size


# relative 2-norm: an accumulator takes 128 products at the most, each of which may
# lose 2^-23 of the sum; P and dS in two pieces 2^-18, S and dP of 4 and 8 products,
# the exponential and the saved log sum (of size 8) less than 2^-18 more.  (With the
# sums of a group of 8 in one accumulator dK and dV are 2.7e-5 off at 1024 tokens and
# 6e-5 at 2200, as they are 4e-6.)
GRAD_LONG_REL_L2 = 128 * 2.0 ** -23 + 2.0 ** -17


@pytest.mark.parametrize("lens,hq,hkv", [([1024], 8, 1), ([1025], 4, 2), ([1100, 300], 8, 4), ([2200], 8, 1), ([2049, 129], 4, 4)])
def test_backward_of_long_sequences_is_the_definition(lens, hq, hkv):
    # dQ leaves its accumulator every 8 key tiles, dV and dK theirs every 8 query tiles of a head
    p = Problem(lens, lens, hq, hkv, seed=39)
    got = p.backward()
    want = _definition(p)
    for x, w, name in zip(got[:3], want[:3], ("dq", "dk", "dv")):
        assert float((x - w).norm() / w.norm()) <= GRAD_LONG_REL_L2, name
        # a lost or doubled tile of any row, head by head, whatever the rows' sizes
        rows = (x - w).norm(dim=2) / w.norm(dim=2).clamp_min(float(w.norm(dim=2).mean()) * 2.0 ** -4)
        assert float(rows.max()) <= 16 * GRAD_LONG_REL_L2, name
    # Delta_2 = dO . O_2: O_2 within 2^-17 of its norm (as in the forward), the sums' roundings less than that
    assert bool(((got[3] - want[3]).abs() <= 2.0 ** -16 * want[4]).all())


@pytest.mark.parametrize("cp,layout", [(2, 1), (3, 0)])
def test_ranks_of_long_sequences(cp, layout):
    # query tiles that do not start on a multiple of 128
    lens = [2200, 1030]
    p = Problem(lens, lens, 4, 2, seed=40)
    dev = p.device()
    fwd = p.forward(dev)
    want = p.backward(dev, fwd)
    _same(p.forward(dev, ranks=range(cp), cp=cp, layout=layout), fwd, "forward")
    _same(p.backward(dev, fwd, ranks=range(cp), cp=cp, layout=layout), want, "backward")


# ---------------------------------------------------------------- groups of the decode

@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode_of_every_group_size(group):
    c = Paged([300, 1, 1409], 2 * group, 2, 16, seed=41 + group)
    want = c.decode(1, ws=False)
    _near_prefill(c, want)
    for split in (0, 2, 5):
        _same(c.decode(split), want, split)
    q, k, v, a, _ = c.p.sequence(0)
    w, _, wl, t, _, tl = od.forward(q, k, v, c.p.lam, c.p.scale)
    _within(_np(want[0][a]), w, t, "out")
    _within(_np(want[2][a]), wl, tl, "lse")
