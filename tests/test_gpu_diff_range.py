"""Differential attention where values are extreme: scores that are NaN or infinite."""
import numpy as np
import pytest

from tests.test_gpu_diff import Paged, Problem, _np, _same

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
