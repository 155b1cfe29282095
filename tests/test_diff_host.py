"""Differential attention on the CPU: the FP64 definition against differences
and by hand, and what the calls refuse before any device work."""
import numpy as np
import pytest

import deterministic_context_attention_gb300 as rlk
import oracle.diff as od


@pytest.fixture(scope="module")
def lib():
    from deterministic_context_attention_gb300 import build as rbuild
    rbuild.build()
    return rlk.load()


# ---------------------------------------------------------------- the definition

def test_forward_by_hand():
    # two keys, one head: map 1 sees scores 0 and ln 3 (weights 1/4, 3/4), map 2 equal ones
    q, k, v = np.zeros((2, 1, 128)), np.zeros((2, 1, 128)), np.zeros((2, 1, 128))
    q[1, 0, 0], k[1, 0, 0] = 2.0, np.log(3.0)
    v[0, 0, 5], v[1, 0, 5] = 8.0, 16.0
    out, out2, lse, *_ = od.forward(q, k, v, [0.5], 0.5)
    assert np.isclose(out[0, 0, 5], 8 - 0.5 * 8) and np.isclose(out[1, 0, 5], (2 + 12) - 0.5 * 12)
    assert np.isclose(out2[1, 0, 5], 12) and np.allclose(lse[1, 0], [np.log(4), np.log(2)])


def test_backward_is_the_difference_quotient():
    g = np.random.default_rng(1)
    n, hq, hkv = 7, 4, 2
    q, dout = g.standard_normal((n, hq, 128)), g.standard_normal((n, hq, 128))
    k, v = (g.standard_normal((n, hkv, 128)) for _ in range(2))
    lam = g.standard_normal(hq)
    grads = od.backward(q, k, v, lam, dout, 0.125)[:4]
    xs = [q, k, v, lam]
    for i, (x, dx) in enumerate(zip(xs, grads)):
        for _ in range(12):
            at = tuple(g.integers(0, d) for d in x.shape)
            ends = []
            for step in (1e-5, -1e-5):
                ys = [y.copy() for y in xs]
                ys[i][at] += step
                ends.append((od.forward(*ys, 0.125)[0] * dout).sum())
            assert abs((ends[0] - ends[1]) / 2e-5 - dx[at]) < 1e-7 * (1 + abs(dx[at])), (i, at)


# ---------------------------------------------------------------- refusals

def _prefill(p, q=16, k=16, v=16, lam=16, cq=(0, 5), ck=(0, 9), rank=-1, out=16, outb=16, out2=16, lse=16):
    rlk.rlk_attn_diff_prefill(p, q, k, v, lam, list(cq), list(ck), rank, out, outb, out2, lse, stream=0)


def _decode(p, q=16, lam=16, kp=16, vp=16, n_pages=8, page=16, table=16, max_pages=4, seqlens=(50,), split=1, out=16,
            outb=None, lse=16, ws=16, ws_bytes=1 << 22):
    rlk.rlk_attn_diff_decode(p, q, lam, kp, vp, n_pages, page, table, max_pages, list(seqlens), split, out, outb, lse,
                             ws, ws_bytes, stream=0)


def _backward(p, q=16, k=16, v=16, lam=16, out=16, out2=16, dout=16, lse=16, cu=(0, 5), rank=-1, dq=16, dk=16, dv=16,
              dlam=16, ws=16, ws_bytes=1 << 22):
    rlk.rlk_attn_diff_backward(p, q, k, v, lam, out, out2, dout, lse, list(cu), rank, dq, dk, dv, dlam, ws, ws_bytes,
                               stream=0)


def _refused(call, status):
    with pytest.raises(rlk.RlkError) as e:
        call()
    assert e.value.status == status, rlk.rlk_attn_last_error()
    assert rlk.rlk_attn_last_error()


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(lam=None), dict(q=24), dict(k=24), dict(v=17), dict(lam=18),
    dict(cq=(1, 5)), dict(ck=(0, 4)), dict(cq=(0, -1)), dict(rank=1), dict(rank=-2), dict(out=None, outb=None),
    dict(out=24), dict(outb=24), dict(out2=24), dict(lse=18)])
def test_prefill_refuses(lib, kw):
    _refused(lambda: _prefill(rlk.make_params(1), **kw), 1)


@pytest.mark.parametrize("split", [0, 1, 3])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(lam=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(table=None), 1),
    (dict(q=24), 1), (dict(lam=17), 1), (dict(kp=24), 1), (dict(vp=24), 1), (dict(table=18), 1), (dict(n_pages=0), 1),
    (dict(max_pages=0), 1), (dict(page=4), 2), (dict(page=24), 2), (dict(page=256), 2), (dict(seqlens=(0,)), 1),
    (dict(seqlens=(65,)), 1), (dict(out=None), 1), (dict(out=24), 1), (dict(outb=24), 1), (dict(lse=18), 1),
    (dict(n_pages=2 ** 31 - 1), 2)])
def test_decode_refuses(lib, kw, status, split):
    _refused(lambda: _decode(rlk.make_params(1), split=split, **kw), status)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(lam=None), 1), (dict(out=None), 1),
    (dict(out2=None), 1), (dict(dout=None), 1), (dict(lse=None), 1), (dict(dq=None), 1), (dict(dk=None), 1),
    (dict(dv=None), 1), (dict(dlam=None), 1), (dict(q=24), 1), (dict(out2=24), 1), (dict(lse=20), 1),
    (dict(dlam=18), 1), (dict(dq=24), 1), (dict(ws=24), 1), (dict(cu=(1, 5)), 1), (dict(cu=(0, -1)), 1),
    (dict(rank=1), 1), (dict(ws=None), 3), (dict(ws_bytes=100), 3)])
def test_backward_refuses(lib, kw, status):
    _refused(lambda: _backward(rlk.make_params(1), **kw), status)


def test_refuses_shapes_and_splits(lib):
    for call in (_prefill, _decode, _backward):
        _refused(lambda: call(rlk.make_params(1, kv_block_size=64)), 2)
        _refused(lambda: call(rlk.make_params(1, head_dim=64)), 2)
        _refused(lambda: call(rlk.make_params(0)), 2)
        _refused(lambda: call(rlk.make_params(1, 30, 8)), 1)
        _refused(lambda: call(rlk.make_params(1, softmax_scale=float("nan"))), 1)
    for split in (0, 1, 2):
        _refused(lambda: _decode(rlk.make_params(1, 36, 4), split=split), 2)  # 9 query heads per KV head
    _refused(lambda: _decode(rlk.make_params(1), split=-1), 1)
    _refused(lambda: _decode(rlk.make_params(1), split=65), 1)
    for split in (0, 2):
        _refused(lambda: _decode(rlk.make_params(1), split=split, ws=None), 3)
        _refused(lambda: _decode(rlk.make_params(1), split=split, ws_bytes=100), 3)
        _refused(lambda: _decode(rlk.make_params(1), split=split, ws=24), 1)


def test_every_range_of_a_large_batch_is_checked_first(lib):
    p = rlk.make_params(300, 8, 2)
    ctx = np.full(300, 50)
    ctx[290] = 0
    for split in (1, 4):
        _refused(lambda: _decode(p, seqlens=ctx, split=split, ws_bytes=1 << 40), 1)
    cu = np.arange(301) * 2
    cu[280:] = 558
    cu[285] = 557
    _refused(lambda: _prefill(p, cq=cu, ck=cu), 1)
    _refused(lambda: _backward(p, cu=cu), 1)
    _refused(lambda: _backward(p, cu=np.arange(301) * 2, ws_bytes=1000), 3)
    # and a refused batch leaves the next call whole: no query is fine
    _prefill(rlk.make_params(2), q=0, k=0, v=0, cq=(0, 0, 0), ck=(0, 5, 9), out=0, outb=0, out2=0, lse=0)


def test_workspace_sizes(lib):
    p = rlk.make_params(2, 32, 8)
    # 520 bytes a (512-key segment, map of a query head), 8 a (sequence, KV head)
    assert rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DIFF_DECODE, None, [513, 1]) == 3 * 64 * 520 + 2 * 8 * 8
    # lse and Delta of two maps, the rows padded by 128
    assert rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DIFF_BACKWARD, [0, 3, 9]) == (9 + 128) * 32 * 4 * 4
    assert rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DIFF_DECODE, None, [129, 0]) == 0


def test_binding_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    host = torch.zeros((9, 32, 128), dtype=torch.bfloat16)
    for call in (_prefill, _decode, _backward):
        with pytest.raises(ValueError):
            call(rlk.make_params(1), q=host)
    for call in (lambda p: _prefill(p, cq=(0, 1), ck=(0, 1, 2)), lambda p: _prefill(p, cq=(0, 1, 2), ck=(0, 1)),
                 lambda p: _decode(p, seqlens=(50,)), lambda p: _backward(p, cu=(0, 1))):
        with pytest.raises(ValueError, match="host integers"):  # lists for one sequence of two
            call(rlk.make_params(2))
