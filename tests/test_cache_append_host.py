"""rlk_attn_cache_append: what it refuses, before any device work (CPU)."""
import numpy as np
import pytest

import deterministic_context_attention_gb300 as rlk


@pytest.fixture(scope="module", autouse=True)
def lib():
    from deterministic_context_attention_gb300 import build as rbuild
    rbuild.build()
    return rlk.load()


def _append(p, q=None, q_out=None, k=16, k_out=None, v=16, cu=(0, 5), pos=(3,), rope=None, max_pos=0, width=128, kp=16,
            vp=16, n_pages=8, page=16, table=16, max_pages=4):
    rlk.rlk_attn_cache_append(p, q, q_out, k, k_out, v, list(cu), None if pos is None else list(pos), rope, max_pos,
                              width, kp, vp, n_pages, page, table, max_pages, stream=0)


def _refused(call, status):
    with pytest.raises(rlk.RlkError) as e:
        call()
    assert e.value.status == status, rlk.rlk_attn_last_error()
    assert rlk.rlk_attn_last_error()


ROPE = dict(rope=16, max_pos=100)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=24), 1), (dict(v=17), 1), (dict(kp=None), 1), (dict(vp=None), 1),
    (dict(kp=24), 1), (dict(vp=8), 1), (dict(table=None), 1), (dict(table=18), 1), (dict(n_pages=0), 1),
    (dict(max_pages=0), 1), (dict(page=4), 2), (dict(page=24), 2), (dict(page=256), 2), (dict(cu=(1, 5)), 1),
    (dict(cu=(0, -1)), 1), (dict(pos=(-1,)), 1), (dict(pos=(60,)), 1), (dict(cu=(0, 65), pos=None), 1),
    (dict(pos=(2 ** 31 - 3,), max_pages=2 ** 31 - 1, page=128), 1),
    (dict(q=16, **ROPE), 1), (dict(q_out=16, **ROPE), 1), (dict(q=16, q_out=16), 1), (dict(k_out=16), 1),
    (dict(q=24, q_out=16, **ROPE), 1), (dict(q=16, q_out=24, **ROPE), 1), (dict(k_out=24, **ROPE), 1),
    (dict(rope=16, max_pos=7), 1), (dict(rope=24, max_pos=100), 1), (dict(width=32, **ROPE), 2),
    (dict(width=0, **ROPE), 2)])
def test_refuses(kw, status):
    _refused(lambda: _append(rlk.make_params(1), **kw), status)


def test_refuses_shapes():
    _refused(lambda: _append(rlk.make_params(1, head_dim=64)), 2)
    _refused(lambda: _append(rlk.make_params(0)), 2)
    _refused(lambda: _append(rlk.make_params(1, 30, 8)), 1)
    _refused(lambda: _append(rlk.make_params(1, kv_block_size=64), page=128), 2)


def test_every_range_of_a_large_batch_is_checked_first():
    p = rlk.make_params(300, 8, 2)
    cu, pos = np.arange(301) * 2, np.full(300, 3)
    pos[280] = 63  # tokens 63 and 64 of 64
    _refused(lambda: _append(p, cu=cu, pos=pos), 1)
    _append(rlk.make_params(2), cu=(0, 0, 0), pos=(0, 64))  # and the next call is whole


def test_calls_without_a_token_take_empty_tensors():
    for n, pos in ((2, (5, 64)), (300, None)):
        _append(rlk.make_params(n), k=0, v=0, cu=(0,) * (n + 1), pos=pos)
    _refused(lambda: _append(rlk.make_params(300), k=0, v=0, cu=[0] * 290 + [1] * 11, pos=None), 1)


def test_binding_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):  # a host tensor
        _append(rlk.make_params(1), k=torch.zeros((5, 8, 128), dtype=torch.bfloat16))
    for kw in (dict(cu=(0, 1), pos=(0, 0)), dict(cu=(0, 1, 2), pos=(0,))):  # lists for one sequence of two
        with pytest.raises(ValueError, match="host integers"):
            _append(rlk.make_params(2), **kw)
