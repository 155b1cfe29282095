"""The 8-bit cache without a GPU: the oracle's codes against hand-worked ones,
the page's independence of the calls that wrote it (the rescaling rule), and
the entry points' refusals, all before any launch."""
import numpy as np
import pytest

import deterministic_context_attention_gb300 as rlk
import oracle.qcache as oq
from deterministic_context_attention_gb300 import build as rbuild
from deterministic_context_attention_gb300 import synth


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rlk.load()


def test_e4m3_values():
    v = oq.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7E] == 448.0 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9
    assert v[0xB8] == -1.0 and np.isnan(v[0x7F]) and np.isnan(v[0xFF])


@pytest.mark.parametrize("x,want", [
    (1.0, 1.0), (1.0625, 1.0), (1.1875, 1.25), (1.0703125, 1.125), (-1.9375, -2.0), (1.9296875, 1.875),
    (3.0e38, 1.75 * 2.0 ** 127), (3.3895313892515355e38, 1.875 * 2.0 ** 127), (2.0 ** -127, 0.0),
    (-2.0 ** -126, -2.0 ** -126), (0.0, 0.0),
])
def test_q4(x, want):
    assert oq.q4(np.array([x]))[0] == want


def test_page_by_hand():
    # the largest value 3 = 1.5 * 2^1 sets e = 1 - 7 = -6: codes up to 192
    rows = np.zeros((2, 128))
    rows[0, :4] = [3.0, -1.0, 2.0 ** -12, 2.0 ** -12 * 1.9375]
    rows[1, :3] = [2.0 ** -11, np.inf, np.nan]
    s = oq.page_scale(rows)
    assert s == 2.0 ** -6
    v = oq.e4m3_values()[oq.page_codes(rows, s)]
    assert list(v[0, :4]) == [192.0, -64.0, 2.0 ** -6, 2.0 ** -5]
    assert v[1, 0] == 2.0 ** -5 and np.isnan(v[1, 1]) and np.isnan(v[1, 2])
    # below 2^-6 of the scale: +0
    assert oq.page_codes(np.full((1, 128), -1.8125 * 2.0 ** -13), s)[0, 0] == 0
    assert oq.page_scale(np.zeros((3, 128))) == 2.0 ** -120


def _rescaled(code, d):
    """A page's earlier code under a scale 2^d times larger."""
    m = int(code) & 0x7F
    if m == 0x7F:
        return code
    m -= 8 * d
    return (int(code) & 0x80) | m if m >= 8 else 0


def test_rescaled_codes_are_the_codes_of_the_larger_scale():
    # the rule that makes a page independent of the calls that wrote it
    g = np.random.default_rng(5)
    x = synth.bf16_round((g.standard_normal((64, 128)) * np.exp2(g.integers(-18, 3, (64, 128)))).astype(np.float32))
    s = oq.page_scale(x)
    for d in (0, 1, 3, 9, 14, 40):
        want = oq.page_codes(x, s * 2.0 ** d)
        got = np.array([_rescaled(c, d) for c in oq.page_codes(x, s).ravel()], np.uint8).reshape(want.shape)
        assert np.array_equal(got, want), d


def test_quantisation_error_bound():
    # half a step of 3 mantissa bits, or a value below 2^-13 of the largest
    g = np.random.default_rng(6)
    x = synth.bf16_round(g.standard_normal((128, 128)).astype(np.float32))
    s = oq.page_scale(x)
    v = oq.e4m3_values()[oq.page_codes(x, s)] * s
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -13 * np.abs(x).max()))


# ---------------------------------------------------------------- refusals

def _write(p, k=16, v=16, cu=(0, 5), pos=(3,), table=16, rope=None, max_pos=0, kp=16, vp=16, ks=16, vs=16, n_pages=8,
           page=16, max_pages=4):
    rlk.rlk_attn_qcache_write(p, k, v, list(cu), None if pos is None else list(pos), rope, max_pos, kp, vp, ks, vs,
                              n_pages, page, table, max_pages, stream=0)


def _read(p, k=16, v=16, cu=(0, 5), pos=(3,), table=16, kp=16, vp=16, ks=16, vs=16, n_pages=8, page=16, max_pages=4):
    rlk.rlk_attn_qcache_read(p, kp, vp, ks, vs, n_pages, page, table, max_pages, list(cu),
                             None if pos is None else list(pos), k, v, stream=0)


def _decode(p, q=16, seqlens=(50,), split=1, table=16, rope=None, max_pos=0, kp=16, vp=16, ks=16, vs=16, n_pages=8,
            page=16, max_pages=4, out=16, outb=None, lse=16, ws=16, ws_bytes=1 << 20):
    rlk.rlk_attn_decode_qcache(p, q, kp, vp, ks, vs, n_pages, page, table, max_pages, list(seqlens), split, rope,
                               max_pos, out, outb, lse, ws, ws_bytes, stream=0)


BAD_CACHE = [(dict(kp=None), 1), (dict(vp=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(table=None), 1),
             (dict(kp=24), 1), (dict(vp=17), 1), (dict(ks=18), 1), (dict(table=17), 1), (dict(n_pages=0), 1),
             (dict(max_pages=0), 1), (dict(page=4), 2), (dict(page=24), 2), (dict(page=256), 2)]


def _refused(call, status):
    with pytest.raises(rlk.RlkError) as e:
        call()
    assert e.value.status == status, rlk.rlk_attn_last_error()
    assert rlk.rlk_attn_last_error()


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=24), 1), (dict(cu=(1, 5)), 1), (dict(cu=(0, -1)), 1),
    (dict(pos=(-1,)), 1), (dict(pos=(60,)), 1), (dict(cu=(0, 65), pos=None), 1),
    (dict(pos=(2 ** 31 - 100,), max_pages=2 ** 31 - 1), 1),
    (dict(rope=16, max_pos=7), 1), (dict(rope=18, max_pos=100), 1)])
def test_write_refuses(lib, kw, status):
    _refused(lambda: _write(rlk.make_params(1), **kw), status)


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(v=24), 1), (dict(cu=(1, 5)), 1), (dict(cu=(0, -1)), 1),
    (dict(pos=(-1,)), 1), (dict(pos=(60,)), 1)])
def test_read_refuses(lib, kw, status):
    _refused(lambda: _read(rlk.make_params(1), **kw), status)


@pytest.mark.parametrize("split", [0, 1, 3])
@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(q=None), 1), (dict(q=24), 1), (dict(seqlens=(0,)), 1), (dict(seqlens=(65,)), 1), (dict(out=None), 1),
    (dict(out=None, outb=24), 1), (dict(lse=18), 1), (dict(rope=16, max_pos=49), 1), (dict(rope=18, max_pos=100), 1)])
def test_decode_refuses(lib, kw, status, split):
    _refused(lambda: _decode(rlk.make_params(1), split=split, **kw), status)


def test_decode_refuses_shapes_and_splits(lib):
    _refused(lambda: _decode(rlk.make_params(1, kv_block_size=64)), 2)
    _refused(lambda: _decode(rlk.make_params(1, 36, 4)), 2)  # 9 query heads per KV head
    _refused(lambda: _decode(rlk.make_params(1), split=-1), 1)
    _refused(lambda: _decode(rlk.make_params(1), split=65), 1)
    _refused(lambda: _decode(rlk.make_params(1), split=2, ws=None), 3)
    _refused(lambda: _decode(rlk.make_params(1), split=0, ws_bytes=100), 3)
    _refused(lambda: _decode(rlk.make_params(1), split=2, ws=24), 1)
    for call in (_write, _read, _decode):
        _refused(lambda: call(rlk.make_params(1, head_dim=64)), 2)
        _refused(lambda: call(rlk.make_params(0)), 2)


def test_every_range_of_a_large_batch_is_checked_first(lib):
    p = rlk.make_params(300, 8, 2)
    ctx = np.full(300, 50)
    ctx[290] = 0
    for split in (1, 4):
        _refused(lambda: _decode(p, seqlens=ctx, split=split, ws_bytes=1 << 40), 1)
    cu = np.arange(301) * 2
    pos = np.full(300, 3)
    pos[280] = 63  # tokens 63 and 64 of 64
    _refused(lambda: _write(p, cu=cu, pos=pos), 1)
    _refused(lambda: _read(p, cu=cu, pos=pos), 1)
    # and a refused batch leaves the next call whole: nothing to write is fine
    _write(rlk.make_params(2), cu=(0, 0, 0), pos=(0, 64))
    _read(rlk.make_params(2), cu=(0, 0, 0), pos=None)


def test_calls_without_a_token_take_empty_tensors(lib):
    # an empty tensor's address is NULL; one with rows is still refused
    for n, pos in ((2, (5, 64)), (300, None)):
        p, cu = rlk.make_params(n), (0,) * (n + 1)
        _write(p, k=0, v=0, cu=cu, pos=pos)
        _read(p, k=0, v=0, cu=cu, pos=pos)
    cu = [0] * 290 + [1] * 11  # the second range of sequences has it
    for call in (_write, _read):
        _refused(lambda: call(rlk.make_params(300), k=0, v=0, cu=cu, pos=None), 1)
        _refused(lambda: call(rlk.make_params(2), k=0, cu=(0, 0, 1), pos=None), 1)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros((5, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _write(rlk.make_params(1), k=k, v=k)


@pytest.mark.parametrize("call", [
    lambda p: _write(p, cu=(0, 1), pos=(0, 0)), lambda p: _write(p, cu=(0, 1, 2), pos=(0,)),
    lambda p: _read(p, cu=(0, 1), pos=None), lambda p: _read(p, cu=(0, 1, 2), pos=(0,)),
    lambda p: _decode(p, seqlens=(50,)),
    lambda p: rlk.rlk_attn_decode_qcache(p, 16, 16, 16, 16, 16, 8, 16, 16, 4, np.array([50], np.int32), 1, None, 0, 16,
                                         None, 16, stream=0)])
def test_binding_refuses_short_lists(call):
    # two sequences, lists for one: the library would read past their ends
    with pytest.raises(ValueError, match="host integers"):
        call(rlk.make_params(2))
