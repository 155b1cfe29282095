"""Decode over the 8-bit pages at the ends of its ranges: scores far past what
FP32 holds to a unit, values whose scales differ by many powers of two inside
a block, products of large query rows and large scales.  Every row against
FP64 attention over the cached values, with a bound relative to the row's own
sum of |weight * value|."""
import numpy as np
import pytest

import oracle.qcache as oq
from deterministic_context_attention_gb300 import synth
from tests import qcache_helpers as qh
from tests.gpu_helpers import assert_bitwise, lib, torch_cuda

pytestmark = pytest.mark.gpu


def write_all(c, kv):
    for s, (k, v) in enumerate(kv):
        oq.write_tokens(c.k, c.ks, c.table[s], synth.bf16_round(k.astype(np.float32)))
        oq.write_tokens(c.v, c.vs, c.table[s], synth.bf16_round(v.astype(np.float32)))
    return c


def rows_of(c, s, g, ctx):
    """(k, v, V scale) of a sequence's cached tokens, float64."""
    at = np.arange(ctx)
    page, slot = c.table[s][at // c.page], at % c.page
    e = oq.e4m3_values()
    return (e[c.k[page, g, slot]] * c.ks[page, g].astype(np.float64)[:, None],
            e[c.v[page, g, slot]] * c.vs[page, g].astype(np.float64)[:, None], c.vs[page, g].astype(np.float64))


def check(got, c, q, ctx, scale, exact_scores, what):
    """A weight w = p sv of a block whose largest is A keeps 2^-19 of itself or
    2^-31 of A (four pieces of 4 bits, each 32 times finer, the last one's
    place fixed); 128 products are summed in FP32 (128 * 2^-23); the block sum
    of p is off by at most 128 * 2^-27 of a sum of at least 1, the reciprocal,
    the exponential and the folds by a few 2^-23 (together under 2^-18 here);
    an exponent x (base 2) carries three roundings, |x| 2^-22 of the weight.
    Scores of 128 FP32 products are off by at most 2^-22 sum |q k| * scale,
    unless they are equal or whole gaps apart (exact_scores)."""
    out, outb, lse = got
    hq, hkv = q.shape[1], c.k.shape[1]
    for s in range(len(ctx)):
        for h in range(hq):
            k, v, sv = rows_of(c, s, h // (hq // hkv), ctx[s])
            qr = q[s, h].astype(np.float64)
            x = (k @ qr) * scale
            mag = (np.abs(k) @ np.abs(qr)).max() * scale
            serr = 2.0 ** -22 * mag
            x2 = (x - x.max()) * np.log2(np.e)
            w = np.exp2(x2)
            l = w.sum()
            ref, ref_lse = (w @ v) / l, x.max() + np.log(l)
            big = np.array([(w * sv)[b - b % 128:b - b % 128 + 128].max() for b in range(ctx[s])])
            floor = np.minimum(w, 2.0 ** -31 * big / sv)
            each = w * (2.0 ** -16 + 2.0 ** -18 + np.abs(x2) * 2.0 ** -22 + (0.0 if exact_scores else 2 * serr)) + floor
            tol = (each @ np.abs(v)) / l + 1e-37
            e = np.abs(out[s, h] - ref)
            assert np.all(e <= tol), (f"{what}: sequence {s} head {h}: {np.sum(~(e <= tol))} elements, "
                                      f"{np.max(np.nan_to_num(e / tol, nan=np.inf)):.3g} times what they may be off")
            el = abs(lse[s, h] - ref_lse)
            assert el <= 4e-6 + 2.0 ** -21 * abs(ref_lse) + serr, f"{what}: lse of sequence {s} head {h}: {el:.3g}"
    assert np.array_equal(outb.view(np.uint32), synth.bf16_round(out).view(np.uint32)), f"{what}: BF16 output"


def both(c, q, ctx, scale):
    torch, rlk = torch_cuda(), lib()
    one = qh.decode(rlk, torch, c, q, ctx, q.shape[1], 1, scale=scale)
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, q.shape[1], 0, scale=scale), one, "even load")
    return one


# ---------------------------------------------------------------- large scores

@pytest.mark.parametrize("qe,ke", [(10, 10), (12, 13), (14, 14), (15, 15), (16, 17), (20, 20), (50, 50)])
def test_equal_keys_with_large_scores(qe, ke):
    # every key the same: the mean of V, however large the score
    g = np.random.default_rng([101, qe, ke])
    ctx, scale = [1, 32, 128, 300, 3001], 128 ** -0.5
    kv = []
    for n in ctx:
        row = synth.bf16_round(np.ldexp(g.standard_normal((1, 2, 128)), ke).astype(np.float32))
        kv.append((np.repeat(row, n, 0), g.standard_normal((n, 2, 128))))
    c = write_all(qh.empty_cache(ctx, 2, 16, seed=102), kv)
    q = synth.bf16_round(np.ldexp(g.standard_normal((len(ctx), 16, 128)), qe).astype(np.float32))
    check(both(c, q, ctx, scale), c, q, ctx, scale, True, f"2^{qe} 2^{ke}")


@pytest.mark.parametrize("qe,ke", [(12, 12), (14, 14), (15, 15), (18, 18), (40, 30)])
def test_largest_keys_with_large_scores(qe, ke):
    # gaps between the scores that leave one key, and its copies in other
    # blocks and segments, all the weight
    g = np.random.default_rng([103, qe])
    ctx, scale, hq = [40, 700, 3000], 128 ** -0.5, 4
    q = synth.bf16_round(np.ldexp(g.standard_normal((len(ctx), hq, 128)), qe).astype(np.float32))
    kv = []
    for s, n in enumerate(ctx):
        k = synth.bf16_round(np.ldexp(g.standard_normal((n, 1, 128)), ke).astype(np.float32))
        # elements below 2^-13 of a page's largest would be 0 in some pages
        k[np.abs(k) < 2.0 ** (ke - 9)] = 0.0
        for h in range(hq):
            top = int(np.argmax(k[:, 0].astype(np.float64) @ q[s, h]))
            for at in (n // 3 + h, n - 1 - h):
                k[at] = k[top]
        kv.append((k, g.standard_normal((n, 1, 128))))
    c = write_all(qh.empty_cache(ctx, 1, 16, seed=104), kv)
    for s, n in enumerate(ctx):  # what the inputs must be for exact_scores
        k, _, _ = rows_of(c, s, 0, n)
        for h in range(hq):
            x = (k @ q[s, h].astype(np.float64)) * scale
            serr = 2.0 ** -22 * scale * (np.abs(k) @ np.abs(q[s, h].astype(np.float64))).max()
            assert np.all((x == x.max()) | (x < x.max() - 150 - 2 * serr))
    check(both(c, q, ctx, scale), c, q, ctx, scale, True, f"2^{qe} 2^{ke}")


# ---------------------------------------------------------------- V scales

@pytest.mark.parametrize("page,heads", [(16, (4, 1)), (8, (8, 1)), (32, (7, 1)), (16, (3, 3))])
@pytest.mark.parametrize("gap,e", [(192, 20), (192, 24), (192, 60), (192, 100), (30, 40), (10, 30), (60, 100),
                                   (60, -100), (192, -110)])
def test_value_scales_of_unattended_pages(page, heads, gap, e):
    # pages whose values are 2^e times the others', `gap` below in score: the
    # rows that attend to the others keep their bits, the rows that attend to
    # these, or to all, are right as well
    g = np.random.default_rng([105, gap, e + 200])
    hq, hkv = heads
    ctx = [127, 300, 1100]
    kv = []
    for n in ctx:
        level = np.broadcast_to(g.choice([0.0, -0.5, -1.0, -1.75], (n, 1, 1)), (n, hkv, 1)).copy()
        v = g.standard_normal((n, hkv, 128))
        apart = np.isin(np.arange(n) // page % 5, (2, 3))
        level[apart] -= gap
        v[apart] = np.ldexp(v[apart], e)
        kv.append((np.broadcast_to(level, (n, hkv, 128)), v))
    c = write_all(qh.empty_cache(ctx, hkv, page, seed=106), kv)
    sign = np.array([1.0, -1.0, 0.0, 0.5, 1.0, -0.25, 2.0, 0.125])[np.arange(hq) % 8]
    q = np.broadcast_to(sign[None, :, None], (len(ctx), hq, 128)).astype(np.float32).copy()
    check(both(c, q, ctx, 2.0 ** -7), c, q, ctx, 2.0 ** -7, False, f"gap {gap} 2^{e}")


def test_values_at_the_smallest_scale():
    # V scales of 2^-120 (values under 2^-112), beside pages of zeros
    g = np.random.default_rng(107)
    ctx = [50, 400]
    kv = []
    for n in ctx:
        v = np.ldexp(g.standard_normal((n, 2, 128)), -116)
        v[32:48] = 0.0
        kv.append((g.standard_normal((n, 2, 128)), v))
    c = write_all(qh.empty_cache(ctx, 2, 16, seed=108), kv)
    assert c.vs[c.table[0, 0]].max() <= 2.0 ** -119
    q = synth.bf16_round(g.standard_normal((2, 8, 128)).astype(np.float32))
    check(both(c, q, ctx, 128 ** -0.5), c, q, ctx, 128 ** -0.5, False, "smallest scale")


# ---------------------------------------------------------------- large scales

@pytest.mark.parametrize("e", [0, 16, 30, 100])
def test_zero_products_of_large_rows_and_large_scales(e):
    # query rows up to 2^(20 + e) over K pages up to 2^(120 - e) in other
    # dimensions: what is left is scores of up to 3 * 2^120, or 0, and a
    # softmax scale that brings them to 3
    g = np.random.default_rng([109, e])
    ctx, scale = [60, 260], 2.0 ** -120
    kv = []
    for n in ctx:
        k = np.zeros((n, 1, 128))
        k[:, 0, 1] = np.ldexp(g.integers(-3, 4, n).astype(np.float64), 110 - e)
        k[::3, 0, 2] = 2.0 ** (123 - e)
        k[:, 0, 3] = np.ldexp(g.standard_normal(n), 115 - e)
        kv.append((k, g.standard_normal((n, 1, 128))))
    c = write_all(qh.empty_cache(ctx, 1, 16, seed=110), kv)
    assert c.ks[c.table[0, 0], 0] == 2.0 ** (116 - e)
    q = np.zeros((2, 4, 128), np.float32)
    q[:, :, 0] = 2.0 ** (20 + e)
    q[:, 1:, 1] = 2.0 ** (10 + e)
    q[:, 2, 0] *= -1
    q[:, 3] *= 2.0 ** -20
    check(both(c, q, ctx, scale), c, q, ctx, scale, False, f"e {e}")


# ---------------------------------------------------------------- nothing to do

def test_calls_without_a_token_change_nothing():
    # a step in which no sequence has a new token: tensors of no rows
    torch, rlk = torch_cuda(), lib()
    c = qh.filled([20, 33], 2, 16, seed=111, spread=False)
    dev = c.device()
    p = rlk.make_params(2, 2, 2)
    pool = (*dev[:4], c.n_pages, 16, dev[4], dev[4].shape[1])
    k, v = (torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rlk.rlk_attn_qcache_write(p, k, v, [0, 0, 0], [20, 33], None, 0, *pool)
    rlk.rlk_attn_qcache_read(p, *pool, [0, 0, 0], None, k, v)
    rlk.rlk_attn_check_device_error()
    for d, a in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
        assert np.array_equal(d.cpu().numpy().view(np.uint8), a.view(np.uint8))
