"""The 8-bit paged KV cache on the GPU: pages against the definition byte for
byte, whatever calls wrote them; read-back; decode against FP64 attention over
the cached values and bit for bit against itself across splits, batches and
page orders; the three together as a serving loop uses them."""
import numpy as np
import pytest

import oracle
import oracle.qcache as oq
from deterministic_context_attention_gb300 import synth
from tests import qcache_helpers as qh
from tests.gpu_helpers import assert_bitwise, lib, torch_cuda

pytestmark = pytest.mark.gpu


def run_calls(c, kv, steps, rope=None, max_pos=0):
    """Write the tokens kv into cache c in calls: each step gives every
    sequence's end position after it.  Returns (k, v, k_scale, v_scale)."""
    torch, rlk = torch_cuda(), lib()
    dev = c.device()
    n, hkv = len(kv), c.k.shape[1]
    at = [0] * n
    for ends in steps:
        rows = [[x[a:e] for (x, a, e) in ((kv[s][i], at[s], ends[s]) for s in range(n))] for i in (0, 1)]
        cu = synth.cu_seqlens([e - a for a, e in zip(at, ends)])
        k, v = (qh.to_bf16(torch, np.concatenate(r)) for r in rows)
        qh.run_write(rlk, torch, dev, rlk.make_params(n, hkv, hkv), k, v, cu, at, c.n_pages, c.page, rope, max_pos)
        at = list(ends)
    rlk.rlk_attn_check_device_error()
    return [d.cpu().numpy() for d in dev[:4]]


def expected(c, kv):
    e = c.copy()
    for s, (k, v) in enumerate(kv):
        oq.write_tokens(e.k, e.ks, e.table[s], k)
        oq.write_tokens(e.v, e.vs, e.table[s], v)
    return e.k, e.v, e.ks, e.vs


def assert_pages(got, want, what):
    for a, b, name in zip(got, want, ("k", "v", "k_scale", "v_scale")):
        bad = int(np.sum(a.view(np.uint8) != b.view(np.uint8)))
        assert bad == 0, f"{what}: {bad} bytes of {name} differ"


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_write_matches_the_definition(page, hkv):
    # one token, part of a page, whole pages, one more; slots behind stay
    lens = [1, page - 1, page, page + 1, 0, 3 * page + 5, 300]
    c = qh.empty_cache(lens, hkv, page, seed=page)
    kv = qh.tokens(lens, hkv, seed=page + hkv)
    assert_pages(run_calls(c, kv, [lens]), expected(c, kv), f"page {page}, {hkv} heads")


@pytest.mark.parametrize("page", [8, 16, 128])
@pytest.mark.parametrize("step", [1, 3, 50])
def test_write_in_pieces_gives_the_same_pages(page, step):
    lens = [70, 129, 5]
    c = qh.empty_cache(lens, 2, page, seed=1)
    kv = qh.tokens(lens, 2, seed=2)
    steps = [[min(n, e) for n in lens] for e in range(step, max(lens) + step, step)]
    assert_pages(run_calls(c, kv, steps), expected(c, kv), f"steps of {step}")


def test_write_settles_special_values():
    # Inf, NaN, zeros of both signs, subnormals, the largest finite values,
    # ties, and pages of nothing but those next to the smallest normal
    bits = np.array([0x7F80, 0xFF80, 0x7FC0, 0x8000, 0x0000, 0x0001, 0x007F, 0x0078, 0x0080, 0x8080, 0x7F7F, 0xFF7F,
                     0x7F78, 0x7F70, 0x3F80, 0x3F88, 0x3F98, 0x3F89, 0x3F87, 0x0780, 0x077F, 0x0778], np.uint16)
    g = np.random.default_rng(8)
    n, hkv = 96, 2
    k = np.empty((n, hkv, 128), np.float32)
    v = np.empty_like(k)
    groups = [bits, bits[3:10], bits[5:10], bits[3:5], bits[14:19], bits[:3]]  # one per page of 16
    for p, vals in enumerate(groups):
        for x in (k, v):
            x[16 * p:16 * p + 16] = synth.bits_to_f32(g.choice(vals, (16, hkv, 128)))
    c = qh.empty_cache([n], hkv, 16, seed=3)
    assert_pages(run_calls(c, [(k, v)], [[n]]), expected(c, [(k, v)]), "special values at once")
    assert_pages(run_calls(c, [(k, v)], [[e] for e in range(1, n + 1)]), expected(c, [(k, v)]), "token by token")


@pytest.mark.parametrize("page", [8, 64])
def test_write_rotates_keys_as_the_rope_pass(page):
    torch, rlk = torch_cuda(), lib()
    lens = [40, 1, 130]
    kv = qh.tokens(lens, 4, seed=4)
    table = torch.from_numpy(rlk.rlk_attn_rope_table(1.0e6, 130)).cuda()
    rotated = []
    for k, v in kv:
        x = qh.to_bf16(torch, k)
        y = torch.empty_like(x)
        rlk.rlk_attn_rope(rlk.make_params(1), x, y, 4, [0, len(k)], None, table, 130)
        rotated.append((y.float().cpu().numpy(), v))
    c = qh.empty_cache(lens, 4, page, seed=5)
    for steps in ([lens], [[min(n, e) for n in lens] for e in range(7, 137, 7)]):
        assert_pages(run_calls(c, kv, steps, table, 130), expected(c, rotated), f"{len(steps)} calls")


def test_write_large_batch():
    # more sequences than one launch's tables hold
    lens = np.random.default_rng(9).integers(0, 40, 300).tolist()
    c = qh.empty_cache(lens, 2, 16, seed=6)
    kv = qh.tokens(lens, 2, seed=7)
    half = [n // 2 for n in lens]
    assert_pages(run_calls(c, kv, [half, lens]), expected(c, kv), "300 sequences")


def test_write_and_read_past_32_bit_offsets():
    # pages whose codes lie past 2^32 bytes of the pool
    torch, rlk = torch_cuda(), lib()
    hkv, page, n_pages = 8, 128, 34000  # 128 KB a page: 4.46 GB
    kv = qh.tokens([200], hkv, seed=11)[0]
    pools = [torch.zeros((n_pages, hkv, page, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((n_pages, hkv), device="cuda") for _ in range(2)]
    table = torch.tensor([[33998, 33001]], dtype=torch.int32, device="cuda")
    p = rlk.make_params(1, hkv, hkv)
    rlk.rlk_attn_qcache_write(p, qh.to_bf16(torch, kv[0]), qh.to_bf16(torch, kv[1]), [0, 200], None, None, 0, *pools,
                              *scales, n_pages, page, table, 2)
    k, v = (torch.empty((200, hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rlk.rlk_attn_qcache_read(p, *pools, *scales, n_pages, page, table, 2, [0, 200], None, k, v)
    ctx = np.array([200], np.int32)
    q = synth.normal_bf16(12, synth.T_Q, (1, hkv, 128))
    small = qh.empty_cache([200], hkv, page)
    for x, pool, scale, got in ((kv[0], small.k, small.ks, k), (kv[1], small.v, small.vs, v)):
        oq.write_tokens(pool, scale, small.table[0], x)
        want = oq.values(pool, scale)[small.table[0]].transpose(0, 2, 1, 3).reshape(-1, hkv, 128)[:200]
        assert np.array_equal(got.float().cpu().numpy(), want.astype(np.float32))
    out = torch.empty((1, hkv, 128), device="cuda")
    lse = torch.empty((1, hkv), device="cuda")
    rlk.rlk_attn_decode_qcache(p, qh.to_bf16(torch, q), *pools, *scales, n_pages, page, table, 2, ctx, 1, None, 0, out,
                               None, lse)
    rlk.rlk_attn_check_device_error()
    ref = qh.decode(rlk, torch, small, q, ctx, hkv, scale=None)
    assert np.array_equal(out.cpu().numpy().view(np.uint32), ref[0].view(np.uint32))


@pytest.mark.parametrize("page", [8, 32, 128])
def test_read_gives_code_times_scale(page):
    # every code, scales of any size: one rounding to BF16 of the exact product
    torch, rlk = torch_cuda(), lib()
    g = np.random.default_rng(13)
    lens, pos = [0, 77, 1, 200], [3, 9, 130, 0]
    hkv = 3
    c = qh.empty_cache([a + b for a, b in zip(lens, pos)], hkv, page, seed=14)
    for p in (c.k, c.v):
        p[:] = g.integers(0, 256, p.shape)
    for s in (c.ks, c.vs):
        s[:] = (np.exp2(g.integers(-118, 118, s.shape)) * g.choice([1.0, 1.0, 1.3, 1.999], s.shape)).astype(np.float32)
    kd, vd, ksd, vsd, td = c.device()
    cu = synth.cu_seqlens(lens)
    k, v = (torch.full((int(cu[-1]) + 2, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rlk.rlk_attn_qcache_read(rlk.make_params(4, hkv, hkv), kd, vd, ksd, vsd, c.n_pages, page, td, td.shape[1], cu, pos,
                             k, v)
    rlk.rlk_attn_check_device_error()
    for got, pool, scale in ((k, c.k, c.ks), (v, c.v, c.vs)):
        vals = oq.values(pool, scale)
        got = got.float().cpu().numpy()
        assert np.all(got[cu[-1]:] == 7.0), "rows behind the last sequence"
        for s in range(4):
            at = np.arange(pos[s], pos[s] + lens[s])
            want = vals[c.table[s][at // page], :, at % page]
            # 448 * 2^118 stays below the FP32 maximum, and a product of 4 and
            # 24 bits is exact in FP64: FP32 rounding, then BF16 rounding
            nan = np.isnan(want)
            want = synth.bf16_round(np.where(nan, 0.0, want).astype(np.float32)) + np.where(nan, np.nan, 0)
            assert np.array_equal(got[cu[s]:cu[s + 1]], want.astype(np.float32), equal_nan=True), f"sequence {s}"


# ---------------------------------------------------------------- decode

def assert_decode(got, q, c, ctx, hq, scale, what):
    """Against FP64 attention over the cached values.  w = p sv is split into
    four E4M3 pieces: a value of [2^E, 2^(E+1)) leaves at most 2^(E-4), which
    times 32 is at most 2^(E+1) again, so four pieces leave 2^(E-19): 2^-19 of
    w.  A block sums 128 products (each addition off by at most one last
    place: 128 * 2^-23 of the sum of |w v|).  Together at most
    (2^-16 + 2^-19) of the largest |v| of the context.  The scores' sums of 128
    products of FP32 or wider (at most 2^-22 of sum |q k| scale with the
    pieces' recombination and the log2 scaling) move p by as much, and lse."""
    kf, vf = qh.bf16_pools(c)
    kf = np.nan_to_num(kf, nan=0.0)
    vf = np.nan_to_num(vf, nan=0.0)
    ref, ref_lse = oracle.decode_paged_f64(q, kf, vf, np.maximum(c.table, 0), ctx, scale)
    out, outb, lse = got
    hkv = c.k.shape[1]
    for s in range(len(ctx)):
        at = np.arange(ctx[s])
        pages, slot = c.table[s][at // c.page], at % c.page
        for h in range(hq):
            g = h // (hq // hkv)
            vmax = np.abs(vf[pages, slot, g]).max()
            serr = 2.0 ** -22 * scale * (np.abs(q[s, h]).astype(np.float64) @ np.abs(kf[pages, slot, g]).T).max()
            tol = vmax * (2.0 ** -16 + 2.0 ** -19 + 2 * serr) + 1e-30
            e = np.abs(out[s, h] - ref[s, h]).max()
            assert e <= tol, f"{what}: sequence {s} head {h}: off by {e:.3g}, at most {tol:.3g}"
            el, tol = abs(lse[s, h] - ref_lse[s, h]), 2e-6 + 2.0 ** -21 * abs(ref_lse[s, h]) + serr
            assert el <= tol, f"{what}: lse of sequence {s} head {h}: {el:.3g}"
    assert np.array_equal(outb.view(np.uint32), synth.bf16_round(out).view(np.uint32)), f"{what}: BF16 output"
    return float(np.abs(out - ref).max()), float(np.abs(lse - ref_lse).max())


CTX = [1, 15, 16, 17, 127, 128, 129, 300, 1000, 2049]


@pytest.mark.parametrize("page", [16, 8, 32, 64, 128])
def test_decode_parity(page):
    torch, rlk = torch_cuda(), lib()
    c = qh.filled(CTX, 8, page, seed=20 + page, spread=False)
    q = synth.normal_bf16(21, synth.T_Q, (len(CTX), 32, 128))
    got = qh.decode(rlk, torch, c, q, CTX, 32, scale=128 ** -0.5)
    print("max error out, lse:", assert_decode(got, q, c, np.array(CTX, np.int32), 32, 128 ** -0.5, f"page {page}"))


@pytest.mark.parametrize("hq,hkv", [(8, 8), (4, 2), (24, 8), (40, 8), (16, 2), (7, 1)])
def test_decode_parity_groups(hq, hkv):
    torch, rlk = torch_cuda(), lib()
    ctx = [5, 300, 1500]
    c = qh.filled(ctx, hkv, 16, seed=22, spread=False)
    q = synth.normal_bf16(23, synth.T_Q, (3, hq, 128))
    got = qh.decode(rlk, torch, c, q, ctx, hq, scale=0.09)
    assert_decode(got, q, c, np.array(ctx, np.int32), hq, 0.09, f"{hq}/{hkv}")


@pytest.mark.parametrize("page", [8, 32])
def test_decode_parity_uneven_scales(page):
    # scales that differ by 2^12 between the pages of a block, outlier
    # channels, zero rows, queries from 2^-20 to 2^8 in one row
    torch, rlk = torch_cuda(), lib()
    ctx = [130, 64, 513]
    c = qh.filled(ctx, 2, page, seed=24, spread=True)
    g = np.random.default_rng(25)
    q = synth.bf16_round((g.standard_normal((3, 8, 128)) * np.exp2(g.integers(-20, 9, (3, 8, 128)))).astype(np.float32))
    q[1, 3] = 0.0
    got = qh.decode(rlk, torch, c, q, ctx, 8, scale=1.0 / 4096)
    assert_decode(got, q, c, np.array(ctx, np.int32), 8, 1.0 / 4096, f"page {page}")


def test_decode_tiny_and_huge_query_rows():
    # rows scaled by powers of two give the scores scaled by them: with the
    # softmax scale scaled back, the same bits
    torch, rlk = torch_cuda(), lib()
    ctx = [200]
    c = qh.filled(ctx, 1, 16, seed=26, spread=False)
    q = synth.normal_bf16(27, synth.T_Q, (1, 4, 128))
    ref = qh.decode(rlk, torch, c, q, ctx, 4, scale=2.0 ** -4)
    for e in (-100, 100):
        got = qh.decode(rlk, torch, c, np.ldexp(q, e).astype(np.float32), ctx, 4, scale=2.0 ** (-4 - e))
        assert_bitwise(got, ref, f"2^{e}")


def test_decode_huge_query_rows_over_tiny_keys():
    # a query's size moved to the keys and back (powers of two) is the same
    # scores, to the ends of the ranges: query elements up to 2^125, keys down
    # to scales of 2^-119
    torch, rlk = torch_cuda(), lib()
    ctx = [200]
    kv = qh.tokens(ctx, 1, 34, spread=False)
    q = synth.normal_bf16(35, synth.T_Q, (1, 4, 128))
    out = []
    for qe, ke in ((0, 0), (60, -60), (108, -108), (-108, 108), (124, -110)):
        c = qh.empty_cache(ctx, 1, 16, seed=36)
        oq.write_tokens(c.k, c.ks, c.table[0], np.ldexp(kv[0][0], ke).astype(np.float32))
        oq.write_tokens(c.v, c.vs, c.table[0], kv[0][1])
        out.append(qh.decode(rlk, torch, c, np.ldexp(q, qe).astype(np.float32), ctx, 4, scale=2.0 ** (-4 - qe - ke)))
    for got in out[1:]:
        assert_bitwise(got, out[0], "moved")


@pytest.fixture(scope="module")
def split_case():
    ctx = [1, 17, 128, 129, 1000, 2049, 4096]
    return qh.filled(ctx, 8, 16, seed=30, spread=False), ctx, synth.normal_bf16(31, synth.T_Q, (len(ctx), 32, 128))


@pytest.mark.parametrize("split_k", [0, 2, 3, 8, 64])
def test_split_equals_single_pass(split_case, split_k):
    torch, rlk = torch_cuda(), lib()
    c, ctx, q = split_case
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 32, split_k), qh.decode(rlk, torch, c, q, ctx, 32), f"k {split_k}")


@pytest.mark.parametrize("hq,hkv,k", [(24, 8, 3), (40, 8, 2), (8, 8, 7), (8, 1, 0)])
def test_split_on_chip_group_shapes(hq, hkv, k):
    torch, rlk = torch_cuda(), lib()
    ctx = [1, 200, 1999, 4097]
    c = qh.filled(ctx, hkv, 64, seed=32, spread=False)
    q = synth.normal_bf16(33, synth.T_Q, (4, hq, 128))
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, hq, k), qh.decode(rlk, torch, c, q, ctx, hq), f"{hq}/{hkv} k {k}")


@pytest.mark.parametrize("hq,hkv", [(3, 3), (10, 5), (14, 7), (12, 12), (20, 20), (32, 32), (160, 160)])
def test_kv_head_counts(hq, hkv):
    # heads that divide the SMs, that do not, and more of them than there are SMs
    torch, rlk = torch_cuda(), lib()
    ctx = [1, 700, 1500]
    c = qh.filled(ctx, hkv, 16, seed=38, spread=False)
    q = synth.normal_bf16(39, synth.T_Q, (3, hq, 128))
    one = qh.decode(rlk, torch, c, q, ctx, hq, 1, scale=0.1)
    for k in (0, 2):
        assert_bitwise(qh.decode(rlk, torch, c, q, ctx, hq, k, scale=0.1), one, f"{hq}/{hkv} k {k}")
    assert_decode(one, q, c, np.array(ctx, np.int32), hq, 0.1, f"{hq}/{hkv}")


@pytest.fixture(scope="module")
def long_case():
    # 79 and 40 segments of 512 keys: cut over many CTAs, folded past 32
    ctx = [40001, 129, 20000]
    return qh.filled(ctx, 1, 128, seed=45, spread=False), ctx, synth.normal_bf16(46, synth.T_Q, (3, 4, 128))


@pytest.mark.parametrize("split_k", [0, 2, 7, 64])
def test_split_long_sequences(long_case, split_k):
    torch, rlk = torch_cuda(), lib()
    c, ctx, q = long_case
    one = qh.decode(rlk, torch, c, q, ctx, 4, 1, scale=0.1)
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 4, split_k, scale=0.1), one, f"k {split_k}")
    if split_k == 0:
        assert_decode(one, q, c, np.array(ctx, np.int32), 4, 0.1, "long")


@pytest.mark.parametrize("ctx,hq,hkv,page", [
    ([20000, 30000, 9000, 500, 20001], 8, 8, 16),            # most pairs cut
    ([100000, 77, 131072, 1, 65000, 40000], 16, 8, 64),      # cut into many pieces
    ([700] * 230 + [3000] * 20, 40, 8, 128),                 # several pairs a CTA
    ([300000, 400000], 8, 1, 32),                            # two pairs on all the CTAs
], ids=["8 heads", "ragged", "short", "long"])
def test_even_load_equals_whole_pairs(ctx, hq, hkv, page):
    # thousands of blocks on all the CTAs, cut where the load is even: the same
    # bits as with every pair on one CTA, on every repetition and replay
    torch, rlk = torch_cuda(), lib()
    g = torch.Generator(device="cuda").manual_seed(len(ctx))
    per = [-(-c // page) for c in ctx]
    n, n_pages = len(ctx), sum(per)
    table = np.full((n, max(per)), -1, np.int32)
    table[np.arange(max(per))[None, :] < np.array(per)[:, None]] = np.random.default_rng(n).permutation(n_pages)
    pools, scales = [], []
    for _ in range(2):
        x = torch.empty((n_pages, hkv, page, 128), dtype=torch.uint8, device="cuda")
        x.random_(0x30, 0x70, generator=g)  # 0.5 .. 120
        x |= torch.randint(0, 2, x.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
        pools.append(x)
        scales.append(torch.exp2(torch.randint(-8, -4, (n_pages, hkv), generator=g, device="cuda").float()))
    q = torch.randn((n, hq, 128), generator=g, device="cuda").to(torch.bfloat16)
    p = rlk.make_params(n, hq, hkv)
    pool = (*pools, *scales, n_pages, page, torch.from_numpy(table).cuda(), table.shape[1])
    size = rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DECODE_QCACHE, None, ctx)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(k, out, lse):
        rlk.rlk_attn_decode_qcache(p, q, *pool, ctx, k, None, 0, out, None, lse, ws)

    ref = torch.empty((n, hq, 128), device="cuda"), torch.empty((n, hq), device="cuda")
    run(1, *ref)
    rlk.rlk_attn_check_device_error()
    assert bool(torch.isfinite(ref[0]).all())
    got = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    for k in (0, 0, 3, 0, 64, 0):
        got[0].fill_(float("nan"))
        run(k, *got)
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(got, ref)), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(0, *got)
    for _ in range(3):
        got[0].fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(got, ref)), "replay"
    rlk.rlk_attn_check_device_error()


def test_workspace_contents_do_not_matter(split_case):
    # zeros, all ones, and what other calls (of other batches) left
    torch, rlk = torch_cuda(), lib()
    c, ctx, q = split_case
    ref = qh.decode(rlk, torch, c, q, ctx, 32)
    dev, qd = c.device(), qh.to_bf16(torch, q)
    p, p1 = rlk.make_params(len(ctx), 32, 8), rlk.make_params(2, 32, 8)
    size = rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DECODE_QCACHE, None, ctx)
    assert size >= rlk.rlk_attn_workspace_size(p1, rlk.RLK_OP_DECODE_QCACHE, None, ctx[-2:])
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((len(ctx), 32, 128), device="cuda"), torch.empty((len(ctx), 32), device="cuda")
    pool = (*dev[:4], c.n_pages, c.page)
    for fill in (0, 0xFF, None, None):
        if fill is not None:
            ws.fill_(fill)
        out.fill_(float("nan"))
        rlk.rlk_attn_decode_qcache(p, qd, *pool, dev[4], dev[4].shape[1], ctx, 0, None, 0, out, None, lse, ws)
        assert np.array_equal(out.cpu().numpy().view(np.uint32), ref[0].view(np.uint32)), fill
        assert np.array_equal(lse.cpu().numpy().view(np.uint32), ref[2].view(np.uint32)), fill
        rlk.rlk_attn_decode_qcache(p1, qd[-2:].contiguous(), *pool, dev[4][-2:].contiguous(), dev[4].shape[1], ctx[-2:],
                                   0, None, 0, out[:2], None, lse[:2], ws)
        assert np.array_equal(out[:2].cpu().numpy().view(np.uint32), ref[0][-2:].view(np.uint32))
    rlk.rlk_attn_check_device_error()


def test_two_graphs_share_a_workspace(split_case):
    torch, rlk = torch_cuda(), lib()
    c, ctx, q = split_case
    ref = qh.decode(rlk, torch, c, q, ctx, 32)
    dev = c.device()
    runs = [[5, 6], [3, 4, 6]]
    size = max(rlk.rlk_attn_workspace_size(rlk.make_params(len(s), 32, 8), rlk.RLK_OP_DECODE_QCACHE, None,
                                           [ctx[i] for i in s]) for s in runs)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graphs = []
    for s in runs:
        qd, td = qh.to_bf16(torch, q[s]), dev[4][s].contiguous()
        out, lse = torch.empty((len(s), 32, 128), device="cuda"), torch.empty((len(s), 32), device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rlk.rlk_attn_decode_qcache(rlk.make_params(len(s), 32, 8), qd, *dev[:4], c.n_pages, c.page, td, td.shape[1],
                                       [ctx[i] for i in s], 0, None, 0, out, None, lse, ws)
        graphs.append((graph, s, out, lse, qd, td))
    for i in (0, 1, 0, 0, 1, 1, 0):
        graph, s, out, lse = graphs[i][:4]
        out.fill_(float("nan"))
        graph.replay()
        assert np.array_equal(out.cpu().numpy().view(np.uint32), ref[0][s].view(np.uint32)), s
        assert np.array_equal(lse.cpu().numpy().view(np.uint32), ref[2][s].view(np.uint32)), s
    rlk.rlk_attn_check_device_error()


def test_decode_does_not_depend_on_batch_or_page_order(split_case):
    torch, rlk = torch_cuda(), lib()
    c, ctx, q = split_case
    full = qh.decode(rlk, torch, c, q, ctx, 32)
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 32), full, "repeat")
    for seqs in ([6], [2, 0], [5, 4, 3]):
        assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 32, seqs=seqs), tuple(x[seqs] for x in full), f"{seqs}")
    perm = np.random.default_rng(34).permutation(c.n_pages)
    moved = c.copy()
    for name in ("k", "v", "ks", "vs"):
        a = getattr(c, name)
        b = np.empty_like(a)
        b[perm] = a
        setattr(moved, name, b)
    moved.table = np.where(c.table >= 0, perm[np.maximum(c.table, 0)], -1).astype(np.int32)
    assert_bitwise(qh.decode(rlk, torch, moved, q, ctx, 32), full, "pages moved")


@pytest.mark.parametrize("split_k", [0, 1, 3])
def test_sequences_that_share_pages(split_case, split_k):
    # sequences with a common prefix hold the same page ids: each gets what it
    # gets alone, from the pages as they are
    torch, rlk = torch_cuda(), lib()
    c, _, _ = split_case
    ctx = [4096, 4095, 3000, 3000, 17, 1]
    table = np.repeat(c.table[6:7], len(ctx), 0)
    q = synth.normal_bf16(37, synth.T_Q, (len(ctx), 32, 128))
    got = qh.decode(rlk, torch, c, q, ctx, 32, split_k, table=table)
    for s in range(len(ctx)):
        one = qh.decode(rlk, torch, c, q, ctx, 32, split_k, seqs=[s], table=table)
        assert_bitwise([x[s:s + 1] for x in got], one, f"sequence {s}")
    assert_decode(got, q, qh.Cache(c.k, c.v, c.ks, c.vs, table, c.page), np.array(ctx, np.int32), 32, 128 ** -0.5,
                  "shared")


def test_decode_300_sequences():
    torch, rlk = torch_cuda(), lib()
    ctx = np.random.default_rng(35).integers(1, 400, 300).tolist()
    c = qh.filled(ctx, 2, 16, seed=36, spread=False)
    q = synth.normal_bf16(37, synth.T_Q, (300, 8, 128))
    full = qh.decode(rlk, torch, c, q, ctx, 8)
    some = [0, 127, 128, 299]
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 8, seqs=some), tuple(x[some] for x in full), "subset")
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 8, split_k=3), full, "split")
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 8, split_k=0), full, "auto")


@pytest.mark.parametrize("split_k", [1, 4])
def test_decode_rotates_queries_as_the_rope_pass(split_k):
    torch, rlk = torch_cuda(), lib()
    ctx = [1, 130, 777]
    c = qh.filled(ctx, 4, 16, seed=38, spread=False)
    q = synth.normal_bf16(39, synth.T_Q, (3, 20, 128))
    table = torch.from_numpy(rlk.rlk_attn_rope_table(1.0e6, 777)).cuda()
    x = qh.to_bf16(torch, q)
    y = torch.empty_like(x)
    rlk.rlk_attn_rope(rlk.make_params(3), x, y, 20, [0, 1, 2, 3], np.array(ctx) - 1, table, 777)
    ref = qh.decode(rlk, torch, c, y.float().cpu().numpy(), ctx, 20)
    assert_bitwise(qh.decode(rlk, torch, c, q, ctx, 20, split_k, rope=table, max_pos=777), ref, f"k {split_k}")


def test_non_finite_values_stay_where_they_are():
    # a NaN in K of a visible key makes that head group's rows NaN, one in V
    # its dimension; other heads and sequences keep their bits; the same
    # values past the context change nothing
    torch, rlk = torch_cuda(), lib()
    ctx = [100, 300]
    kv = qh.tokens(ctx, 2, 40, spread=False)
    q = synth.normal_bf16(41, synth.T_Q, (2, 8, 128))
    clean = qh.filled(ctx, 2, 16, seed=40, spread=False)
    ref = qh.decode(rlk, torch, clean, q, ctx, 8)
    c = clean.copy()
    c.v[c.table[1][3], 1, 5, 7] = 0x7F
    c.k[c.table[0][2], 0, 1, 9] = 0xFF
    out, _, lse = qh.decode(rlk, torch, c, q, ctx, 8)
    assert np.isnan(out[1, 4:, 7]).all() and np.isnan(out[0, :4]).all() and np.isnan(lse[0, :4]).all()
    ok = np.ones(out.shape, bool)
    ok[1, 4:, 7] = ok[0, :4] = False
    assert np.array_equal(out[ok].view(np.uint32), ref[0][ok].view(np.uint32))
    q2 = q.copy()
    q2[1, 2, 50] = np.inf
    out, _, _ = qh.decode(rlk, torch, clean, q2, ctx, 8)
    assert np.isnan(out[1, 2]).all() and np.array_equal(out[0].view(np.uint32), ref[0][0].view(np.uint32))
    del kv


def test_bad_pages_are_reported_and_never_written():
    torch, rlk = torch_cuda(), lib()
    lens = [40, 20]
    c = qh.empty_cache(lens, 2, 16, seed=42)
    kv = qh.tokens(lens, 2, seed=43)
    want = expected(c, kv)
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        b = c.copy()
        lost = b.table[0, 1]
        b.table[0, 1] = bad
        dev = b.device()
        k, v = (qh.to_bf16(torch, np.concatenate([x[i] for x in kv])) for i in (0, 1))
        p = rlk.make_params(2, 2, 2)
        qh.run_write(rlk, torch, dev, p, k, v, [0, 40, 60], None, b.n_pages, 16)
        with pytest.raises(rlk.RlkError) as e:
            rlk.rlk_attn_check_device_error()
        assert e.value.status == 8
        for got, full, init in zip(dev[:4], want, (c.k, c.v, c.ks, c.vs)):
            exp = full.copy()
            exp[lost] = init[lost]
            assert np.array_equal(got.cpu().numpy().view(np.uint8), exp.view(np.uint8))
        ko, vo = torch.ones_like(k), torch.ones_like(v)
        rlk.rlk_attn_qcache_read(p, *dev[:4], b.n_pages, 16, dev[4], dev[4].shape[1], [0, 40, 60], None, ko, vo)
        with pytest.raises(rlk.RlkError) as e:
            rlk.rlk_attn_check_device_error()
        assert e.value.status == 8 and not ko[16:32].any() and not vo[16:32].any() and ko[:16].any()
        q = synth.normal_bf16(44, synth.T_Q, (2, 2, 128))
        good = qh.decode(rlk, torch, b, q, lens, 2, dev=dev, check=False)
        with pytest.raises(rlk.RlkError) as e:
            rlk.rlk_attn_check_device_error()
        assert e.value.status == 8
        assert np.isfinite(good[0]).all()
        # the page reads as zeros (codes 0 under scale 1)
        z = b.copy()
        z.k, z.v, z.ks, z.vs = (d.cpu().numpy() for d in dev[:4])
        z.k[lost] = z.v[lost] = 0
        z.ks[lost] = z.vs[lost] = 1.0
        z.table[0, 1] = lost
        assert_bitwise(good, qh.decode(rlk, torch, z, q, lens, 2), f"page {bad}")


# ---------------------------------------------------------------- together

def test_serving_loop_against_the_definition():
    """Prompts written in chunks with their keys rotated, each chunk's queries
    attending to the cache read back, then decode steps that append a token
    and attend to it: every row against FP64 attention over the cached
    values, and the pages against those of writing everything at once."""
    torch, rlk = torch_cuda(), lib()
    from tests.gpu_helpers import TOL_LSE, TOL_OUT
    hq, hkv, page, theta = 8, 2, 16, 1.0e6
    prompts, steps, chunk = [70, 33, 150], 20, 64
    lens = [n + steps for n in prompts]
    n = len(lens)
    kv = qh.tokens(lens, hkv, seed=50, spread=False)
    qs = [synth.normal_bf16(51 + s, synth.T_Q, (lens[s], hq, 128)) for s in range(n)]
    table = torch.from_numpy(rlk.rlk_attn_rope_table(theta, 200)).cuda()
    c = qh.empty_cache(lens, hkv, page, seed=52)
    dev = c.device()
    p = rlk.make_params(n, hq, hkv)
    pool = (*dev[:4], c.n_pages, page, dev[4], dev[4].shape[1])
    rot_k = [oracle.rope_f32(kv[s][0], np.arange(lens[s]), theta) for s in range(n)]
    rot_q = [oracle.rope_f32(qs[s], np.arange(lens[s]), theta) for s in range(n)]
    scale = 1.0 / np.sqrt(128)

    def quantised(s, upto):
        e = qh.empty_cache([upto], hkv, page)
        oq.write_tokens(e.k, e.ks, e.table[0], rot_k[s][:upto])
        oq.write_tokens(e.v, e.vs, e.table[0], kv[s][1][:upto])
        return [oq.values(a, b)[e.table[0]].transpose(0, 2, 1, 3).reshape(-1, hkv, 128)[:upto].astype(np.float32)
                for a, b in ((e.k, e.ks), (e.v, e.vs))]

    def append(at, to):
        cu = synth.cu_seqlens([b - a for a, b in zip(at, to)])
        k, v = (qh.to_bf16(torch, np.concatenate([kv[s][i][at[s]:to[s]] for s in range(n)])) for i in (0, 1))
        rlk.rlk_attn_qcache_write(p, k, v, cu, at, table, 200, *pool)

    at = [0] * n
    while at != prompts:
        to = [min(a + chunk, m) for a, m in zip(at, prompts)]
        append(at, to)
        cu_k = synth.cu_seqlens(to)
        cu_q = synth.cu_seqlens([b - a for a, b in zip(at, to)])
        k, v = (torch.empty((int(cu_k[-1]), hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        rlk.rlk_attn_qcache_read(p, *pool, cu_k, None, k, v)
        q = qh.to_bf16(torch, np.concatenate([qs[s][at[s]:to[s]] for s in range(n)]))
        out = torch.empty(q.shape, device="cuda")
        lse = torch.empty(q.shape[:2], device="cuda")
        rlk.rlk_attn_prefill_rope(p, q, k, v, cu_q, cu_k, -1, table, 200, out, None, lse)
        rlk.rlk_attn_check_device_error()
        for s in range(n):
            if to[s] == at[s]:
                continue
            kk, vv = quantised(s, to[s])
            ref, ref_lse = oracle.attention_f64(rot_q[s][at[s]:to[s]], kk, vv, [0, to[s] - at[s]], [0, to[s]], scale)
            a, b = cu_q[s], cu_q[s + 1]
            assert np.abs(out[a:b].cpu().numpy() - ref).max() <= TOL_OUT * np.abs(vv).max()
            assert np.abs(lse[a:b].cpu().numpy() - ref_lse).max() <= TOL_LSE
        at = to
    out = torch.empty((n, hq, 128), device="cuda")
    outb = torch.empty((n, hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, hq), device="cuda")
    for _ in range(steps):
        to = [a + 1 for a in at]
        append(at, to)
        ctx = np.array(to, np.int32)
        ws = torch.empty(rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DECODE_QCACHE, None, ctx), dtype=torch.uint8,
                         device="cuda")
        q = qh.to_bf16(torch, np.stack([qs[s][at[s]] for s in range(n)]))
        rlk.rlk_attn_decode_qcache(p, q, *pool, ctx, 0, table, 200, out, outb, lse, ws)
        rlk.rlk_attn_check_device_error()
        for s in range(n):
            kk, vv = quantised(s, to[s])
            ref, ref_lse = oracle.attention_f64(rot_q[s][at[s]:to[s]], kk, vv, [0, 1], [0, to[s]], scale)
            assert np.abs(out[s].cpu().numpy() - ref[0]).max() <= TOL_OUT * np.abs(vv).max()
            assert np.abs(lse[s].cpu().numpy() - ref_lse[0]).max() <= TOL_LSE
        at = to
    final = expected(c, [(rot_k[s], kv[s][1]) for s in range(n)])
    assert_pages([d.cpu().numpy() for d in dev[:4]], final, "after the loop")


def test_other_stream_and_graph_replay():
    # write and decode captured together on a side stream; a replay with new
    # inputs copied in gives what eager calls on those inputs give
    torch, rlk = torch_cuda(), lib()
    ctx = [4097, 2000, 300, 128]
    hq, hkv = 32, 8
    base = qh.filled(ctx, hkv, 16, seed=60, spread=False)
    p = rlk.make_params(4, hq, hkv)
    q, k, v = (synth.normal_bf16(s, synth.T_Q, (4, h, 128)) for s, h in ((61, hq), (62, hkv), (63, hkv)))
    pos = [x - 1 for x in ctx]
    dev = base.device()
    pool = (*dev[:4], base.n_pages, 16, dev[4], dev[4].shape[1])
    qd, kd, vd = (qh.to_bf16(torch, x) for x in (q, k, v))
    out, outb = torch.empty((4, hq, 128), device="cuda"), torch.empty((4, hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, hq), device="cuda")
    size = rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DECODE_QCACHE, None, ctx)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step():
        rlk.rlk_attn_qcache_write(p, kd, vd, [0, 1, 2, 3, 4], pos, None, 0, *pool)
        rlk.rlk_attn_decode_qcache(p, qd, *pool, ctx, 4, None, 0, out, outb, lse, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    first = [x.clone() for x in (out, lse)]
    state = [d.clone() for d in dev[:4]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0, 1):
        for d, x in zip(dev[:4], state):
            d.copy_(x)
        for t, x in ((qd, q), (kd, k), (vd, v)):
            t.copy_(qh.to_bf16(torch, np.roll(x, i, 0)))
        graph.replay()
        torch.cuda.synchronize()
        rlk.rlk_attn_check_device_error()
        got = [x.clone() for x in (out, lse)]
        after = [d.clone() for d in dev[:4]]
        for d, x in zip(dev[:4], state):
            d.copy_(x)
        step()
        rlk.rlk_attn_check_device_error()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, lse))), f"replay {i}"
        assert all(torch.equal(a, b) for a, b in zip(after, dev[:4])), f"pages after replay {i}"
        if i == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_two_streams_at_once():
    # two decodes of different batches in flight together, each with its own
    # workspace, keep their bits
    torch, rlk = torch_cuda(), lib()
    probs = []
    for seed, ctx in ((70, [3000, 900]), (71, [5000])):
        c = qh.filled(ctx, 2, 16, seed=seed, spread=False)
        q = synth.normal_bf16(seed, synth.T_Q, (len(ctx), 8, 128))
        probs.append((c, q, ctx, qh.decode(rlk, torch, c, q, ctx, 8), c.device(), qh.to_bf16(torch, q)))
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    runs = []
    for rep in range(6):
        for (c, q, ctx, ref, dev, qd), s in zip(probs, streams):
            p = rlk.make_params(len(ctx), 8, 2)
            with torch.cuda.stream(s):
                out = torch.empty((len(ctx), 8, 128), device="cuda")
                ws = torch.empty(rlk.rlk_attn_workspace_size(p, rlk.RLK_OP_DECODE_QCACHE, None, ctx), dtype=torch.uint8,
                                 device="cuda")
                rlk.rlk_attn_decode_qcache(p, qd, *dev[:4], c.n_pages, 16, dev[4], dev[4].shape[1], ctx, 2, None, 0,
                                           out, None, None, ws, stream=s)
            runs.append((out, ref[0], ws))
    torch.cuda.synchronize()
    rlk.rlk_attn_check_device_error()
    for out, ref, _ in runs:
        assert np.array_equal(out.cpu().numpy().view(np.uint32), ref.view(np.uint32))


def test_binding_refuses_wrong_tensors():
    torch, rlk = torch_cuda(), lib()
    c = qh.filled([20], 2, 16, seed=80, spread=False)
    dev = c.device()
    pool = (*dev[:4], c.n_pages, 16, dev[4], dev[4].shape[1])
    p = rlk.make_params(1, 2, 2)
    q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros((1, 2, 128), device="cuda"), torch.zeros((1, 2), device="cuda")
    for bad in (q.float(), q.cpu(), torch.zeros((1, 128, 2), dtype=torch.bfloat16, device="cuda").transpose(1, 2)):
        with pytest.raises(ValueError):
            rlk.rlk_attn_decode_qcache(p, bad, *pool, [20], 1, None, 0, out, None, lse)
        with pytest.raises(ValueError):
            rlk.rlk_attn_qcache_write(p, bad, q, [0, 1], [19], None, 0, *pool)
    with pytest.raises(ValueError):
        rlk.rlk_attn_qcache_read(p, dev[0].float(), *pool[1:], [0, 1], None, q, q)
