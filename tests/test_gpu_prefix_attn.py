"""Attention over a shared prefix and own pages against 64 bits.

Bounds.  With u the relative rounding of an fp32 operation (2^-24; 2^-23 is allowed for a tensor
core's sums, which may truncate), a score of d products is off by at most (d + 3) u times the sum of its
products' sizes (a), and exp2 by a few u, so a weight is off by a factor within 1 +- e, e = (d + 3) u a +
8 u; numerator and denominator are sums of n weights, each off by n u more.  The output is off by at most
(2 e + 2 (n + 64) u) sum(p |v|).  Weights rounded to bf16 for the product with V add 2^-8 of that sum,
weights kept as three bf16 numbers 2^-24, and a bf16 output half a step, 2^-8 of itself.  (An eighth of the weights for
a bf16 output have an exp2 that is off by 1.1e-4 of itself, which is 3% of that rounding and added.)
"""
from __future__ import annotations

import numpy as np
import pytest

from pages_model import attend64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _give_memory_back():
    yield  # the largest pools here hold several GB
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def _zha():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tree_indexed_sparse_build_b200 import zha
    zha.lib()
    return zha


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(zha, heads, group, d, page, prefix, lens, nq, kv, q, seed=0, width=None, spread=1.0):
    """A cache whose slots share the first pages; rows without a token hold NaN and infinity."""
    gen = torch.Generator().manual_seed(seed)
    width = width or max(1, -(-max(lens + [prefix]) // page))
    shared = prefix // page
    need = shared + sum(max(1, -(-n // page) - shared) for n in lens) + 3
    ids = torch.randperm(need, generator=gen).tolist()
    K, V = (torch.full((need, heads, page, d), x) for x in (float("nan"), float("inf")))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = shared
    for s, n in enumerate(lens):
        k = -(-n // page)
        own = max(0, k - shared)
        table[s, :k] = torch.tensor((ids[:shared] + ids[at:at + own])[:k], dtype=torch.int32)
        at += own
        if k <= shared and n % page:  # shorter than the prefix: its partial page is its own (and not read)
            table[s, k - 1] = ids[at]
            at += 1
        for j in range(k):
            r = min(page, n - j * page)
            p = int(table[s, j])
            if j >= shared or (r == page and torch.isnan(K[p, 0, 0, 0])):
                K[p, :, :r] = torch.randn((heads, r, d), generator=gen)
                V[p, :, :r] = torch.randn((heads, r, d), generator=gen)
    K, V = K.to(kv), V.to(kv)
    Q = (spread * torch.randn((len(lens), heads * group, nq, d), generator=gen)).to(q)
    pages = zha.Pages(heads, d, page, need, len(lens), width, kv)
    pages.load(table.cuda(), _i32(lens))
    return pages, Q, K, V, table


def _bound(o, w, a, d, n, tensor, out):
    u = 2.0 ** (-23 if tensor else -24)
    e = (d + 3) * u * a[..., None] + 8 * u
    lim = (2 * e + 2 * (n + 64) * u) * w
    if tensor:
        lim = lim + (2.0 ** -8 + 2.2e-4 if out == BF16 else 2.0 ** -24) * w
    return lim + (2.0 ** -8 * np.abs(o) if out == BF16 else 2.0 ** -24 * np.abs(o)) + 1e-30


def _compare(got, Q, K, V, table, lens, seqs, scale, prefix_seq, prefix, causal, kv, q, out):
    o, w, a = attend64(Q, K, V, table, lens, seqs, scale, prefix_seq, prefix, causal)
    x = got.double().cpu().numpy()
    assert np.isfinite(x).all()
    lim = _bound(o, w, a, Q.shape[-1], max(lens), kv == BF16 and q == BF16, out)
    off = np.abs(x - o)
    assert (off <= lim).all(), f"off by {np.max(off / lim):.3g} of the bound"


def _run(zha, heads, group, d, page, prefix, lens, nq, causal, kv, q, out, seqs=None, prefix_seq=0, scale=None, seed=0):
    pages, Q, K, V, table = _case(zha, heads, group, d, page, prefix, lens, nq, kv, q, seed)
    seqs = list(range(len(lens))) if seqs is None else seqs
    Q = Q[:len(seqs)].contiguous() if len(seqs) <= len(lens) else Q.repeat(-(-len(seqs) // len(lens)), 1, 1, 1)[:len(seqs)].contiguous()
    scale = d ** -0.5 if scale is None else scale
    got = pages.attend(Q.cuda(), K.cuda(), V.cuda(), scale, _i32(seqs), prefix_seq, prefix, causal, out)
    assert pages.check() == zha.ZHA_OK
    assert got.dtype == out and got.shape == Q.shape
    _compare(got, Q, K, V, table, lens, seqs, scale, prefix_seq, prefix, causal, kv, q, out)


TYPES = [(F32, F32, F32), (BF16, BF16, BF16), (BF16, BF16, F32), (BF16, F32, F32), (F32, BF16, BF16)]

SHAPES = {
    # heads, group, d, page, prefix, lens, nq, causal
    "one token": (1, 1, 64, 8, 0, [1], 1, False),
    "one prefix page": (1, 1, 128, 16, 16, [16], 1, False),
    "prefix only": (2, 4, 128, 16, 48, [48, 48, 48], 1, False),
    "empty, shorter than the prefix, at its end, behind it": (2, 3, 64, 16, 160, [300, 0, 7, 160, 161, 128, 0], 1, False),
    "all empty": (1, 2, 128, 32, 0, [0, 0], 3, True),
    "tile borders": (1, 4, 128, 32, 128, [255, 256, 257, 383, 384, 385, 191, 192, 193, 129], 1, False),
    "page of 8": (2, 2, 64, 8, 136, [140, 301, 399, 136], 2, True),
    "page of 256": (1, 5, 128, 256, 256, [256, 300, 511, 512, 513, 900], 1, False),
    "page of 256, nothing shared": (3, 1, 64, 256, 0, [1, 129, 257, 640], 1, False),
    "causal, more queries than tokens": (2, 3, 64, 16, 0, [1, 2, 5, 40], 5, True),
    "causal inside the prefix": (1, 2, 128, 16, 64, [64, 66, 70, 200], 7, True),
    "rows that do not divide a tile": (2, 7, 64, 16, 96, [100 + 13 * i for i in range(20)], 3, False),
    "more rows than a tile": (1, 3, 64, 16, 128, [150, 400, 129], 50, True),
    "many more rows than a tile": (1, 8, 128, 32, 256, [300, 257], 40, False),
    "one row tile of a pair left over": (2, 4, 128, 16, 512, [520 + i for i in range(80)], 1, False),
    "two row tiles": (1, 8, 64, 16, 1024, [1030 + 3 * i for i in range(32)], 1, False),
    "more sequences than threads": (1, 1, 64, 8, 16, [17 + (7 * i) % 60 for i in range(700)], 1, False),
    "long own parts beside short ones": (2, 2, 128, 64, 64, [64, 9000, 65, 3000, 70], 1, False),
}


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("name", SHAPES)
def test_against_64_bits(name, types):
    _run(_zha(), *SHAPES[name], *types)


@pytest.mark.parametrize("types", TYPES[:3], ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(types, scale):
    _run(_zha(), 2, 4, 64, 16, 256, [256, 300, 700], 1, False, *types, scale=scale)


@pytest.mark.parametrize("types", TYPES[:2], ids=lambda t: "-".join(str(x)[6:] for x in t))
def test_slots_in_any_order_and_repeated(types):
    zha = _zha()
    # the prefix is a slot that the batch does not name
    _run(zha, 2, 2, 128, 16, 96, [130, 96, 200, 99, 111], 1, False, *types, seqs=[4, 2, 2, 3, 4, 2], prefix_seq=1)
    _run(zha, 2, 2, 128, 16, 0, [130, 96, 200, 99, 111], 1, False, *types, seqs=[1])


@pytest.mark.parametrize("types", TYPES[:2], ids=lambda t: "-".join(str(x)[6:] for x in t))
def test_growing_maximum(types):
    # scores that rise along the sequence by far more than a weight's range, so the running
    # maximum moves in every tile
    zha = _zha()
    kv, q, out = types
    pages, Q, K, V, table = _case(zha, 1, 2, 64, 16, 512, [512, 1500], 1, kv, q)
    n = 1500
    for j in range(-(-n // 16)):
        K[int(table[1, j])] = (K[int(table[1, j])].float() * 0.1 + 0.02 * j).to(kv)
    Q = (Q.float().abs()).to(q)
    got = pages.attend(Q.cuda(), K.cuda(), V.cuda(), 1.0, _i32([0, 1]), 0, 512, False, out)
    _compare(got, Q, K, V, table, [512, 1500], [0, 1], 1.0, 0, 512, False, kv, q, out)


@pytest.mark.parametrize("types", TYPES[:3], ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("step", [0.05, 1.0])
def test_maximum_that_grows_over_many_tiles(types, step):
    # rows whose scores rise (and fall) by up to a hundred and more within the tiles of one sum
    zha = _zha()
    kv, q, out = types
    n = [6000, 2111]
    pages, Q, K, V, table = _case(zha, 1, 4, 64, 16, 0, n, 2, kv, q)
    for s in range(2):
        for j in range(-(-n[s] // 16)):
            r = min(16, n[s] - 16 * j)
            K[int(table[s, j]), :, :r] = (K[int(table[s, j]), :, :r].float() * 0.1 + step * j).to(kv)
    got = pages.attend(Q.cuda(), K.cuda(), V.cuda(), 0.125, _i32([0, 1]), out_dtype=out)
    assert pages.check() == zha.ZHA_OK
    _compare(got, Q, K, V, table, n, [0, 1], 0.125, 0, 0, False, kv, q, out)


def test_long_sums_of_an_fp32_output_do_not_shrink():
    # The tensor core cuts its sums off: up to 2^-23 of a sum at each product, half of that on average.  A sum takes at most
    # 96 products before it is added in fp32, so outputs are short by no more than 96 * 2^-24 = 5.7e-6 on average (the
    # sums of every CTA here would take 1,600 products and more).
    zha = _zha()
    heads, group, d, page, prefix, batch, nq = 8, 8, 128, 64, 32768, 40, 4
    lens = [prefix] * batch
    gen = torch.Generator().manual_seed(3)
    K, V = (torch.randn((prefix // page, heads, page, d), generator=gen).to(BF16).cuda() for _ in "KV")
    Q = torch.randn((batch, heads * group, nq, d), generator=gen).to(BF16).cuda()
    pages = zha.Pages(heads, d, page, prefix // page, batch, prefix // page, BF16)
    pages.load(torch.arange(prefix // page, dtype=torch.int32, device="cuda").repeat(batch, 1), _i32(lens))
    got = pages.attend(Q, K, V, d ** -0.5, _i32(list(range(batch))), 0, prefix, False, F32)
    assert pages.check() == zha.ZHA_OK
    short, size = 0.0, 0.0
    for h in range(heads):
        q = Q[:, h * group:(h + 1) * group].reshape(-1, d).double()
        k, v = (x[:, h].reshape(-1, d).double() for x in (K, V))
        o = torch.softmax(q @ k.T * d ** -0.5, -1) @ v
        x = got[:, h * group:(h + 1) * group].reshape(-1, d).double()
        short += float(((o - x) * o).sum())
        size += float((o * o).sum())
    assert abs(short / size) <= 96 * 2.0 ** -24


@pytest.mark.parametrize("own", [1, 200])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
def test_a_nan_reaches_the_rows_that_see_it_and_no_others(types, value, own):
    # a score that is NaN, or infinite, of the only key behind the prefix or of one of many; and a query row that is NaN
    zha = _zha()
    kv, q, out = types
    lens = [256 + own, 300, 256, 290]
    pages, Q, K, V, table = _case(zha, 2, 2, 64, 16, 256, lens, 1, kv, q)
    last = lens[0] - 1
    Qn = Q.clone()
    if value == value:  # one infinite product, positive
        Qn[0, :, :, 0] = Qn[0, :, :, 0].abs() + 1
        K[int(table[0, last // 16]), :, last % 16, 0] = value
    else:
        K[int(table[0, last // 16]), :, last % 16] = value
    Qn[3, 1] = float("nan")
    seqs = [0, 1, 2, 3]
    got = pages.attend(Qn.cuda(), K.cuda(), V.cuda(), 0.125, _i32(seqs), 0, 256, False, out)
    assert pages.check() == zha.ZHA_OK
    assert torch.isnan(got[0]).all() and torch.isnan(got[3, 1]).all()
    K[int(table[0, last // 16]), :, last % 16] = 0
    o, w, a = attend64(Q, K, V, table, lens, seqs, 0.125, 0, 256, False)
    keep = np.ones(o.shape[:2], dtype=bool)
    keep[0] = keep[3, 1] = False
    off = np.abs(got.double().cpu().numpy() - o)
    lim = _bound(o, w, a, 64, max(lens), kv == BF16 and q == BF16, out)
    assert (off <= lim)[keep].all()


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
def test_masked_values_of_any_size_weigh_nothing(types):
    # tokens that only later queries of a sequence see hold the largest finite values
    zha = _zha()
    kv, q, out = types
    lens, nq = [261, 290, 140], 5
    pages, Q, K, V, table = _case(zha, 2, 2, 64, 16, 128, lens, nq, kv, q)
    K2, V2 = K.clone(), V.clone()
    for s, n in enumerate(lens):
        for t in range(n - nq + 1, n):
            V2[int(table[s, t // 16]), :, t % 16] = 3e38
    seqs = [0, 1, 2]
    got = [pages.attend(Q.cuda(), K.cuda(), v.cuda(), 0.125, _i32(seqs), 0, 128, True, out) for v in (V, V2)]
    assert pages.check() == zha.ZHA_OK
    assert torch.equal(got[0][:, :, 0], got[1][:, :, 0])


def test_random_shapes():
    import random
    zha = _zha()
    rng = random.Random(11)
    for seed in range(40):
        page = rng.choice([8, 16, 32, 64, 128, 256])
        prefix = rng.choice([0, 1, 2, 3, 9]) * page
        nq = rng.choice([1, 1, 2, 3, 8])
        lens = [rng.choice([0, prefix, prefix + rng.randint(1, 40), rng.randint(1, 2 * prefix + 700)])
                for _ in range(rng.choice([1, 2, 5, 17, 60]))]
        types = rng.choice(TYPES)
        _run(zha, rng.choice([1, 2, 3]), rng.choice([1, 2, 5, 8]), rng.choice([64, 128]), page, prefix,
             lens if max(lens) >= prefix else lens + [prefix], nq, rng.random() < 0.5, *types,
             prefix_seq=0 if lens[0] >= prefix else (lens + [prefix]).index(max(lens + [prefix])), seed=seed)


@pytest.mark.parametrize("keys", [1, 3, 5, 13, 16, 19, 25, 32, 40, 50])
def test_shares_that_start_inside_the_last_tile_of_a_kind(keys):
    # two row tiles against `keys` key tiles, then own parts: at these lengths some CTA's share starts inside the
    # last tile of the shared part (cut for 148 CTAs), which is the CTA's before
    prefix = 128 * keys
    _run(_zha(), 2, 8, 64, 128, prefix, [prefix + 130 * (1 + i % 3) for i in range(32)], 1, False, BF16, BF16, BF16)


def test_bad_slots_pages_and_prefixes_are_reported():
    zha = _zha()
    for kv in (F32, BF16):
        lens = [64, 100, 40]
        pages, Q, K, V, table = _case(zha, 1, 2, 64, 16, 32, lens, 1, kv, kv)
        q, k, v = Q.cuda(), K.cuda(), V.cuda()
        got = pages.attend(q, k, v, 0.1, _i32([1, 3, -1]), 0, 32, out_dtype=F32)
        assert pages.check() == zha.ZHA_ERR_DEVICE
        assert (got[1:] == 0).all()  # as empty sequences
        want = pages.attend(q[:1].contiguous(), k, v, 0.1, _i32([1]), 0, 32, out_dtype=F32)
        assert pages.check() == zha.ZHA_OK
        assert (got[0] - want[0]).abs().max() < 1e-5
        pages.attend(q, k, v, 0.1, _i32([0, 1, 2]), 2, 48, out_dtype=F32)  # slot 2 has 40 tokens
        assert pages.check() == zha.ZHA_ERR_DEVICE
        # a page id the table's owner wrote past the library: read as a page of zeros
        pages.table[1, 3] = 10 ** 6
        pages.table[2, 2] = -7
        got = pages.attend(q, k, v, 0.1, _i32([0, 1, 2]), 0, 32, out_dtype=F32)
        assert pages.check() == zha.ZHA_ERR_DEVICE
        assert torch.isfinite(got).all()


def test_a_run_of_them_together():
    """A prompt in pages, forks that go their own ways, attention, freeing, compacting, and the
    survivor in a tree's dense cache, routed over with a beam that keeps every leaf."""
    zha = _zha()
    heads, group, d, page, n = 2, 2, 128, 16, 200
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    pages = zha.Pages(heads, d, page, 80, 6, 16, BF16)
    K, V = pages.pools()
    K.fill_(float("nan"))
    V.fill_(float("nan"))
    prompt = rnd(1, heads, n, d), rnd(1, heads, n, d)
    pages.append(K, V, _i32([5]), *prompt)
    pages.fork(K, V, _i32([5, 5, 5]), _i32([0, 1, 2]))
    mine = [[p[0].clone()] * 3 for p in prompt]
    for step in range(20):
        Kn, Vn = rnd(3, heads, 1, d), rnd(3, heads, 1, d)
        pages.append(K, V, _i32([0, 1, 2]), Kn, Vn)
        for i in range(3):
            mine[0][i] = torch.cat([mine[0][i], Kn[i]], 1)
            mine[1][i] = torch.cat([mine[1][i], Vn[i]], 1)
        if step == 9:  # the second sample loses to a fork of the first
            pages.free(_i32([1]))
            pages.fork(K, V, _i32([0]), _i32([1]))
            for m in mine:
                m[1] = m[0].clone()
        if step == 12:
            pages.compact(K, V)
    Q = rnd(3, heads * group, 1, d)
    got = pages.attend(Q, K, V, d ** -0.5, _i32([0, 1, 2]), 5, n // page * page, out_dtype=F32)
    for i in range(3):
        k, v = (m[i].double().repeat_interleave(group, 0) for m in mine)
        p = torch.softmax(Q[i].double() @ k.transpose(1, 2) * d ** -0.5, -1)
        lim = (2.0 ** -24 + 2 * 284 * 2.0 ** -23 + 2 * 131 * 2.0 ** -23 * 64) * (p @ v.abs())
        assert ((got[i].double() - p @ v).abs() <= lim).all()
    pages.free(_i32([5, 0, 2]))
    assert int(pages.compact(K, V)) == -(-220 // page)
    dense = [torch.zeros((1, heads, 256, d), dtype=BF16, device="cuda") for _ in "KV"]
    pages.gather(K, V, _i32([1]), *dense)
    tree = zha.Tree(1, heads, d, 4, 16, 256, BF16)
    tree.build(dense[0], 220)
    O, _, _ = tree.decode(Q[1:2].contiguous(), *dense, 14, d ** -0.5, out_dtype=F32)
    assert (O[0] - got[1]).abs().max() < 1e-3
    assert pages.check() == zha.ZHA_OK and tree.check() == zha.ZHA_OK


@pytest.mark.parametrize("kv", [F32, BF16])
def test_graph_replays_while_sequences_grow(kv):
    zha = _zha()
    lens = [70, 64, 90]
    pages, Q, K, V, table = _case(zha, 2, 2, 64, 16, 64, lens, 1, kv, kv, width=12)
    pages2 = zha.Pages(2, 64, 16, K.shape[0] + 12, 3, 12, kv)
    K, V = (torch.cat([x, torch.full((12,) + tuple(x.shape[1:]), float("nan"), dtype=kv)]) for x in (K, V))
    pages2.load(table.cuda(), _i32(lens))
    k, v, q, seqs = K.cuda(), V.cuda(), Q.cuda(), _i32([0, 1, 2])
    new = torch.zeros((3, 2, 5, 64), dtype=kv, device="cuda"), torch.zeros((3, 2, 5, 64), dtype=kv, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for _ in range(2):  # two graphs: each has its scratch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pages2.append(k, v, seqs, *new)
            outs.append(pages2.attend(q, k, v, 0.125, seqs, 0, 64, out_dtype=F32))
        graphs.append(g)
    for step in range(6):
        for x in new:
            x.copy_(torch.randn(x.shape, device="cuda"))
        graphs[step % 2].replay()
        got = outs[step % 2]
        lens = [n + 5 for n in lens]
        assert pages2.lens.tolist() == lens
        _compare(got, Q, k.cpu(), v.cpu(), pages2.table.cpu(), lens, [0, 1, 2], 0.125, 0, 64, False, kv, kv, F32)
    assert pages2.check() == zha.ZHA_OK


@pytest.mark.parametrize("kv", [F32, BF16])
def test_calls_on_several_streams_at_once(kv):
    zha = _zha()
    lens = [600 + 37 * i for i in range(12)]
    pages, Q, K, V, table = _case(zha, 2, 4, 128, 32, 512, lens, 1, kv, kv)
    q, k, v, seqs = Q.cuda(), K.cuda(), V.cuda(), _i32(list(range(12)))
    want = pages.attend(q, k, v, 0.1, seqs, 0, 512, out_dtype=F32)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [pages.attend(q, k, v, 0.1, seqs, 0, 512, out_dtype=F32, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    for x in got:
        assert torch.equal(x, want)  # the order of the work does not show


@pytest.mark.parametrize("kv", [F32, BF16])
def test_pools_behind_two_to_the_31(kv):
    zha = _zha()
    heads, d, page = 2, 128, 256
    num = 2 ** 31 // (heads * d * page) + 9
    lens = [page + 40, 2 * page + 7]
    pages = zha.Pages(heads, d, page, num, 2, 3, kv)
    K, V = pages.pools()
    table = torch.tensor([[num - 1, num - 3, -1], [num - 1, num - 2, 0]], dtype=torch.int32)
    small = torch.tensor([[0, 1, -1], [0, 2, 3]], dtype=torch.int32)
    gen = torch.Generator().manual_seed(1)
    ks, vs = (torch.randn((4, heads, page, d), generator=gen).to(kv) for _ in "KV")
    for a, b in zip((0, 1, 2, 3), (num - 1, num - 3, num - 2, 0)):
        K[b], V[b] = ks[a].cuda(), vs[a].cuda()
    pages.load(table.cuda(), _i32(lens))
    Q = torch.randn((2, 4, 1, d), generator=gen).to(kv)
    got = pages.attend(Q.cuda(), K, V, 0.1, _i32([0, 1]), 0, page, out_dtype=F32)
    assert pages.check() == zha.ZHA_OK
    _compare(got, Q, ks, vs, small, lens, [0, 1], 0.1, 0, page, False, kv, kv, F32)


@pytest.mark.parametrize("heads,group,d,page,prefix,lens,nq", [
    (8, 4, 128, 64, 8192, [8192 + 1 + 37 * i for i in range(64)], 1),   # dual tiles, many own items of several lengths
    (2, 8, 128, 16, 16384, [16384 + (i * 211) % 500 for i in range(16)], 1),  # one row tile, long runs of single tiles
    (8, 4, 64, 32, 4096, [4096 + 129 * (i % 4) for i in range(300)], 1),
    (1, 4, 128, 8, 0, [1 + (97 * i) % 4000 for i in range(70)], 3),
    (4, 1, 64, 256, 512, [513 + i for i in range(200)], 1),
    (3, 5, 128, 128, 2048, [2048 + 300 * i for i in range(9)], 11),
])
def test_long_pipelines_against_the_fp32_kernel(heads, group, d, page, prefix, lens, nq):
    # many tiles per CTA on the tensor cores against the fp32 kernel on the same numbers (an fp32 query tensor
    # of bf16 values), and the same bits in three calls
    zha = _zha()
    gen = torch.Generator(device="cuda").manual_seed(5)
    width = -(-max(lens) // page)
    shared = prefix // page
    num = shared + sum(-(-n // page) - shared for n in lens)
    pages = zha.Pages(heads, d, page, num, len(lens), width, BF16)
    K, V = (torch.randn((num, heads, page, d), generator=gen, device="cuda").to(BF16) for _ in "KV")
    ids, at = torch.randperm(num, generator=gen, device="cuda").int(), shared
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[:, :shared] = ids[:shared]
    for s, n in enumerate(lens):
        k = -(-n // page) - shared
        table[s, shared:shared + k] = ids[at:at + k]
        at += k
        if n % page and k > 0:  # rows without a token
            K[ids[at - 1].long(), :, n % page:] = float("nan")
            V[ids[at - 1].long(), :, n % page:] = float("inf")
    pages.load(table, _i32(lens))
    seqs = _i32(list(range(len(lens))))
    Q = torch.randn((len(lens), heads * group, nq, d), generator=gen, device="cuda").to(BF16)
    got = [pages.attend(Q, K, V, d ** -0.5, seqs, 0, prefix, nq > 1, F32) for _ in range(3)]
    want = pages.attend(Q.float(), K, V, d ** -0.5, seqs, 0, prefix, nq > 1, F32).double()
    assert pages.check() == zha.ZHA_OK
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    # as above, with sum(|scale q k|) below 4 sqrt(d) and sum(p |v|) below max |v| < 6
    bound = 2.0 ** -24 + 2 * (d + 3) * 2.0 ** -23 * d ** -0.5 * d * 4 + 2 * (max(lens) + 64) * 2.0 ** -23
    assert ((got[0].double() - want).abs().amax(-1) <= bound * 6).all()
    # and rounded to bf16 at the end: 2^-8 of sum(p |v|) (below E|v| + 6 sigma / sqrt(n) < 6) and of the output
    bf = pages.attend(Q, K, V, d ** -0.5, seqs, 0, prefix, nq > 1).double()
    assert ((bf - want).abs() <= (2.0 ** -8 + 2.2e-4 + bound) * 6).all()


def test_more_entries_than_slots():
    zha = _zha()
    for kv in (F32, BF16):
        lens = [70, 90, 64]
        pages, Q, K, V, table = _case(zha, 2, 2, 64, 16, 64, lens, 1, kv, kv)
        q, k, v = Q.repeat(40, 1, 1, 1).cuda(), K.cuda(), V.cuda()
        seqs = [0, 1, 2] * 40
        got = pages.attend(q, k, v, 0.2, _i32(seqs), 0, 64, out_dtype=F32)
        _compare(got, q.cpu(), K, V, table, lens, seqs, 0.2, 0, 64, False, kv, kv, F32)


def test_output_in_the_place_of_the_queries():
    zha = _zha()
    for kv in (F32, BF16):
        lens = [300, 640, 257]
        pages, Q, K, V, table = _case(zha, 2, 2, 64, 16, 256, lens, 2, kv, kv)
        q = Q.cuda()
        got = pages.attend(q, K.cuda(), V.cuda(), 0.2, _i32([0, 1, 2]), 0, 256, True, O=q)
        assert got is q
        _compare(q, Q, K, V, table, lens, [0, 1, 2], 0.2, 0, 256, True, kv, kv, kv)


def test_refusals_with_a_cache():
    zha = _zha()
    pages, Q, K, V, table = _case(zha, 2, 2, 64, 16, 32, [40, 50], 1, F32, F32)
    q, k, v, s = Q.cuda(), K.cuda(), V.cuda(), _i32([0, 1])
    for status, call in [
        (zha.ZHA_ERR_INVALID_ARG, lambda: pages.attend(q, k, v, float("nan"), s)),
        (zha.ZHA_ERR_INVALID_ARG, lambda: pages.attend(q, k, v, float("inf"), s)),
        (zha.ZHA_ERR_INVALID_ARG, lambda: pages.attend(q[:, :3].contiguous(), k, v, 0.1, s)),  # 3 heads over 2
        (zha.ZHA_ERR_INVALID_ARG, lambda: pages.attend(q, k, v, 0.1, s, prefix_tokens=24)),    # inside a page
        (zha.ZHA_ERR_INVALID_ARG, lambda: pages.attend(q, k, v, 0.1, s, prefix_tokens=-16)),
        (zha.ZHA_ERR_INVALID_ARG, lambda: pages.attend(q, k, v, 0.1, s, prefix_seq=2, prefix_tokens=16)),
        (zha.ZHA_ERR_CAPACITY, lambda: pages.attend(q, k, v, 0.1, s, prefix_tokens=16 * 100)),
        (zha.ZHA_ERR_INVALID_ARG, lambda: pages.free(_i32([0, 1, 0]))),                         # more than slots
        (zha.ZHA_ERR_INVALID_ARG, lambda: zha.zha_prefix_attn_decode(
            pages.handle, q, k, v, s, 0, 32, False, 0.1, q.clone(), torch.zeros(64, device="cuda"))),  # scratch
    ]:
        with pytest.raises(zha.ZhaError) as e:
            call()
        assert e.value.status == status
    for what, call in [
        ("contiguous", lambda: pages.attend(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, 0.1, s)),
        ("device tensors", lambda: pages.attend(Q, k, v, 0.1, s)),
        ("device tensors", lambda: pages.free(s.cpu())),
        ("K: ", lambda: pages.attend(q, k[1:].contiguous(), v, 0.1, s)),
        ("Q: shape", lambda: pages.attend(q[0], k, v, 0.1, s)),
    ]:
        with pytest.raises(ValueError, match=what):
            call()
    assert pages.check() == zha.ZHA_OK


def test_a_wait_that_runs_out():
    # the waits for the loads are bounded; here to one clock, which no load keeps
    zha = _zha()
    lens = [700 + 100 * i for i in range(40)]
    pages, Q, K, V, table = _case(zha, 2, 8, 128, 64, 640, lens, 1, BF16, BF16)
    q, k, v, seqs = Q.cuda(), K.cuda(), V.cuda(), _i32(list(range(40)))
    want = pages.attend(q, k, v, 0.1, seqs, 0, 640)
    assert pages.check() == zha.ZHA_OK
    for _ in range(3):
        zha.zha_pages_set_wait_limit(pages.handle, 1)
        lost = pages.attend(q, k, v, 0.1, seqs, 0, 640)
        assert torch.isnan(lost.float()).all()
        assert pages.check() == zha.ZHA_ERR_TIMEOUT
        zha.zha_pages_set_wait_limit(pages.handle, 0)
        assert torch.equal(pages.attend(q, k, v, 0.1, seqs, 0, 640), want)
        assert pages.check() == zha.ZHA_OK


def test_nothing_to_do():
    zha = _zha()
    pages, Q, K, V, table = _case(zha, 1, 1, 64, 8, 0, [5], 1, F32, F32)
    before = pages.launches
    assert pages.attend(Q[:0].cuda(), K.cuda(), V.cuda(), 0.1, _i32([])).shape == (0, 1, 1, 64)
    assert pages.attend(Q[:, :, :0].contiguous().cuda(), K.cuda(), V.cuda(), 0.1, _i32([0])).shape == (1, 1, 0, 64)
    assert pages.launches == before


def test_scratch_of_a_call_that_only_bf16_queries_fit():
    # 128 entries of up to 16,777,216 tokens on 32 heads: more than 2^31 tiles of 32 keys, a quarter as many of 128
    zha = _zha()
    heads, d, page, batch = 32, 128, 256, 128
    pages, Q, K, V, table = _case(zha, heads, 1, d, page, 0, [300], 1, BF16, BF16, width=65536)
    q, k, v, seqs = Q.repeat(batch, 1, 1, 1).cuda(), K.cuda(), V.cuda(), _i32([0] * batch)
    for out in (BF16, F32):
        O = torch.full(q.shape, 7.0, dtype=out, device="cuda")
        with pytest.raises(zha.ZhaError) as e:
            zha.zha_prefix_attn_decode(pages.handle, q, k, v, seqs, 0, 0, False, 0.1, O,
                                       torch.zeros(16, dtype=torch.uint8, device="cuda"))
        assert e.value.status == zha.ZHA_ERR_INVALID_ARG and (O == 7).all()
        got = pages.attend(q, k, v, 0.1, seqs, out_dtype=out)
        assert pages.check() == zha.ZHA_OK
        _compare(got, q.cpu(), K, V, table, [300], [0] * batch, 0.1, 0, 0, False, BF16, BF16, out)
    with pytest.raises(zha.ZhaError) as e:
        pages.attend(q.float(), k, v, 0.1, seqs)
    assert e.value.status == zha.ZHA_ERR_UNSUPPORTED


def test_calls_ask_for_shared_memory_once():
    # what a call asks of the CUDA runtime after the first of its kind: two launches, and nothing about its kernels
    from torch.profiler import ProfilerActivity, profile
    zha = _zha()
    for kv, out in ((BF16, BF16), (BF16, F32), (F32, F32)):
        for d in (64, 128):
            pages, Q, K, V, table = _case(zha, 2, 2, d, 16, 32, [40, 50], 1, kv, kv)
            q, k, v, s = Q.cuda(), K.cuda(), V.cuda(), _i32([0, 1])
            pages.attend(q, k, v, 0.1, s, 0, 32, out_dtype=out)
            torch.cuda.synchronize()
            with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as prof:
                pages.attend(q, k, v, 0.1, s, 0, 32, out_dtype=out)
                torch.cuda.synchronize()
            names = [e.name for e in prof.events()]
            launches = sum(n.startswith(("cudaLaunchKernelExC", "cuLaunchKernelEx")) for n in names)
            if launches == 0:
                pytest.skip("the profiler sees no calls of the runtime")
            assert launches == 2, names
            assert not any("FuncSetAttribute" in n for n in names), names
