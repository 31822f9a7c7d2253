"""Attention over long prefixes: that no key tile is lost, doubled or stale on the way through many tiles
per CTA, and what long sums may lose."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _give_memory_back():
    yield  # the largest pools here hold a GB and more
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


def _shared(zha, heads, d, page, prefix, batch):
    """A cache of `batch` slots that all hold the same prefix and nothing else, in order."""
    n = prefix // page
    pages = zha.Pages(heads, d, page, n, batch, n, BF16)
    pages.load(torch.arange(n, dtype=torch.int32, device="cuda").repeat(batch, 1), _i32([prefix] * batch))
    return pages


def test_long_sums_of_a_bf16_output_do_not_shrink():
    # The tensor core cuts its sums off: up to 2^-23 of a sum at each product, half of that on average.  A sum takes at most
    # 256 tiles of eight products, so outputs are short by no more than 2048 * 2^-24 = 1.22e-4 on average (a sum
    # without an end takes 8,192 tiles here).  The roundings of weights and output, at most 2^-8 of each and 2^-8 /
    # sqrt(3) in the mean square, are as often up as down: over 300,000 outputs (at least 100,000 of them independent;
    # E o^4 = 3 (E o^2)^2) their mean is 0 with a deviation of sqrt(2) 2^-8 / sqrt(3) sqrt(3 / 1e5) = 1.75e-5.  Six of those.
    zha = _zha()
    d, page, prefix, batch, nq = 128, 64, 1 << 20, 64, 640
    gen = torch.Generator(device="cuda").manual_seed(3)
    K, V = (torch.randn((prefix // page, 1, page, d), generator=gen, device="cuda").to(BF16) for _ in "KV")
    Q = torch.randn((batch, 1, nq, d), generator=gen, device="cuda").to(BF16)
    pages = _shared(zha, 1, d, page, prefix, batch)
    got = pages.attend(Q, K, V, d ** -0.5, _i32(list(range(batch))), 0, prefix)
    assert pages.check() == zha.ZHA_OK
    k, v = (x.view(-1, d).double() for x in (K, V))
    short, size = 0.0, 0.0
    for b in (0, 21, 42, 63):
        for q, x in zip(Q[b, 0].double().split(160), got[b, 0].double().split(160)):
            o = torch.softmax(q @ k.T * d ** -0.5, -1) @ v
            short += float(((o - x) * o).sum())
            size += float((o * o).sum())
    assert abs(short / size) <= 2048 * 2.0 ** -24 + 6 * 1.75e-5


def test_a_maximum_that_moves_between_long_sums():
    # Rows whose scores rise or fall along 131,072 tokens by 0 to 300 (base 2), so that from one sum of 256 tiles to the
    # next the maximum stays, moves by less than 2^16 or by more, in lanes of one warp.
    #
    # Bound, here and below: weights rounded to bf16 are off by at most 2^-8 of themselves.  For independent normal
    # values the squared norms of a row's error and of the row are sum(p^2 delta^2) and sum(p^2) times a chi-square of
    # d = 64 or more, which in 10^5 rows stays within 0.3 and 2.1 of d: their quotient is below 2^-8 sqrt(2.1 / 0.3) = 2.7 2^-8.  The
    # rounding of the output adds 2^-8, the rest (scores, exp2, sums) less than 0.3 2^-8: 4 2^-8.
    zha = _zha()
    d, page, prefix, batch, nq = 64, 128, 131072, 32, 1280
    gen = torch.Generator(device="cuda").manual_seed(4)
    K = 0.3 * torch.randn((prefix // page, 1, page, d), generator=gen, device="cuda")
    K[..., 0] = torch.linspace(-8, 8, prefix, device="cuda").view(prefix // page, 1, page)
    K = K.to(BF16)
    V = torch.randn(K.shape, generator=gen, device="cuda").to(BF16)
    Q = torch.randn((batch, 1, nq, d), generator=gen, device="cuda")
    rise = torch.tensor([0, 1, 5, 20, 60, 110, 200, 300], device="cuda") * math.log(2.0) / 16  # by 16 = 8 - -8
    Q[..., 0] = (rise.repeat(nq // 8) * (1 - 2 * (torch.arange(nq, device="cuda") // 8 % 2)))
    Q = Q.to(BF16)
    pages = _shared(zha, 1, d, page, prefix, batch)
    got = pages.attend(Q, K, V, 1.0, _i32(list(range(batch))), 0, prefix)
    assert pages.check() == zha.ZHA_OK
    k, v = (x.view(-1, d).double() for x in (K, V))
    for b in (0, 9, 31):
        for q, x in zip(Q[b, 0].double().split(320), got[b, 0].double().split(320)):
            o = torch.softmax(q @ k.T, -1) @ v
            off = (x - o).norm(dim=-1) / o.norm(dim=-1)
            assert (off <= 4 * 2.0 ** -8).all(), off.max()


LONG = [
    # heads, group, d, page, prefix, lens, nq, causal
    (8, 4, 128, 64, 8192, [8192 + 1 + 37 * i for i in range(64)], 1, False),   # dual tiles, many own items of several lengths
    (2, 8, 128, 16, 16384, [16384 + (i * 211) % 500 for i in range(16)], 1, False),  # one row tile, runs of single tiles
    (1, 4, 64, 32, 65536, [65536 + (i * 97) % 300 for i in range(96)], 1, False),  # one and a half pairs on one head
    (8, 4, 64, 32, 4096, [4096 + 129 * (i % 4) for i in range(300)], 1, False),
    (1, 4, 128, 8, 0, [1 + (97 * i) % 4000 for i in range(70)], 3, True),
    (1, 1, 128, 64, 0, [100000], 1, False),                                    # one sequence on one head
    (4, 1, 64, 256, 512, [513 + i for i in range(200)], 1, False),
    (3, 5, 128, 128, 2048, [2048 + 300 * i for i in range(9)], 11, True),
]


def _table(heads, page, prefix, lens, gen):
    """Page ids by slot, the first prefix // page of them common, and how many there are."""
    width, shared = -(-max(lens) // page), prefix // page
    num = shared + sum(-(-n // page) - shared for n in lens)
    ids = torch.randperm(num, generator=gen, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[:, :shared] = ids[:shared]
    at = shared
    for s, n in enumerate(lens):
        k = -(-n // page) - shared
        table[s, shared:shared + k] = ids[at:at + k]
        at += k
    return table, num


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,group,d,page,prefix,lens,nq,causal", LONG)
def test_every_tile_counts_once(heads, group, d, page, prefix, lens, nq, causal, out):
    # Scale 0 and values that say which 64 tokens of their sequence they belong to (one of d columns is 1): an output is the
    # share of the tokens that a query sees in each class, so a key tile that is lost, doubled or stale shows
    # (it changes two classes by a sixteenth where they are largest; the bound is a 250th).  All weights are 1 within 2 2^-22 (for bf16 outputs
    # 1.1e-4, which rounds to 1; the sum of the weights takes an eighth of it), so sums of weights and values are whole
    # numbers below 2^24 but for that, and cut off by 96 times 2^-23 at most.
    zha = _zha()
    gen = torch.Generator(device="cuda").manual_seed(6)
    table, num = _table(heads, page, prefix, lens, gen)
    pages = zha.Pages(heads, d, page, num, len(lens), table.shape[1], BF16)
    pages.load(table, _i32(lens))
    K = torch.randn((num, heads, page, d), generator=gen, device="cuda").to(BF16)
    V = torch.zeros((num, heads, page, d), dtype=BF16, device="cuda")
    V.fill_(float("nan"))  # rows without a token
    for s, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        V[table[s].long()[t // page], :, t % page] = torch.eye(d, dtype=BF16, device="cuda")[t // 64 % d][:, None]
    Q = torch.randn((len(lens), heads * group, nq, d), generator=gen, device="cuda").to(BF16)
    got = pages.attend(Q, K, V, 0.0, _i32(list(range(len(lens)))), 0, prefix, causal, out).double()
    assert pages.check() == zha.ZHA_OK
    relative = (2.0 ** -8 + 1.1e-4 / 8 + 1e-6 if out == BF16 else 4 * 2.0 ** -22 + 96 * 2.0 ** -23 + max(lens) / 512 * 2.0 ** -24)
    for s, n in enumerate(lens):
        for i in range(nq):
            m = n - (nq - 1 - i) if causal else n
            want = torch.bincount(torch.arange(max(m, 0), device="cuda") // 64 % d, minlength=d).double() / max(m, 1)
            assert ((got[s, :, i] - want).abs() <= relative * want).all(), (s, i)


@pytest.mark.parametrize("heads,group,d,page,prefix,lens,nq,causal", LONG)
def test_long_pipelines_by_norm(heads, group, d, page, prefix, lens, nq, causal):
    # As against the fp32 kernel elsewhere, but by the norm of each row's error: a 128-key tile left out of 65,536 keys
    # changes a row by 4% of its norm, out of 8,192 by 12%; with the bound derived above 1.6% are allowed for a bf16 output.  For an
    # fp32 one scores are off by at most (d + 3) 2^-23 sum |scale q k| (below 4 sqrt(d) here), weights by twice that of themselves and
    # 8 2^-23, sums by 96 2^-23; 2.7 times all of it, as above, is below 2e-3.
    zha = _zha()
    gen = torch.Generator(device="cuda").manual_seed(7)
    table, num = _table(heads, page, prefix, lens, gen)
    pages = zha.Pages(heads, d, page, num, len(lens), table.shape[1], BF16)
    pages.load(table, _i32(lens))
    K, V = (torch.randn((num, heads, page, d), generator=gen, device="cuda").to(BF16) for _ in "KV")
    Q = torch.randn((len(lens), heads * group, nq, d), generator=gen, device="cuda").to(BF16)
    seqs = _i32(list(range(len(lens))))
    want = pages.attend(Q.float(), K, V, d ** -0.5, seqs, 0, prefix, causal, F32).double()
    size = want.norm(dim=-1)
    for out, limit in ((BF16, 4 * 2.0 ** -8), (F32, 2e-3)):
        got = pages.attend(Q, K, V, d ** -0.5, seqs, 0, prefix, causal, out).double()
        off = (got - want).norm(dim=-1)
        assert (off <= limit * size).all(), (out, (off / size).max())
    assert pages.check() == zha.ZHA_OK


def test_weights_for_an_fp32_output_keep_24_bits():
    # Two keys, one with a weight of 1 and a value of 0, the other with a weight w < 1 and values of 1: the output is w / (1 +
    # w), off by as much as w is.  Scores are exact (whole products), times scale log2(e) they are rounded to 2^-24 of up to 9 (in the
    # exponent: 9 ln 2 2^-24 of w, and as much for the constant), ex2 is off by 2^-22, the sum, the quotient and the
    # output by 2^-24 each: 1.15e-6.  Weights in two bf16 numbers instead of three are off by up to 2^-17 = 7.6e-6.
    zha = _zha()
    n, d, page = 96, 64, 8
    pages = zha.Pages(1, d, page, n, n, 1, BF16)
    pages.load(torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1), _i32([2] * n))
    K, V = (torch.zeros((n, 1, page, d), dtype=BF16, device="cuda") for _ in "KV")
    less = torch.arange(1, n + 1, device="cuda")
    K[:, 0, 1, 0] = -less.to(BF16)
    V[:, 0, 1] = 1
    Q = torch.zeros((n, 1, 1, d), dtype=BF16, device="cuda")
    Q[..., 0] = 1
    scale = 0.0625
    got = pages.attend(Q, K, V, scale, _i32(list(range(n))), out_dtype=F32).double().view(n, d)
    assert pages.check() == zha.ZHA_OK
    w = torch.exp(-scale * less.double())
    want = w / (1 + w)
    limit = 2 * 9 * math.log(2.0) * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24
    assert ((got - want[:, None]).abs() <= limit * want[:, None]).all()
    # (the bound is one that two numbers do not keep)
    high = w.float().to(BF16)
    two = high.double() + (w.float() - high.float()).to(BF16).double()
    assert ((two / w - 1).abs() > limit).any()


@pytest.mark.parametrize("shared,batch,group", [(True, 4, 2), (True, 16, 4), (False, 1, 4), (False, 1, 48)])
def test_long_sums_of_few_rows(shared, batch, group):
    # 276 tiles a stream and CTA, so that its sum ends once on the way, of rows that fill a warp, a tile in part, or
    # more than a warp of one sequence's own tokens.  A sum that is lost or counted twice is a fortieth of
    # the keys, 16% of a row's norm; the bound is 4 2^-8 as above.
    zha = _zha()
    heads, d, page, n = 8, 64, 256, 1310720
    gen = torch.Generator(device="cuda").manual_seed(8)
    K, V = (torch.randn((n // page, heads, page, d), generator=gen, device="cuda", dtype=BF16) for _ in "KV")
    Q = torch.randn((batch, heads * group, 1, d), generator=gen, device="cuda").to(BF16)
    pages = _shared(zha, heads, d, page, n, batch)
    got = pages.attend(Q, K, V, d ** -0.5, _i32(list(range(batch))), 0, n if shared else 0)
    assert pages.check() == zha.ZHA_OK
    for h in range(heads):
        q, x = (t[:, h * group:(h + 1) * group].reshape(-1, d).double() for t in (Q, got))
        k, v = (t[:, h].reshape(-1, d).double() for t in (K, V))
        for i in range(0, len(q), 16):
            o = torch.softmax(q[i:i + 16] @ k.T * d ** -0.5, -1) @ v
            assert ((x[i:i + 16] - o).norm(dim=-1) <= 4 * 2.0 ** -8 * o.norm(dim=-1)).all(), (h, i)
