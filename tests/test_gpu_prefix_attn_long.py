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
    yield  # the largest pools here hold half a GB
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
