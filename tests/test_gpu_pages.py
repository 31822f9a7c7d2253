"""The paged cache against a plain Python model: pages, tables, counts and rows, bit for bit."""
from __future__ import annotations

import random

import pytest

from pages_model import PagesModel

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


class Both:
    """The same calls on the device and on the model."""

    def __init__(self, zha, heads, d, page, num_pages, slots, width, dtype, seed=0):
        self.gen = torch.Generator().manual_seed(seed)
        shape = (num_pages, heads, page, d)
        K, V = (torch.randn(shape, generator=self.gen).to(dtype) for _ in "KV")
        K[::3], V[::2] = float("nan"), float("inf")  # pools start as whatever memory held
        self.model = PagesModel(num_pages, slots, width, page, K, V)
        self.K, self.V = K.cuda(), V.cuda()
        self.pages = zha.Pages(heads, d, page, num_pages, slots, width, dtype)
        self.heads, self.d, self.dtype, self.zha = heads, d, dtype, zha

    def new(self, n, T):
        return [torch.randn((n, self.heads, T, self.d), generator=self.gen).to(self.dtype) for _ in "KV"]

    def append(self, seqs, T, counts=None):
        Kn, Vn = self.new(len(seqs), T)
        self.pages.append(self.K, self.V, _i32(seqs), Kn.cuda(), Vn.cuda(), None if counts is None else _i32(counts))
        self.model.append(seqs, Kn, Vn, counts)

    def fork(self, src, dst):
        self.pages.fork(self.K, self.V, _i32(src), _i32(dst))
        self.model.fork(src, dst)

    def copy(self, src, dst):
        self.pages.copy(self.K, self.V, _i32(src), _i32(dst))
        self.model.copy(src, dst)

    def free(self, seqs):
        self.pages.free(_i32(seqs))
        self.model.free(seqs)

    def compact(self):
        live = self.pages.compact(self.K, self.V)
        assert int(live) == self.model.compact()

    def gather(self, seqs, capacity):
        out = [torch.full((len(seqs), self.heads, capacity, self.d), 7.0, dtype=self.dtype) for _ in "KV"]
        got = [x.cuda() for x in out]
        self.pages.gather(self.K, self.V, _i32(seqs), *got)
        m = self.model
        for i, s in enumerate(seqs):
            for pool, x in ((m.K, out[0]), (m.V, out[1])):
                if m.lens[s]:
                    x[i, :, :m.lens[s]] = pool[m.rows[s]].transpose(0, 1).flatten(1, 2)[:, :m.lens[s]]
        for x, y in zip(got, out):
            assert torch.equal(x.cpu(), y)

    def check(self):
        assert self.pages.check() == self.zha.ZHA_OK
        self.model.check(self.pages, self.K, self.V)


@pytest.mark.parametrize("heads,d,page,dtype", [(1, 64, 8, F32), (3, 128, 16, BF16), (2, 64, 32, BF16),
                                                (2, 128, 128, F32), (1, 128, 256, BF16)])
def test_lengths_around_page_borders(heads, d, page, dtype):
    b = Both(_zha(), heads, d, page, 40, 9, 5, dtype)
    lens = [0, 1, page - 1, page, page + 1, 2 * page]
    b.append(list(range(6)), 2 * page, lens)
    b.check()
    b.append([5, 0, 3], 1)  # a full page's next token, an empty sequence's first
    b.check()
    b.fork([1, 3, 0], [6, 7, 8])
    b.check()
    b.append([6, 7, 1], 3, [3, 0, 2])
    b.gather([7, 1, 6, 2], 2 * page + 3)
    b.free([2, 1, 4])
    b.check()
    b.compact()
    b.check()
    b.append([2, 1], page + 1, [page + 1, 1])
    b.check()


@pytest.mark.parametrize("seed", range(6))
def test_random_programs(seed):
    rng = random.Random(seed)
    page = rng.choice([8, 16, 64])
    slots = rng.choice([5, 12])
    b = Both(_zha(), rng.choice([1, 2, 5]), rng.choice([64, 128]), page, rng.randint(300, 400), slots, 12,
             rng.choice([BF16, F32]), seed)
    m = b.model
    for step in range(60):
        empty = [s for s in range(slots) if not m.lens[s]]
        held = [s for s in range(slots) if m.lens[s]]
        what = rng.choice(["append", "append", "fork", "copy", "free", "compact"])
        if what == "append":
            seqs = rng.sample(range(slots), rng.randint(1, 4))
            T = rng.choice([1, 1, 5, page, 2 * page + 3])
            counts = [min(rng.randint(0, T), 12 * page - m.lens[s]) for s in seqs]
            if sum(-(-c // page) + 1 for c in counts) <= m.refs.count(0):
                b.append(seqs, T, counts)
        elif what in ("fork", "copy") and held and empty:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            src = [rng.choice(held + empty[:1]) for _ in dst]
            src = [s if s not in dst or not m.lens[s] else held[0] for s in src]
            if sum(len(m.rows[s]) for s in src) <= m.refs.count(0):
                (b.fork if what == "fork" else b.copy)(src, dst)
        elif what == "free" and held:
            b.free(rng.sample(range(slots), rng.randint(1, 3)))
        elif what == "compact":
            b.compact()
        if step % 6 == 5:
            b.check()
    b.gather(list(range(slots)), 12 * page)
    b.check()


def test_more_entries_and_pages_than_one_round_of_the_plan():
    # 1,500 slots (a list of more than 1,024), 40,000 pages (more than 32,768)
    zha = _zha()
    n, pages = 1500, 40000
    b = Both(zha, 1, 64, 8, pages, n + 2, 33000, F32)
    big = 32900 * 8 + 3
    b.model.rows[n], b.model.lens[n] = list(range(100, 33001)), big
    for p in range(100, 33001):
        b.model.refs[p] = 1
    b.pages.load(b.model.table().cuda(), _i32(b.model.lens))
    b.check()
    order = random.Random(1).sample(range(n), n)
    b.append(order, 1)
    b.check()
    b.free(order[::2] + [n])
    b.check()
    b.compact()
    b.check()
    b.append(order[::2], 3)
    b.fork([order[1]], [n + 1])
    b.check()


def test_copy_into_another_cache():
    zha = _zha()
    a = Both(zha, 2, 128, 16, 30, 4, 6, BF16, 1)
    b = Both(zha, 2, 128, 16, 9, 3, 3, BF16, 2)
    a.append([0, 1, 2], 40, [33, 16, 5])
    b.append([1], 4)
    b.pages.copy(b.K, b.V, _i32([0, 2]), _i32([2, 0]), source=a.pages, K_from=a.K, V_from=a.V)
    b.model.copy([0, 2], [2, 0], a.model)
    a.check()
    b.check()


def test_a_call_that_cannot_be_done_changes_nothing():
    zha = _zha()
    b = Both(zha, 1, 64, 8, 6, 5, 3, F32)
    b.append([0, 1], 10, [10, 8])
    b.check()
    Kn, Vn = (x.cuda() for x in b.new(2, 24))
    refused = [
        (lambda: b.pages.append(b.K, b.V, _i32([0, 5]), Kn, Vn, _i32([1, 1])), zha.ZHA_ERR_DEVICE),   # no such slot
        (lambda: b.pages.append(b.K, b.V, _i32([-1, 0]), Kn, Vn, _i32([1, 1])), zha.ZHA_ERR_DEVICE),
        (lambda: b.pages.append(b.K, b.V, _i32([0, 0]), Kn, Vn, _i32([1, 1])), zha.ZHA_ERR_DEVICE),   # named twice
        (lambda: b.pages.append(b.K, b.V, _i32([0, 1]), Kn, Vn, _i32([1, 25])), zha.ZHA_ERR_DEVICE),  # bad counts
        (lambda: b.pages.append(b.K, b.V, _i32([0, 1]), Kn, Vn, _i32([-1, 1])), zha.ZHA_ERR_DEVICE),
        (lambda: b.pages.append(b.K, b.V, _i32([0, 2]), Kn, Vn, _i32([15, 1])), zha.ZHA_ERR_CAPACITY),  # row full
        (lambda: b.pages.append(b.K, b.V, _i32([2, 3]), Kn, Vn, _i32([24, 8])), zha.ZHA_ERR_CAPACITY),  # pool empty
        (lambda: b.pages.fork(b.K, b.V, _i32([0]), _i32([1])), zha.ZHA_ERR_DEVICE),   # destination in use
        (lambda: b.pages.fork(b.K, b.V, _i32([0, 1]), _i32([2, 2])), zha.ZHA_ERR_DEVICE),
        (lambda: b.pages.fork(b.K, b.V, _i32([7]), _i32([2])), zha.ZHA_ERR_DEVICE),
        (lambda: b.pages.copy(b.K, b.V, _i32([0, 0]), _i32([2, 3])), zha.ZHA_ERR_CAPACITY),
        (lambda: b.pages.copy(b.K, b.V, _i32([1]), _i32([9])), zha.ZHA_ERR_DEVICE),
    ]
    for call, status in refused:
        call()
        assert b.pages.check() == status
        b.check()
    b.pages.free(_i32([9, 1, 1, 3]))  # a bad slot is skipped; twice and empty are fine
    assert b.pages.check() == zha.ZHA_ERR_DEVICE
    b.model.free([1])
    b.check()
    out = torch.full((2, 1, 8, 64), 3.0, device="cuda")
    b.pages.gather(b.K, b.V, _i32([0, 1]), out, out.clone())  # 10 tokens do not fit 8
    assert b.pages.check() == zha.ZHA_ERR_CAPACITY
    assert (out == 3.0).all()
    b.pages.gather(b.K, b.V, _i32([-3, 1]), out, out.clone())
    assert b.pages.check() == zha.ZHA_ERR_DEVICE
    assert (out == 3.0).all()
    b.append([4], 8)  # and the cache works on
    b.check()


def test_load_refuses_what_does_not_hold():
    zha = _zha()
    b = Both(zha, 1, 64, 8, 10, 4, 3, F32)
    good = torch.tensor([[4, 7, -1], [4, 2, 9], [-1, -1, -1], [9, 99, 99]], dtype=torch.int32)
    lens = [16, 20, 0, 0]
    b.pages.load(good.cuda(), _i32(lens))
    b.model.rows, b.model.lens = [[4, 7], [4, 2, 9], [], []], list(lens)
    for p, n in ((4, 2), (7, 1), (2, 1), (9, 1)):
        b.model.refs[p] = n
    b.check()
    b.pages.load(b.pages.table, b.pages.lens)  # its own state
    b.check()
    empty = PagesModel(10, 4, 3, 8, b.model.K, b.model.V)
    for bad_table, bad_lens in (([4, 10, -1], 16), ([4, -1, -1], 9), ([4, 7, 2], 25), ([4, 7, 2], -1), ([9, 3, -1], 3)):
        t = good.clone()
        t[0] = torch.tensor(bad_table)
        b.pages.load(t.cuda(), _i32([bad_lens] + lens[1:]))
        assert b.pages.check() == zha.ZHA_ERR_DEVICE
        empty.check(b.pages, b.K, b.V)
    b.pages.load(good.cuda(), _i32(lens))
    b.check()
    b.append([0, 1, 3], 3, [1, 3, 2])
    b.check()


def test_empty_lists_are_no_calls():
    b = Both(_zha(), 1, 64, 8, 4, 2, 2, F32)
    none = _i32([])
    b.append([0], 3)
    before = b.pages.launches
    e = torch.zeros((0, 1, 5, 64), device="cuda")
    b.pages.append(b.K, b.V, none, e, e)
    b.pages.append(b.K, b.V, _i32([0]), torch.zeros((1, 1, 0, 64), device="cuda"), torch.zeros((1, 1, 0, 64), device="cuda"))
    b.pages.fork(b.K, b.V, none, none)
    b.pages.copy(b.K, b.V, none, none)
    b.pages.free(none)
    b.pages.gather(b.K, b.V, none, e, e)
    assert b.pages.launches == before
    b.check()


def test_replayed_graph_moves_on():
    zha = _zha()
    b = Both(zha, 2, 64, 8, 64, 6, 8, BF16)
    b.append([0, 1], 13, [13, 8])
    src, dst, losers = _i32([0, 1, 0]), _i32([2, 3, 4]), _i32([2, 3, 4])
    Kn, Vn = b.new(5, 1)
    kd, vd, every = Kn.cuda(), Vn.cuda(), _i32([0, 1, 2, 3, 4])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.pages.fork(b.K, b.V, src, dst)
        b.pages.append(b.K, b.V, every, kd, vd)
        b.pages.free(losers)
    for step in range(9):
        Kn, Vn = b.new(5, 1)
        kd.copy_(Kn)
        vd.copy_(Vn)
        g.replay()
        b.model.fork([0, 1, 0], [2, 3, 4])
        b.model.append([0, 1, 2, 3, 4], Kn, Vn)
        b.model.free([2, 3, 4])
        b.check()


def test_rows_far_behind_two_to_the_31():
    # a pool of 2^31 and some elements: the last pages' rows
    zha = _zha()
    heads, d, page = 2, 128, 256
    num = 2 ** 31 // (heads * d * page) + 9
    pages = zha.Pages(heads, d, page, num, 3, 4, BF16)
    K, V = pages.pools()
    table = torch.full((3, 4), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor([num - 1, num - 2, num - 5])
    n = 2 * page + 5
    rows = torch.randn(1, heads, n + 3, d, device="cuda").to(BF16)
    for j, p in enumerate([num - 1, num - 2, num - 5]):
        m = min(page, n - j * page)
        K[p, :, :m] = rows[0, :, j * page:j * page + m]
        V[p, :, :m] = -rows[0, :, j * page:j * page + m]
    pages.load(table.cuda(), _i32([n, 0, 0]))
    pages.append(K, V, _i32([0]), rows[:, :, n:].contiguous(), -rows[:, :, n:].contiguous())
    out = torch.zeros((2, heads, n + 3, d), dtype=BF16, device="cuda")
    vout = torch.zeros_like(out)
    pages.fork(K, V, _i32([0]), _i32([1]))
    pages.gather(K, V, _i32([0, 1]), out, vout)
    assert torch.equal(out[:1], rows) and torch.equal(out[1:], rows) and torch.equal(vout[:1], -rows)
    pages.free(_i32([0]))
    pages.compact(K, V)
    assert pages.table[1].tolist() == [2, 1, 0, -1]
    out.zero_()
    pages.gather(K, V, _i32([1]), out[:1], vout[:1])
    assert torch.equal(out[:1], rows)
    assert pages.check() == zha.ZHA_OK


def test_launches_are_counted_from_several_threads():
    # calls that only read a cache may overlap; sixteen threads gather from one
    import threading
    zha = _zha()
    pages = zha.Pages(1, 64, 8, 4, 2, 2, torch.float32)
    K, V = pages.pools()
    pages.append(K, V, _i32([0]), torch.zeros((1, 1, 5, 64), device="cuda"), torch.zeros((1, 1, 5, 64), device="cuda"))
    seqs = _i32([0])
    out = [torch.empty((1, 1, 8, 64), device="cuda") for _ in "KV"]
    before, each, threads = pages.launches, 1000, 16
    call, args = zha.lib().zha_pages_gather, (K.data_ptr(), V.data_ptr(), seqs.data_ptr(), 1, out[0].data_ptr(),
                                              out[1].data_ptr(), 8, torch.cuda.current_stream().cuda_stream)
    start, bad = threading.Barrier(threads), []

    def work():
        with torch.cuda.device(0):
            start.wait()
            bad.extend(s for s in (call(pages.handle, *args) for _ in range(each)) if s)

    all_threads = [threading.Thread(target=work) for _ in range(threads)]
    for t in all_threads:
        t.start()
    for t in all_threads:
        t.join()
    assert not bad and pages.check() == zha.ZHA_OK
    assert pages.launches == before + each * threads
