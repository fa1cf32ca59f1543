"""The page operators through the C ABI against a plain implementation of the
table, the counts and the rows: random runs of reserving, writing, forking,
compacting and freeing, with shared pages, full pools and wrong arguments.
Everything is compared exactly."""
import numpy as np
import pytest

from tests import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from prompt_compression_b200 import build
    build.build_library()
    import prompt_compression_b200 as P
    P.spk_device_error(clear=True)
    return P


class Cache:
    """The cache on the GPU next to its plain copy."""

    def __init__(self, P, L, n_pages, hkv, page, d, n_seqs, max_pages, dtype="bfloat16", seed=0):
        import torch
        g = torch.Generator().manual_seed(seed)
        shape = (L, n_pages, hkv, page, d)
        kind = getattr(torch, dtype)
        self.kh = torch.randn(shape, generator=g).to(kind)
        self.vh = torch.randn(shape, generator=g).to(kind)
        self.k, self.v = self.kh.cuda(), self.vh.cuda()
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.book = R.Book(n_pages, n_seqs, max_pages, page)
        self.P, self.g, self.page, self.kind = P, g, page, kind

    @property
    def all(self):
        return self.k, self.v, self.refs, self.table, self.lens

    def i32(self, x):
        import torch
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def check(self):
        import torch
        torch.cuda.synchronize()
        assert self.refs.tolist() == self.book.refs
        assert self.table.tolist() == self.book.table
        assert self.lens.tolist() == self.book.lens
        assert torch.equal(self.k.cpu().view(torch.int16), self.kh.view(torch.int16))
        assert torch.equal(self.v.cpu().view(torch.int16), self.vh.view(torch.int16))

    def reserve(self, seqs, n_new):
        got = self.P.kv_pages_reserve(*self.all, self.i32(seqs), self.i32(n_new)).item()
        want = self.book.reserve(seqs, n_new)
        for a, b, r in self.book.copies:
            for x in (self.kh, self.vh):
                x[:, b, :, :r] = x[:, a, :, :r]
        assert got == want
        return got

    def rows(self, n, n_src):
        import torch
        L, _, H, _, d = self.k.shape
        return tuple(torch.randn((n, L, H, n_src, d), generator=self.g).to(self.kind) for _ in range(2))

    def write(self, seqs, n_src, idx=None, counts=None, units_per_idx=1):
        k, v = self.rows(len(seqs), n_src)
        L, _, H, _, _ = self.k.shape
        self.P.kv_pages_write(k.cuda(), v.cuda(), *self.all, self.i32(seqs), idx=None if idx is None else self.i32(idx),
                              counts=None if counts is None else self.i32(counts), units_per_idx=units_per_idx)
        n_idx = n_src if idx is None else len(idx[0])
        for i, s in enumerate(seqs):
            c = n_idx if counts is None else counts[i]
            for t in range(c):
                pos = self.book.lens[s] - c + t
                pg = self.book.table[s][pos // self.page]
                for l in range(L):
                    for h in range(H):
                        u = (i * L + l) * H + h
                        r = t if idx is None else idx[u // units_per_idx][t]
                        self.kh[l, pg, h, pos % self.page] = k[i, l, h, r]
                        self.vh[l, pg, h, pos % self.page] = v[i, l, h, r]

    def compact(self, src, dst, idx, units_per_idx):
        import torch
        got = self.P.kv_pages_compact(*self.all, self.i32(src), self.i32(dst), torch.tensor(idx, dtype=torch.int32).cuda(),
                                      units_per_idx=units_per_idx).item()
        want, old = self.book.compact(src, dst, len(idx[0]))
        assert got == want
        if want != 0:
            return got
        L, _, H, _, _ = self.k.shape
        kh, vh = self.kh.clone(), self.vh.clone()
        for i, b in enumerate(dst):
            for l in range(L):
                for h in range(H):
                    for t, r in enumerate(idx[((i * L + l) * H + h) // units_per_idx]):
                        a, z = old[i][r // self.page], self.book.table[b][t // self.page]
                        self.kh[l, z, h, t % self.page] = kh[l, a, h, r % self.page]
                        self.vh[l, z, h, t % self.page] = vh[l, a, h, r % self.page]
        return got

    def fork(self, src, dst, n_rows=None):
        got = self.P.kv_pages_fork(*self.all[2:], self.i32(src), self.i32(dst), page_rows=self.page,
                                   n_rows=None if n_rows is None else self.i32(n_rows)).item()
        assert got == self.book.fork(src, dst, n_rows)
        return got

    def free(self, seqs, keep=None):
        self.P.kv_pages_free(*self.all[2:], self.i32(seqs), page_rows=self.page,
                             keep_rows=None if keep is None else self.i32(keep))
        self.book.free(seqs, keep)

    def no_error(self):
        assert self.P.spk_device_error() == (0, 0)


@pytest.mark.parametrize("page,d,hkv,L", [(16, 64, 2, 1), (8, 128, 1, 2), (24, 8, 3, 1), (1, 16, 1, 1), (64, 64, 1, 1)])
def test_a_sequence_grows_row_by_row(P, page, d, hkv, L):
    c = Cache(P, L, 40, hkv, page, d, 3, 20, seed=page)
    for n in (1, page, 2, 3):
        if c.book.lens[1] + n > 20 * page:
            break
        assert c.reserve([1], [n]) == 0
        c.write([1], n)
        c.check()
    c.free([1], [1])
    c.check()
    c.free([1])
    c.check()
    assert sum(c.book.refs) == 0
    c.no_error()


def test_selected_rows_and_accepted_nodes_are_written(P):
    c = Cache(P, 2, 60, 2, 16, 64, 4, 8, seed=5)
    rng = np.random.default_rng(5)
    assert c.reserve([3, 0], [21, 21]) == 0
    idx = [sorted(rng.choice(50, 21, replace=False).tolist()) for _ in range(2 * 2 * 2)]
    c.write([3, 0], 50, idx=idx)                                    # a row list for each unit
    c.check()
    assert c.reserve([0, 3, 2], [3, 0, 1]) == 0                     # 0 .. 3 accepted nodes of trees of 7
    c.write([0, 3, 2], 7, idx=[[0, 4, 6], [1, 2, 3], [5, 0, 0]], counts=[3, 0, 1], units_per_idx=4)
    c.check()
    c.no_error()


def test_forks_share_pages_until_they_grow(P):
    c = Cache(P, 1, 50, 2, 16, 64, 6, 10, seed=6)
    assert c.reserve([0], [37]) == 0
    c.write([0], 37)
    c.fork([0, 0, 0], [1, 2, 3])
    c.check()
    assert c.book.refs[c.book.table[0][2]] == 4
    assert c.reserve([1, 2], [1, 20]) == 0                          # each leaves the shared last page
    c.write([1, 2], 20, counts=[1, 20])
    c.check()
    assert c.reserve([0, 3], [2, 2]) == 0                           # the last holder keeps it
    c.write([0, 3], 2)
    c.check()
    c.fork([1, 0, 3, 2], [0, 1, 2, 3])                              # sources that are destinations
    c.check()
    c.fork([2], [2], [5])                                           # onto itself, shortened
    c.fork([0], [4], [100])
    c.check()
    c.free([0, 1, 2, 3, 4, 0])                                      # one of them twice
    c.check()
    assert sum(c.book.refs) == 0
    c.no_error()


def test_only_the_first_rows_are_forked(P):
    c = Cache(P, 1, 30, 1, 8, 16, 4, 6, seed=7)
    assert c.reserve([0], [45]) == 0
    c.write([0], 45)
    c.fork([0, 0, 0], [1, 2, 3], [0, 16, 17])
    c.check()
    assert c.reserve([2, 3], [1, 1]) == 0                           # 16 rows: a new page; 17: its own copy of the third
    c.write([2, 3], 1)
    c.check()
    c.no_error()


@pytest.mark.parametrize("page,keep", [(16, 20), (8, 1), (24, 48), (16, 0)])
def test_compaction(P, page, keep):
    c = Cache(P, 2, 80, 2, page, 64, 6, 20, seed=page + keep)
    rng = np.random.default_rng(keep)
    assert c.reserve([0, 1], [100, 61]) == 0
    c.write([0, 1], 100, counts=[100, 61])

    def pick(n, lists):
        return [sorted(rng.choice(n, keep, replace=False).tolist()) for _ in range(lists)]

    c.compact([0, 1], [2, 3], pick(61, 2 * 4) if keep else [[]] * 8, 1)          # a row list for each unit
    c.check()
    c.compact([0, 1], [2, 3], pick(61, 2) if keep else [[]] * 2, 4)              # one for each sequence; onto old pages
    c.check()
    c.fork([0], [4])
    c.compact([1, 0], [1, 0], pick(61, 2) if keep else [[]] * 2, 4)              # in place; 4 keeps the pages
    c.check()
    c.compact([4, 4], [5, 1], pick(100, 2) if keep else [[]] * 2, 4)             # a source twice
    c.check()
    c.free([0, 1, 2, 3, 4, 5])
    c.check()
    assert sum(c.book.refs) == 0
    c.no_error()


def test_too_few_pages_change_nothing(P):
    c = Cache(P, 1, 10, 1, 16, 64, 4, 12, seed=8)
    assert c.reserve([0, 1], [70, 40]) == 0                         # 5 + 3 pages
    c.write([0, 1], 70, counts=[70, 40])
    assert c.reserve([2, 0, 1], [33, 11, 0]) == 2                   # 3 + 1 wanted, 2 free
    c.check()
    c.fork([0], [3])
    assert c.reserve([3, 0, 2], [1, 1, 32]) == 1                    # a copy and 2 pages wanted
    c.check()
    assert c.compact([0, 1], [2, 3], [list(range(30))] * 2, 1) == 2
    c.check()
    assert c.compact([0], [1], [list(range(48))], 1) == 0           # what 1 held is enough with the rest
    c.check()
    c.no_error()


def test_a_pool_of_many_pages(P):
    c = Cache(P, 1, 9001, 1, 1, 16, 1024, 40, seed=9)
    rng = np.random.default_rng(9)
    seqs = rng.permutation(1024).tolist()
    assert c.reserve(seqs, [int(x) for x in rng.integers(0, 8, 1024)]) == 0
    c.check()
    c.free(seqs[::3])
    c.check()
    assert c.reserve(seqs, [int(x) for x in rng.integers(0, 5, 1024)]) == 0
    c.check()
    c.fork(seqs[:500], seqs[500:1000])
    c.check()
    c.no_error()


def test_wrong_arguments_change_nothing_and_are_recorded(P):
    c = Cache(P, 1, 20, 1, 16, 64, 4, 5, seed=10)
    assert c.reserve([0, 1], [20, 20]) == 0
    c.write([0, 1], 20)
    E = P.binding.SPK_ERR_ARG
    for call in (lambda: P.kv_pages_reserve(*c.all, c.i32([0, 0]), c.i32([1, 1])),
                 lambda: P.kv_pages_reserve(*c.all, c.i32([0, 4]), c.i32([1, 1])),
                 lambda: P.kv_pages_reserve(*c.all, c.i32([-1]), c.i32([1])),
                 lambda: P.kv_pages_reserve(*c.all, c.i32([0]), c.i32([-1])),
                 lambda: P.kv_pages_reserve(*c.all, c.i32([0]), c.i32([61])),
                 lambda: P.kv_pages_fork(*c.all[2:], c.i32([0, 1]), c.i32([2, 2]), page_rows=16),
                 lambda: P.kv_pages_fork(*c.all[2:], c.i32([9]), c.i32([2]), page_rows=16),
                 lambda: P.kv_pages_fork(*c.all[2:], c.i32([0]), c.i32([2]), page_rows=16, n_rows=c.i32([-1])),
                 lambda: P.kv_pages_compact(*c.all, c.i32([0, 1]), c.i32([2, 2]), c.i32([[0], [0]])),
                 lambda: P.kv_pages_compact(*c.all, c.i32([0]), c.i32([4]), c.i32([[0]]))):
        assert call().item() == -1
        assert P.spk_device_error(clear=True)[0] == E
        c.check()
    P.kv_pages_free(*c.all[2:], c.i32([7]), page_rows=16)
    assert P.spk_device_error(clear=True)[0] == E
    c.check()


def test_rows_that_may_not_be_written(P):
    import torch
    c = Cache(P, 1, 20, 1, 16, 64, 4, 5, seed=11)
    E = P.binding.SPK_ERR_ARG
    assert c.reserve([0], [20]) == 0
    c.write([0], 20)
    c.fork([0], [1])
    k, v = (x.cuda() for x in c.rows(1, 4))
    for seqs, idx, counts in (([1], None, None),                    # a shared page
                              ([2], None, None),                    # fewer rows than are written
                              ([9], None, None),                    # no such sequence
                              ([1], [[0, 1, 2, 4]], None),          # no such row (and a shared page)
                              ([0], None, [5])):                    # more than there are
        P.kv_pages_write(k, v, *c.all, c.i32(seqs), idx=None if idx is None else c.i32(idx),
                         counts=None if counts is None else c.i32(counts))
        assert P.spk_device_error(clear=True)[0] == E
        c.check()
    c.free([1])
    P.kv_pages_write(k, v, *c.all, c.i32([0]), idx=c.i32([[3, -1, 1, 4]]))
    assert P.spk_device_error(clear=True)[0] == E
    pg = c.book.table[0][1]
    c.kh[:, pg, :, 0], c.kh[:, pg, :, 2] = k.cpu()[0, :, :, 3], k.cpu()[0, :, :, 1]
    c.vh[:, pg, :, 0], c.vh[:, pg, :, 2] = v.cpu()[0, :, :, 3], v.cpu()[0, :, :, 1]
    c.check()
    P.kv_pages_compact(*c.all, c.i32([0]), c.i32([2]), c.i32([[0, 20, 19]]))     # row 20 does not exist
    assert P.spk_device_error(clear=True)[0] == E
    torch.cuda.synchronize()
    a, z = c.table[0].tolist(), c.table[2].tolist()
    assert torch.equal(c.k[0, z[0], 0, 0], c.k[0, a[0], 0, 0]) and torch.equal(c.k[0, z[0], 0, 2], c.k[0, a[1], 0, 3])
    assert torch.equal(c.k[0, z[0], 0, 1].cpu(), c.kh[0, z[0], 0, 1])


def test_a_sequence_listed_twice_is_written_by_its_first_entry(P):
    c = Cache(P, 1, 30, 2, 16, 64, 4, 5, seed=13)
    assert c.reserve([2, 0], [20, 20]) == 0
    k, v = c.rows(3, 20)
    P.kv_pages_write(k.cuda(), v.cuda(), *c.all, c.i32([2, 0, 2]))
    assert P.spk_device_error(clear=True)[0] == P.binding.SPK_ERR_ARG
    for i, s in enumerate([2, 0]):
        for t in range(20):
            pg = c.book.table[s][t // 16]
            c.kh[:, pg, :, t % 16], c.vh[:, pg, :, t % 16] = k[i, :, :, t], v[i, :, :, t]
    c.check()


def test_bookkeeping_is_captured_and_replayed(P):
    # a decoding loop's step: room for one row, the row; the graph's second run
    # takes the next page where the sequence has come to one
    import torch
    c = Cache(P, 1, 20, 1, 8, 64, 2, 8, seed=12)
    seqs, one, res = c.i32([1]), c.i32([1]), c.i32([5])
    k, v = (x.cuda() for x in c.rows(1, 1))
    ws = torch.empty(P.kv_pages_workspace_size(P.pages_shape(*c.all), 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.kv_pages_reserve(*c.all, seqs, one, result=res, workspace=ws)
        P.kv_pages_write(k, v, *c.all, seqs)
    for step in range(17):
        graph.replay()
        assert c.book.reserve([1], [1]) == 0
        pg = c.book.table[1][step // 8]
        c.kh[:, pg, :, step % 8], c.vh[:, pg, :, step % 8] = k.cpu()[0, :, :, 0], v.cpu()[0, :, :, 0]
    c.check()
    assert res.item() == 0
    c.no_error()


@pytest.mark.parametrize("seed", range(4))
def test_random_runs(P, seed):
    rng = np.random.default_rng(seed)
    page = int(rng.choice([1, 8, 16, 24]))
    c = Cache(P, int(rng.integers(1, 3)), 60, int(rng.integers(1, 3)), page, 16, 7, 12, seed=seed)
    L, _, H, _, _ = c.k.shape
    for _ in range(25):
        n = int(rng.integers(1, 4))
        a, b = rng.permutation(7)[:n].tolist(), rng.permutation(7)[:n].tolist()
        kind = rng.integers(0, 4)
        if kind == 0:
            new = [int(min(x, 12 * page - c.book.lens[s])) for s, x in zip(a, rng.integers(0, 3 * page + 1, n))]
            if c.reserve(a, new) == 0 and max(new) > 0:
                c.write(a, max(new), counts=new)
        elif kind == 1:
            c.fork(a, b, [int(x) for x in rng.integers(0, 8 * page, n)] if rng.random() < 0.5 else None)
        elif kind == 2:
            c.free(a, [int(x) for x in rng.integers(0, 4 * page, n)])
        elif min(c.book.lens[s] for s in a) > 0:
            m = min(c.book.lens[s] for s in a)
            keep = int(rng.integers(1, m + 1))
            per = bool(rng.random() < 0.5)
            idx = [sorted(rng.choice(m, keep, replace=False).tolist()) for _ in range(n * (L * H if per else 1))]
            c.compact(a, b, idx, 1 if per else L * H)
        c.check()
    c.no_error()


def test_the_binding_refuses_what_does_not_fit(P):
    import torch
    c = Cache(P, 2, 10, 2, 16, 64, 3, 4)
    s, i32 = c.i32([0, 1]), c.i32
    k = torch.zeros((2, 2, 2, 5, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 2, 4, 3, 64), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros((2, 2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    book = (c.refs, c.table, c.lens)
    bad = [
        ("n_new has", lambda: P.kv_pages_reserve(*c.all, s, i32([1]))),
        ("int|Int", lambda: P.kv_pages_reserve(*c.all, s, i32([1, 1]).long())),
        ("cuda:0", lambda: P.kv_pages_reserve(*c.all, s.cpu(), i32([1, 1]))),
        ("n_new is required", lambda: P.kv_pages_reserve(*c.all, s, None)),
        ("result has", lambda: P.kv_pages_reserve(*c.all, s, i32([1, 1]), result=i32([1, 1]))),
        ("page_refs has", lambda: P.kv_pages_reserve(c.k, c.v, c.refs[:9], c.table, c.lens, s, s)),
        ("seq_lens has", lambda: P.kv_pages_reserve(c.k, c.v, c.refs, c.table, c.lens[:2], s, s)),
        ("same dtype", lambda: P.kv_pages_reserve(c.k, c.v.half(), *book, s, s)),
        ("contiguous", lambda: P.kv_pages_reserve(c.k, c.v, c.refs, torch.zeros((4, 3), dtype=torch.int32, device="cuda").t(),
                                                  c.lens, s, s)),
        ("multiple", lambda: P.kv_pages_write(k, k, *c.all, s, units_per_idx=3)),
        ("k and v are", lambda: P.kv_pages_write(k[:1], k[:1], *c.all, s)),
        ("BFloat16", lambda: P.kv_pages_write(k.half(), k.half(), *c.all, s)),
        ("idx has", lambda: P.kv_pages_write(k, k, *c.all, s, idx=i32([[0, 1]]), units_per_idx=1)),
        ("counts has", lambda: P.kv_pages_write(k, k, *c.all, s, counts=i32([1]))),
        ("dst has", lambda: P.kv_pages_compact(*c.all, s, i32([2]), i32([[0], [1]]), units_per_idx=4)),
        ("n_rows has", lambda: P.kv_pages_fork(*book, s, i32([1, 2]), page_rows=16, n_rows=i32([1]))),
        ("out of range", lambda: P.kv_pages_free(*book, s, page_rows=1 << 40)),
        ("disagree", lambda: P.tree_attention(q[:, :1].contiguous(), c.k, c.v, c.table, c.lens)),
        ("Half", lambda: P.tree_attention(q.float(), c.k.float(), c.v.float(), c.table, c.lens)),
        ("BFloat16", lambda: P.tree_attention(q, c.k.half(), c.v.half(), c.table, c.lens)),
        ("together", lambda: P.tree_attention(q, c.k, c.v, c.table, c.lens, t)),
        ("must be", lambda: P.tree_attention(q, c.k, c.v, c.table, c.lens, t[:, :, :, :2], t[:, :, :, :2])),
        ("mask has", lambda: P.tree_attention(q, c.k, c.v, c.table, c.lens, t, t, mask=i32([[1, 1, 1]]))),
        ("lse2 has", lambda: P.tree_attention(q, c.k, c.v, c.table, c.lens, lse2=torch.zeros(5, device="cuda"))),
        ("out has", lambda: P.tree_attention(q, c.k, c.v, c.table, c.lens, out=q[:1])),
        ("contiguous", lambda: P.tree_attention(q.transpose(2, 3).contiguous().transpose(2, 3), c.k, c.v, c.table, c.lens)),
        ("depth has", lambda: P.tree_mask(i32([[-1, 0]]), depth=i32([0]))),
    ]
    for needle, call in bad:
        with pytest.raises(ValueError, match=needle):
            call()
    for status, call in ((P.binding.SPK_ERR_WORKSPACE, lambda: P.kv_pages_reserve(*c.all, s, s, workspace=k[0, 0, 0, 0, :2])),
                         (P.binding.SPK_ERR_ARG, lambda: P.kv_pages_free(*book, s, page_rows=0)),
                         (P.binding.SPK_ERR_UNSUPPORTED, lambda: P.tree_mask(torch.zeros((1, 1025), dtype=torch.int32, device="cuda")))):
        with pytest.raises(P.SpeckvError) as e:
            call()
        assert e.value.status == status
    c.check()
    c.no_error()


@pytest.mark.parametrize("length", [-1, 81, 1 << 30])
def test_a_length_beyond_the_table_is_refused(P, length):
    c = Cache(P, 1, 20, 1, 16, 64, 4, 5, seed=14)
    assert c.reserve([0, 1], [20, 20]) == 0
    c.write([0, 1], 20)
    c.lens[1] = length                                              # not a length that five pages of 16 rows can have
    c.book.lens[1] = length
    for call in (lambda: P.kv_pages_compact(*c.all, c.i32([0, 1]), c.i32([2, 3]), c.i32([[0, 19], [100, 19]])),
                 lambda: P.kv_pages_compact(*c.all, c.i32([1]), c.i32([1]), c.i32([[max(length - 1, 0)]])),
                 lambda: P.kv_pages_fork(*c.all[2:], c.i32([1]), c.i32([2]), page_rows=16),
                 lambda: P.kv_pages_reserve(*c.all, c.i32([1]), c.i32([1]))):
        assert call().item() == -1
        assert P.spk_device_error(clear=True)[0] == P.binding.SPK_ERR_ARG
        c.check()


def _sorted_rows(rng, n, keep, lists):
    return [sorted(rng.choice(n, keep, replace=False).tolist()) for _ in range(lists)]


def test_compaction_of_hundreds_of_sequences(P):
    # tables large enough for the bookkeeping in a cluster of CTAs: into others, in place,
    # a source twice, too few free pages, refused lists
    c = Cache(P, 1, 2000, 1, 2, 16, 700, 12, seed=15)
    rng = np.random.default_rng(15)
    seqs = rng.permutation(700).tolist()
    a, b = seqs[:300], seqs[300:600]
    assert c.reserve(a, [int(x) for x in rng.integers(5, 9, 300)]) == 0
    c.check()
    assert c.compact(a, b, _sorted_rows(rng, 5, 3, 300), 1) == 0
    c.check()
    assert c.compact(a[:200], a[:200], _sorted_rows(rng, 5, 4, 200), 1) == 38    # in place: the new pages come first
    c.check()
    # a source a hundred times
    assert c.compact([a[0]] * 100 + a[100:200], b[200:300] + b[:100], _sorted_rows(rng, 4, 2, 200), 1) == 0
    c.check()
    assert c.compact(b[100:300], a[100:300], _sorted_rows(rng, 2, 1, 200), 1) == 0
    c.check()
    c.fork(a[:250], seqs[440:690])                                               # shared pages
    c.check()
    assert c.compact(a[:250], a[:250], _sorted_rows(rng, 1, 1, 250), 1) == 0     # in place, the others keep the pages
    c.check()
    c.no_error()
    E = P.binding.SPK_ERR_ARG
    i32, rows = c.i32, c.i32([[0]] * 250)
    dup = a[1:250] + [a[1]]
    for call in (lambda: P.kv_pages_compact(*c.all, i32(a[:250]), i32(dup), rows),
                 lambda: P.kv_pages_compact(*c.all, i32(a[:249] + [700]), i32(b[:250]), rows),
                 lambda: P.kv_pages_fork(*c.all[2:], i32(a[:250]), i32(dup), page_rows=2),
                 lambda: P.kv_pages_fork(*c.all[2:], i32(a[:249] + [-1]), i32(b[:250]), page_rows=2)):
        assert call().item() == -1
        assert P.spk_device_error(clear=True)[0] == E
        c.check()


def test_refusals_with_a_pool_of_many_pages(P):
    c = Cache(P, 1, 9001, 1, 1, 16, 64, 300, seed=16)
    assert c.reserve(list(range(30)), [300] * 30) == 0                           # 9000 of 9001 pages
    c.check()
    assert c.reserve([30, 31], [1, 1]) == 1
    c.check()
    assert c.compact([0, 1], [32, 33], [[0, 5, 7]] * 2, 1) == 5
    c.check()
    assert c.compact([0, 1], [0, 1], [[0, 5, 7]] * 2, 1) == 5                    # in place: the new pages come first
    c.check()
    assert c.compact([0, 1], [2, 3], [[0, 5, 299]] * 2, 1) == 0                  # what 2 and 3 held is enough
    c.check()
    c.no_error()
    E = P.binding.SPK_ERR_ARG
    for call in (lambda: P.kv_pages_reserve(*c.all, c.i32([5, 5]), c.i32([0, 0])),
                 lambda: P.kv_pages_reserve(*c.all, c.i32([64]), c.i32([1])),
                 lambda: P.kv_pages_compact(*c.all, c.i32([0, 1]), c.i32([4, 4]), c.i32([[0], [0]])),
                 lambda: P.kv_pages_fork(*c.all[2:], c.i32([0, 1]), c.i32([4, 4]), page_rows=1)):
        assert call().item() == -1
        assert P.spk_device_error(clear=True)[0] == E
        c.check()
