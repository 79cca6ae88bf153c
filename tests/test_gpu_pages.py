"""Page operations against a plain Python allocator, exactly."""
import numpy as np
import pytest
import torch

import synth
from _dense_util import check, queries, reference

pytestmark = pytest.mark.gpu
DEV_SLOT, DEV_PAGE, DEV_LEN, DEV_POOL = 0x1, 0x2, 0x8, 0x40


@pytest.fixture(scope="module")
def csa2():
    import fp4_kv_cache_nvfp4_b200 as m
    assert torch.cuda.is_available()
    m.lib()
    return m


class Pool:
    """Caches, table, counts and lengths on the GPU, and the same state in numpy."""

    def __init__(self, csa2, lens, rows, n_pages, page=8, cols=None, caches=1, idx=True, pooled=True, seed=0):
        self.csa2, self.page, self.n_pages = csa2, page, n_pages
        g = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.cols = cols or max(need + [1]) + 1
        self.table = np.full((rows, self.cols), -1, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.lens = np.zeros(rows, np.int32)
        perm = g.permutation(n_pages)
        o = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[o:o + n]
            self.refs[perm[o:o + n]] = 1
            self.lens[b] = lens[b]
            o += n
        r = lambda *s: g.integers(0, 256, s, dtype=np.uint8)  # noqa: E731
        n = n_pages * page
        self.planes = [[r(n, 128), r(n, 16)] + ([r(n, 128)] if idx else []) + ([r(n // 8, 128)] if idx and pooled else [])
                       for _ in range(caches)]
        self.d_table = torch.from_numpy(self.table.copy()).cuda()
        self.d_refs = torch.from_numpy(self.refs.copy()).cuda()
        self.d_lens = torch.from_numpy(self.lens.copy()).cuda()
        self.d_planes = [[torch.from_numpy(p.copy()).cuda() for p in ps] for ps in self.planes]
        v16 = lambda p: p.view(torch.int16)  # noqa: E731
        self.caches = [csa2.KVCache.from_tensors(p[0], p[1], self.d_table, page, idx_k=v16(p[2]) if len(p) > 2 else None,
                                                 pooled=v16(p[3]) if len(p) > 3 else None) for p in self.d_planes]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((csa2.kv_pages_workspace_bytes(n_pages, 1024),), 0xFF, dtype=torch.uint8, device="cuda")

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def copy_page(self, s, d):
        for ps in self.planes:
            for p in ps:
                v = p.reshape(self.n_pages, -1)
                v[d] = v[s]

    # the plain forms
    def fork(self, parents, children):
        rows, n, pg = len(self.lens), len(parents), self.page
        free = [p for p in range(self.n_pages) if self.refs[p] == 0]
        ok, want = [], 0
        before = self.lens.copy()
        for i, (f, c) in enumerate(zip(parents, children)):
            if not (0 <= c < rows and 0 <= f < rows) or before[c] != 0 or c in children[:i] or c in parents:
                continue
            L = int(before[f])
            if L < 0 or -(-L // pg) > self.cols:
                continue
            page = None
            if L % pg:
                tail = self.table[f, L // pg]
                if not 0 <= tail < self.n_pages:
                    continue
                want += 1
                if want > len(free):
                    continue
                page = free[want - 1]
            ok.append((f, c, L, page))
        for f, c, L, page in ok:
            full = L // pg
            self.table[c] = -1
            for j in range(full):
                p = self.table[f, j]
                if 0 <= p < self.n_pages:
                    self.table[c, j] = p
                    self.refs[p] += 1
            if page is not None:
                self.copy_page(self.table[f, full], page)
                self.table[c, full] = page
                self.refs[page] = 1
            self.lens[c] = L

    def free(self, seqs):
        for b in seqs:
            if 0 <= b < len(self.lens):
                for j in range(self.cols):
                    p = self.table[b, j]
                    if 0 <= p < self.n_pages and self.refs[p] > 0:
                        self.refs[p] -= 1
                    self.table[b, j] = -1
                self.lens[b] = 0

    def compact(self):
        live = [p for p in range(self.n_pages) if self.refs[p] > 0]
        n = len(live)
        holes, high = [p for p in range(n) if self.refs[p] <= 0], [p for p in live if p >= n]
        m = np.full(self.n_pages, -1, np.int32)
        m[live] = live
        for s, d in zip(high, holes):
            m[s] = d
            self.copy_page(s, d)
            self.refs[d], self.refs[s] = self.refs[s], 0
        for r in self.table:
            for j in range(self.cols):
                r[j] = m[r[j]] if 0 <= r[j] < self.n_pages else -1
        return m, n

    # the calls
    def d_fork(self, parents, children):
        self.csa2.kv_pages_fork(self.caches, self.d_refs, self.d_lens, self.i32(parents), self.i32(children), self.ws,
                                err=self.err)

    def d_free(self, seqs):
        self.csa2.kv_pages_free(self.caches[0], self.d_refs, self.d_lens, self.i32(seqs), err=self.err)

    def d_compact(self):
        m, n = self.i32([7] * self.n_pages), self.i32([7])
        self.csa2.kv_pages_compact(self.caches, self.d_refs, m, n, self.ws, err=self.err)
        return m, n

    def check(self, err=0, what=""):
        torch.cuda.synchronize()
        assert int(self.err.item()) == err, what
        self.err.zero_()
        assert np.array_equal(self.d_table.cpu().numpy(), self.table), f"{what}: table"
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs), f"{what}: counts"
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens), f"{what}: lengths"
        for ps, qs in zip(self.planes, self.d_planes):
            for k, (p, q) in enumerate(zip(ps, qs)):
                assert np.array_equal(q.cpu().numpy(), p), f"{what}: plane {k}"


@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("idx,pooled", [(True, True), (True, False), (False, False)])
def test_copy(csa2, page, idx, pooled):
    p = Pool(csa2, [], 1, 37, page, caches=2, idx=idx, pooled=pooled)
    src, dst = [3, 36, -1, 5, 9, 11], [0, 1, 2, -1, 35, 11]
    p.csa2.kv_pages_copy(p.caches, p.i32(src), p.i32(dst), err=p.err)
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            p.copy_page(s, d)
    p.check(0)
    p.csa2.kv_pages_copy(p.caches, p.i32([37, 4, -2, 6]), p.i32([0, 37, 3, 7]), err=p.err)
    p.copy_page(6, 7)
    p.check(DEV_PAGE)


@pytest.mark.parametrize("caches", [1, 3])
@pytest.mark.parametrize("page,lens", [(8, [1]), (8, [8, 7, 9, 40]), (64, [64, 1, 200, 0, 333]), (16, [100] * 20)])
def test_fork_free_compact_together(csa2, page, lens, caches):
    """Forks of forks, frees, compactions and forks again, as a server would run them."""
    n = len(lens)
    p = Pool(csa2, lens, 4 * n, sum(-(-x // page) for x in lens) * 3 + 5, page, caches=caches, seed=n)
    a, b, c = list(range(n)), list(range(n, 2 * n)), list(range(2 * n, 3 * n))
    p.d_fork(a, b); p.fork(a, b); p.check(0, "fork")  # noqa: E702
    rev = b[::-1]
    p.d_fork([rev[0]] * n, c); p.fork([rev[0]] * n, c); p.check(0, "one parent, many children")  # noqa: E702
    p.d_free(a); p.free(a); p.check(0, "free the first")  # noqa: E702
    m, live = p.d_compact()
    want, n_live = p.compact()
    p.check(0, "compact")
    assert np.array_equal(m.cpu().numpy(), want) and int(live) == n_live
    p.d_fork(c, a); p.fork(c, a); p.check(0, "fork into freed rows")  # noqa: E702
    p.d_free(a + b + c + [-1]); p.free(a + b + c); p.check(0, "free all")  # noqa: E702
    assert (p.refs == 0).all()
    m, live = p.d_compact()
    p.check(0, "nothing live")
    assert int(live) == 0 and (m == -1).all()


@pytest.mark.parametrize("P", [3 * 4096 + 77, 18 * 4096 + 5, 4096])
def test_large_pool_many_chunks(csa2, P):
    """Pools of one, several and many chunks of the scans (each counts its own way), holes everywhere."""
    page = 8
    p = Pool(csa2, [], 300, P, page, cols=41, idx=False)
    g = np.random.default_rng(1)
    used = g.permutation(P)[:min(9000, P - 100)]
    for b in range(250 if P > 9000 else 100):
        p.table[b, :36] = used[36 * b:36 * b + 36]
        p.refs[used[36 * b:36 * b + 36]] = 1
        p.lens[b] = 36 * page - b % page
    p.d_table.copy_(torch.from_numpy(p.table)), p.d_refs.copy_(torch.from_numpy(p.refs))
    p.d_lens.copy_(torch.from_numpy(p.lens))
    par, chi = list(range(0, 50)), list(range(250, 300))
    p.d_fork(par, chi); p.fork(par, chi); p.check(0, "fork")  # noqa: E702
    gone = list(range(3, 200 if P > 9000 else 90, 2))
    p.d_free(gone); p.free(gone); p.check(0, "free")  # noqa: E702
    m, live = p.d_compact()
    want, n = p.compact()
    p.check(0, "compact")
    assert np.array_equal(m.cpu().numpy(), want) and int(live) == n


def test_fork_refusals_on_the_device(csa2):
    mk = lambda: Pool(csa2, [20, 8, 33], 8, 24, 8)  # noqa: E731
    for parents, children, err in (
            ([0, 0], [3, 3], DEV_SLOT),           # the same child twice: the first counts
            ([0, 3], [3, 4], DEV_SLOT),           # a child that is a parent
            ([0], [0], DEV_SLOT),                 # itself
            ([0], [1], DEV_SLOT),                 # a row in use
            ([-1, 8, 0, -1, 1], [3, 4, 8, -1, 5], DEV_SLOT)):
        p = mk()
        p.d_fork(parents, children); p.fork(parents, children); p.check(err, str((parents, children)))  # noqa: E702
    p = mk()
    p.lens[1] = -3
    p.lens[2] = 8 * p.cols + 1
    p.d_lens.copy_(torch.from_numpy(p.lens))
    p.d_fork([1, 2, 0], [3, 4, 5]); p.fork([1, 2, 0], [3, 4, 5]); p.check(DEV_LEN)  # noqa: E702
    p = mk()
    p.table[0, 1], p.table[2, 4] = 99, -1         # a full page and a partial last page that are missing
    p.d_table.copy_(torch.from_numpy(p.table))
    p.d_fork([0, 2], [3, 4]); p.fork([0, 2], [3, 4]); p.check(DEV_PAGE)  # noqa: E702


def test_a_main_kv_in_pinned_host_memory(csa2):
    """Forks and compactions of a tiered cache: codes and scales in mapped host memory."""
    table = torch.tensor([[5, 2, -1], [-1, -1, -1]], dtype=torch.int32).cuda()
    c = csa2.KVCache(6, 8, table, main_kv_on_host=True)
    g = torch.Generator().manual_seed(1)
    for t in (c.codes, c.scales):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    want = [t.clone() for t in (c.codes, c.scales)]
    refs = torch.tensor([0, 0, 1, 0, 0, 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([13, 0], dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(csa2.kv_pages_workspace_bytes(6, 1), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    csa2.kv_pages_fork([c], refs, lens, i32([0]), i32([1]), ws, err=err)
    m, n = i32([0] * 6), i32([0])
    csa2.kv_pages_compact([c], refs, m, n, ws, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and int(n) == 3 and m.tolist() == [0, -1, 2, -1, -1, 1]
    assert c.page_table.tolist() == [[1, 2, -1], [1, 0, -1]] and refs.tolist() == [1, 2, 1, 0, 0, 0]
    for t, w in zip((c.codes, c.scales), want):
        v, w = t.view(6, -1), w.view(6, -1)
        assert torch.equal(v[0], w[2]) and torch.equal(v[1], w[5]) and torch.equal(v[2], w[2])


def test_caches_that_kernels_cannot_write_are_refused(csa2):
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)  # noqa: E731
    c = csa2.KVCache.from_tensors(z(64, 128), z(64, 16), z(2, 4, dt=torch.int32).cuda(), 8)
    refs, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (8, 2))
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(csa2.kv_pages_workspace_bytes(8, 1), dtype=torch.uint8, device="cuda")
    for bad in (lambda: csa2.kv_pages_copy([c], one, one), lambda: csa2.kv_pages_fork([c], refs, lens, one, one, ws)):
        with pytest.raises(ValueError):
            bad()


def test_fork_until_the_pool_is_empty(csa2):
    p = Pool(csa2, [20, 16, 33], 10, 12, 8)       # 3 + 2 + 5 pages, two free
    par, chi = [0, 1, 2, 0, 1], [3, 4, 5, 6, 7]
    p.d_fork(par, chi); p.fork(par, chi); p.check(DEV_POOL)  # noqa: E702
    assert list(p.lens[3:8]) == [20, 16, 33, 0, 16]  # no page for the fourth; none needed by the fifth


def test_free_reports_and_frees_once(csa2):
    p = Pool(csa2, [20, 16, 33], 5, 24, 8)
    p.d_free([0, 0, 2, 0]); p.free([0, 0, 2, 0]); p.check(0, "listed twice")  # noqa: E702
    p.d_free([-1, 5, -7]); p.check(DEV_SLOT)  # noqa: E702
    p.refs[p.table[1, 0]] = 0                     # held, but not counted
    p.table[1, 1] = 24
    p.d_refs.copy_(torch.from_numpy(p.refs)), p.d_table.copy_(torch.from_numpy(p.table))
    p.d_free([1]); p.free([1]); p.check(DEV_PAGE)  # noqa: E702


def test_compact_drops_entries_that_name_no_live_page(csa2):
    p = Pool(csa2, [20, 16, 33], 4, 24, 8)
    dead = int(np.nonzero(p.refs == 0)[0][0])
    p.table[3, 0], p.table[3, 1], p.table[3, 2] = dead, 24, -9
    p.d_table.copy_(torch.from_numpy(p.table))
    p.d_compact(); p.compact(); p.check(DEV_PAGE)  # noqa: E702


def test_captured_beam_step(csa2):
    """Fork and free in one graph, replayed on other parents."""
    p = Pool(csa2, [37, 37, 37, 37], 8, 60, 8, caches=2)
    par, chi, old = p.i32([0, 0, 0, 0]), p.i32([4, 5, 6, 7]), p.i32([0, 1, 2, 3])

    def step():
        csa2.kv_pages_fork(p.caches, p.d_refs, p.d_lens, par, chi, p.ws, err=p.err)
        csa2.kv_pages_free(p.caches[0], p.d_refs, p.d_lens, old, err=p.err)

    par.fill_(-1), chi.fill_(-1), old.fill_(-1)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k, (pp, cc, oo) in enumerate((([1, 1, 2, 0], [4, 5, 6, 7], [0, 1, 2, 3]), ([5, 7, 5, 4], [0, 1, 2, 3], [4, 5, 6, 7]))):
        par.copy_(p.i32(pp)), chi.copy_(p.i32(cc)), old.copy_(p.i32(oo))
        g.replay()
        p.fork(pp, cc)
        p.free(oo)
        p.check(0, f"replay {k}")


def test_append_fork_append_attend(csa2):
    """The set as it is used: two hypotheses of one prompt append different
    tokens, attend over what they hold, then the pages are compacted and they
    attend again with the same result."""
    page, L, seed = 16, 100, 1001
    table = torch.full((3, 10), -1, dtype=torch.int32)
    table[0, :7] = torch.tensor([20, 3, 17, 9, 25, 1, 14])
    cache = csa2.KVCache(32, page, table)
    refs = torch.zeros(32, dtype=torch.int32, device="cuda")
    refs[table[0, :7].long().cuda()] = 1
    lens = torch.tensor([L, 0, 0], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(csa2.kv_pages_workspace_bytes(32, 2), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def append(b, start, kv, ik):
        t = cache.page_table.cpu().numpy()
        sl = synth.slots(t, b, np.arange(start, start + len(kv)), page)
        csa2.kv_quant_append(cache, torch.from_numpy(kv).cuda(), torch.from_numpy(ik.view(np.int16)).cuda(),
                             torch.from_numpy(sl).cuda(), err=err)

    append(0, 0, synth.kv_rows(seed, 0, 0, L), synth.idx_k_rows(seed, 0, 0, L))
    csa2.kv_pages_fork([cache], refs, lens, i32([0, 0]), i32([1, 2]), ws, err=err)
    for b in (1, 2):  # six more tokens each, into their own copies of the last page
        append(b, L, synth.kv_rows(seed, b, L, 6), synth.idx_k_rows(seed, b, L, 6))
    lens += i32([0, 6, 6])
    csa2.kv_pages_free(cache, refs, lens, i32([0]), err=err)
    d = csa2.default_desc(csa2.FULL, 1)
    q = queries(3)
    dws = torch.empty(csa2.dense_attn_workspace_bytes(d, 3), dtype=torch.uint8, device="cuda")

    def attend():
        out, lse = torch.empty((3, 16, 128), device="cuda"), torch.empty((3, 16), device="cuda")
        csa2.dense_attn_decode(d, cache, q.cuda(), lens, out, lse, 160, dws, err=err)
        return out, lse

    before = attend()
    import oracle
    oracle.build()
    assert int(err.item()) == 0
    for b in (1, 2):
        kv = np.concatenate([synth.kv_rows(seed, 0, 0, L), synth.kv_rows(seed, b, L, 6)])
        from _dense_util import E2M1
        codes, scales = (torch.from_numpy(np.ascontiguousarray(x)) for x in oracle.quant_rows(kv))
        x = torch.stack([E2M1[(codes & 15).int()], E2M1[(codes >> 4).int()]], 2).view(-1, 256)
        rows = x * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
        check(before[0][b:b + 1], before[1][b:b + 1], reference(q[b:b + 1], rows, [L + 6]), f"hypothesis {b}")
    m, n = i32([0] * 32), i32([0])
    csa2.kv_pages_compact([cache], refs, m, n, ws, err=err)
    after = attend()
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and int(n) == 8 and int(cache.page_table.max()) == 7
    assert all(torch.equal(x, y) for x, y in zip(before, after))
