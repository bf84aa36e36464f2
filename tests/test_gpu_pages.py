"""Pages of a cache on the GPU against the oracle's bookkeeping, whole numbers and
bytes equal, and the operators of the compressed cache run together."""
import random

import pytest
import torch

from oracle import kv8_oracle as O

pytestmark = pytest.mark.gpu


def lib():
    import block_diffusion_speculative_flush_gb300 as D
    return D


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """Rows of random lengths over a pool, some of them sharing their first pages."""

    def __init__(self, n_pages, page, lens, width, seed=0, shared=0.0):
        rng = random.Random(seed)
        free = list(range(n_pages))
        rng.shuffle(free)
        self.page, self.width, self.n_pages, self.lens = page, width, n_pages, list(lens)
        self.refs, self.table = [0] * n_pages, []
        for i, n in enumerate(lens):
            k = O.n_pages_of(n, page)
            row = []
            if i and rng.random() < shared:
                other = self.table[rng.randrange(i)]
                row = [p for p in other if p >= 0][:k]
            row += [free.pop() for _ in range(k - len(row))]
            for p in row:
                self.refs[p] += 1
            self.table.append(row + [-1] * (width - k))

    def cuda(self):
        return i32(self.refs), i32(self.table), i32(self.lens)


def buffers_of(n_pages, shapes, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, (n_pages, *s), generator=g, dtype=torch.uint8).cuda() for s in shapes]


SHAPES = [(16, 2, 64), (4,), (20,), (4100,), (16, 1, 128), (8192,)]


@pytest.mark.parametrize("n_buffers", [1, 6, 300])
@pytest.mark.parametrize("count", [0, 1, 37])
def test_copy(n_buffers, count):
    D = lib()
    n = 80
    shapes = [SHAPES[i % len(SHAPES)] if n_buffers <= 6 else SHAPES[i % 3] for i in range(n_buffers)]
    bufs = buffers_of(n, shapes)
    before = [b.cpu() for b in bufs]
    ids = random.Random(count).sample(range(n), 2 * count)
    src, dst = ids[:count], ids[count:]
    status = i32([0])
    D.dflash_pages_copy(D.dflash_page_buffers(bufs), i32(src), i32(dst), status=status)
    D.dflash_status_check(status)
    for b, x in zip(bufs, before):
        x[dst] = x[src]
        assert torch.equal(b.cpu(), x)


def test_copy_between_strided_pages_and_bad_ids():
    """K and V of a page side by side in one tensor: two buffers whose pages are apart."""
    D = lib()
    kv = torch.randint(0, 256, (30, 2, 16, 1, 64), dtype=torch.uint8, device="cuda")
    want = kv.cpu()
    status = i32([0])
    D.dflash_pages_copy(D.dflash_page_buffers([kv[:, 0]]), i32([3, -1, 5, 30]), i32([7, 8, 99, 9]), status=status)
    want[7, 0] = want[3, 0]
    assert torch.equal(kv.cpu(), want)
    with pytest.raises(D.DFlashError, match="page id"):
        D.dflash_status_check(status)


@pytest.mark.parametrize("seed", range(6))
def test_reorder(seed):
    D = lib()
    rng = random.Random(seed)
    n, page = [1, 2, 9, 40, 300, 3][seed], [16, 8, 32, 16, 64, 1024][seed]
    lens = [rng.choice([0, 1, page, page + 1, rng.randrange(1, 9 * page)]) for _ in range(n)]
    P = Pool(12 * n + 5, page, lens, 11, seed, shared=0.5)
    out = rng.randrange(1, 2 * n + 2)
    parents = [rng.randrange(-1, n) for _ in range(out)]
    refs, table, ln = P.cuda()
    nt, nl, status = torch.full((out, 13), 99, dtype=torch.int32, device="cuda"), i32([5] * out), i32([0])
    D.dflash_pages_reorder(refs, table, ln, i32(parents), nt, nl, page_size=page, status=status)
    D.dflash_status_check(status)
    r, t, l = O.reorder(P.refs, P.table, P.lens, parents, page, 13)
    assert refs.tolist() == r and nt.tolist() == t and nl.tolist() == l
    assert table.tolist() == P.table and ln.tolist() == P.lens


def test_reorder_of_bad_rows():
    D = lib()
    P = Pool(20, 16, [20, 40], 4)
    for parents, lens, what in (([0, 2], [20, 40], "bounds"), ([-2, 1], [20, 40], "bounds"), ([0, 1], [20, 65], "bounds"),
                                ([0, 1], [-1, 40], "bounds")):
        refs, table, _ = P.cuda()
        nt, nl, status = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), i32([7, 7]), i32([0])
        D.dflash_pages_reorder(refs, table, i32(lens), i32(parents), nt, nl, page_size=16, status=status)
        with pytest.raises(D.DFlashError, match=what):
            D.dflash_status_check(status)
        ok = [parents[i] == i and 0 <= lens[i] <= 64 for i in range(2)]
        for i in range(2):
            assert nt[i].tolist() == (P.table[i] if ok[i] else [-1] * 4)
            assert nl[i].item() == (lens[i] if ok[i] else 0)
    refs, table, ln = P.cuda()
    table[1, 1] = 20                                        # a page that the pool does not have
    nt, nl, status = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), i32([7]), i32([0])
    D.dflash_pages_reorder(refs, table, ln, i32([1]), nt, nl, page_size=16, status=status)
    with pytest.raises(D.DFlashError, match="page id"):
        D.dflash_status_check(status)
    assert nt[0, 1].item() == -1


@pytest.mark.parametrize("seed", range(12))
def test_resize(seed):
    D = lib()
    rng = random.Random(seed)
    n = [1, 2, 5, 30, 200, 9000, 4, 4, 64, 1, 33, 12][seed]
    page, width = [16, 8, 32, 16, 64, 8, 16, 1024, 16, 256, 8, 16][seed], 9
    pick = lambda: rng.choice([0, 1, page - 1, page, rng.randrange(1, 5 * page), rng.randrange(1, 9 * page)])
    lens = [pick() for _ in range(n)]
    spare = rng.choice([0, 3, n, 12 * n])                   # too few pages for some
    P = Pool(sum(O.n_pages_of(x, page) for x in lens) + spare + 1, page, lens, width, seed, shared=0.0)
    if seed % 2:                                            # forks: rows that share all their pages
        parents = [rng.randrange(n) for _ in range(n)]
        P.refs, P.table, P.lens = O.reorder(P.refs, P.table, P.lens, parents, page, width)
    want = [rng.choice([x, pick(), min(x + rng.randrange(1, 2 * page), width * page)]) for x in P.lens]
    bufs = buffers_of(P.n_pages, [(8,), (page, 16)], seed)
    data = [b.cpu() for b in bufs]
    refs, table, ln = P.cuda()
    free, status = i32([-5]), i32([0])
    D.dflash_pages_resize(refs, table, ln, i32(want), D.dflash_page_buffers(bufs), page_size=page, free_pages=free,
                          status=status)
    r, t, l, copies, refused = O.resize(P.refs, P.table, P.lens, want, page)
    assert refs.tolist() == r and ln.tolist() == l and table.tolist() == t
    assert free.item() == sum(c <= 0 for c in r)
    for b, x in zip(bufs, data):
        for s, d in copies:
            x[d] = x[s]
        assert torch.equal(b.cpu(), x)
    if refused:
        with pytest.raises(D.DFlashError, match="free page"):
            D.dflash_status_check(status)
    else:
        D.dflash_status_check(status)


def test_resize_of_bad_rows():
    D = lib()
    P = Pool(30, 16, [20, 40, 10], 4)
    refs, table, ln = P.cuda()
    status = i32([0])
    D.dflash_pages_resize(refs, table, ln, i32([65, -1, 17]), None, page_size=16, status=status)
    with pytest.raises(D.DFlashError, match="bounds"):
        D.dflash_status_check(status)
    r, t, l, _, _ = O.resize(P.refs, P.table, P.lens, [20, 40, 17], 16)
    assert refs.tolist() == r and table.tolist() == t and ln.tolist() == l


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_compact(seed, in_place):
    D = lib()
    rng = random.Random(seed)
    n, page = [1, 3, 20, 100, 2, 400][seed], [16, 8, 32, 16, 1024, 64][seed]
    lens = [rng.randrange(0, 9 * page) for _ in range(n)]
    P = Pool([40, 27, 1000, 1500, 18, 9000][seed], page, lens, 9, seed, shared=0.3)
    bufs = buffers_of(P.n_pages, [(32,), (page, 16), (4,)], seed)
    data = [b.cpu() for b in bufs]
    refs, table, ln = P.cuda()
    nr, nt = (refs, table) if in_place else (torch.full_like(refs, 9), torch.full_like(table, 9))
    used, status = i32([-1]), i32([0])
    D.dflash_pages_compact(refs, table, ln, nr, nt, D.dflash_page_buffers(bufs), page_size=page, used=used, status=status)
    D.dflash_status_check(status)
    r, t, u, moves = O.compact(P.refs, P.table, P.lens, page)
    assert nr.tolist() == r and nt.tolist() == t and used.item() == u and ln.tolist() == P.lens
    for b, x in zip(bufs, data):
        for s, d in moves:
            x[d] = x[s]
        assert torch.equal(b.cpu(), x)


def test_compact_of_a_table_that_names_free_pages():
    D = lib()
    P = Pool(30, 16, [60, 40], 4, seed=3)
    refs, table, ln = P.cuda()
    free = [p for p in range(30) if P.refs[p] == 0 and p >= 7][0]
    table[0, 0], table[1, 0] = free, 31
    used, status = i32([0]), i32([0])
    D.dflash_pages_compact(refs, table, ln, refs, table, None, page_size=16, used=used, status=status)
    assert table[0, 0].item() == -1 and table[1, 0].item() == -1
    with pytest.raises(D.DFlashError, match="page id"):
        D.dflash_status_check(status)


def test_a_captured_step_of_the_whole_cache():
    """Rotary positions, append into 8-bit pages and attention of two layers, pages forked and grown in
    front of them: the captured step replayed, against the same calls one by one and the oracle."""
    D = lib()
    layers, hq, hkv, d, page, n_pages, width = 2, 4, 2, 64, 16, 64, 12
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()
    table = D.dflash_rope_table(d, 10000.0)

    def fresh():
        s = dict(refs=torch.zeros(n_pages, dtype=torch.int32, device="cuda"))
        for name, rows in (("a", 1), ("b", 3)):
            s["t" + name] = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
            s["l" + name] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["pages"] = [[torch.zeros((n_pages, page, hkv, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                       for _ in range(2)] + [torch.zeros((n_pages, hkv), device="cuda") for _ in range(2)] for _ in range(layers)]
        s["buffers"] = D.dflash_page_buffers([x for p in s["pages"] for x in p])
        s["out"] = [torch.zeros((6, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        return s

    prompt = [[rnd(39, h, d) for h in (hq, hkv, hkv)] for _ in range(layers)]
    step = [[rnd(6, h, d) for h in (hq, hkv, hkv)] for _ in range(layers)]
    parents, want, st = i32([0, 0, 0]), i32([41, 41, 41]), i32([0, 2, 4, 6])

    def read_prompt(s):
        D.dflash_pages_resize(s["refs"], s["ta"], s["la"], i32([39]), s["buffers"], page_size=page)
        for (q, k, v), P in zip(prompt, s["pages"]):
            k2 = k.clone()
            D.dflash_rope(table, None, k2, i32([0, 39]), s["la"])
            D.dflash_kv8_append(k2, v, *P, i32([0, 39]), s["la"], s["ta"])

    def one_step(s, work):
        D.dflash_pages_reorder(s["refs"], s["ta"], s["la"], parents, s["tb"], s["lb"], page_size=page)
        D.dflash_pages_resize(s["refs"], s["tb"], s["lb"], want, s["buffers"], page_size=page, workspace=s.get("ws"))
        for (q, k, v), P, o, (q2, k2) in zip(step, s["pages"], s["out"], work):
            D.dflash_rope(table, q, k, st, s["lb"], q2, k2)
            D.dflash_kv8_append(k2, v, *P, st, s["lb"], s["tb"])
            D.dflash_kv8_attention(q2, *P, st, s["lb"], s["tb"], o, max_rows=2, max_len=64)

    work = [(torch.empty_like(q), torch.empty_like(k)) for q, k, v in step]
    a, b = fresh(), fresh()
    read_prompt(a)
    one_step(a, work)
    read_prompt(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_step(b, work)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a["out"], b["out"]):
        assert torch.equal(x, y)
    assert torch.equal(a["refs"], b["refs"]) and torch.equal(a["tb"], b["tb"]) and a["lb"].tolist() == [41] * 3
    assert len(set(a["tb"][:, 2].tolist())) == 3 and len(set(a["tb"][:, 1].tolist())) == 1   # the begun page is each one's own
    # the oracle, on the rotated rows that the calls made (theirs are tested beside the rotation): the prompt's and
    # the step's codes of each row in turn
    for layer in range(layers):
        k0 = prompt[layer][1].clone()
        D.dflash_rope(table, None, k0, i32([0, 39]), i32([39]))
        kp, ks = torch.zeros((3, page, hkv, d), dtype=torch.uint8), torch.zeros((3, hkv))
        vp, vs = kp.clone(), ks.clone()
        tb = torch.arange(3, dtype=torch.int32)[None]
        kp, ks = O.append8(kp, ks, k0.cpu(), [0, 39], [39], tb)
        vp, vs = O.append8(vp, vs, prompt[layer][2].cpu(), [0, 39], [39], tb)
        for row in range(3):
            sl = slice(2 * row, 2 * row + 2)
            k2, s2 = O.append8(kp, ks, work[layer][1][sl].cpu(), [0, 2], [41], tb)
            v2, t2 = O.append8(vp, vs, step[layer][2][sl].cpu(), [0, 2], [41], tb)
            o, _, tol, _ = O.attention8(work[layer][0][sl].cpu(), O.gather8(k2, s2, [41], tb), O.gather8(v2, t2, [41], tb),
                                        [0, 2], [41], True, 0, d ** -0.5, True, True)
            err = (a["out"][layer][sl].double().cpu() - o).abs()
            assert bool((err <= tol).all()), float((err - tol).max())


def grown(refs, table, lens, want, page, bufs=None):
    """dflash_pages_resize of lists: refs, table and lens afterwards, the free pages and the status word."""
    D = lib()
    r, t, l, free, status = i32(refs), i32(table), i32(lens), i32([-1]), i32([0])
    D.dflash_pages_resize(r, t, l, i32(want), None if bufs is None else D.dflash_page_buffers(bufs), page_size=page,
                          free_pages=free, status=status)
    return r.tolist(), t.tolist(), l.tolist(), free.item(), status.item()


SHARED = [  # refs, table, lens, want: rows that write to begun pages of one another in a pool without pages for all
    ([2, 2], [[0, 1], [0, 1]], [18, 20], [21, 22]),
    ([2, 2], [[0, 1], [0, 1]], [20, 18], [21, 22]),
    ([3, 3, 0], [[0, 1], [0, 1], [0, 1]], [18, 20, 19], [21, 22, 23]),
    ([3, 3, 0, 0], [[0, 1], [0, 1], [0, 1]], [18, 20, 19], [21, 22, 23]),
    ([3, 3, 0, 0], [[0, 1, -1], [0, 1, -1], [0, 1, -1]], [18, 20, 19], [40, 22, 23]),
    ([2, 2, 1, 0], [[0, 1, -1], [2, -1, -1], [0, 1, -1]], [18, 16, 20], [21, 48, 22]),
    ([2, 2, 2, 2, 0], [[0, 1, -1], [0, 1, -1], [2, 3, -1], [2, 3, -1]], [18, 20, 18, 20], [21, 22, 21, 22]),
    ([2, 2, 0, 0, 0], [[0, 1, -1, -1], [0, 1, -1, -1]], [18, 20], [50, 60]),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
@pytest.mark.parametrize("clusters", [False, True])
def test_nobody_writes_to_a_page_that_a_refused_row_still_holds(case, clusters):
    refs, table, lens, want = SHARED[case]
    n_pages, rows = len(refs), len(lens)
    if clusters:   # the form of large pools: rows of nothing behind these
        table = table + [[-1] * len(table[0])] * 1100
        lens, want = lens + [0] * 1100, want + [0] * 1100
    r, t, l, free, status = grown(refs, table, lens, want, 16)
    er, et, el, copies, refused = O.resize(refs, table, lens, want, 16)
    assert (r, t, l) == (er, et, el) and free == sum(c <= 0 for c in er) and status == (16 if refused else 0)
    for i in range(rows):
        if l[i] == want[i] and want[i] > lens[i] and lens[i] % 16:
            assert r[t[i][(lens[i] - 1) // 16]] == 1, (i, r, t)
        if l[i] != want[i]:
            assert t[i] == table[i] and l[i] == lens[i]


@pytest.mark.parametrize("seed", range(8))
def test_forks_that_grow_in_a_pool_without_room(seed):
    """Rows forked, some of them cut back within the shared page, all grown with any number of pages left."""
    rng = random.Random(100 + seed)
    n, page, width = [3, 8, 40, 500, 9000, 5, 17, 300][seed], [16, 8, 16, 8, 8, 64, 16, 16][seed], 6
    heads = max(1, n // 4)
    lens = [rng.randrange(1, 3 * page) for _ in range(heads)]
    P = Pool(sum(O.n_pages_of(x, page) for x in lens) + 1 + rng.randrange(0, n), page, lens, width, seed)
    P.refs, P.table, P.lens = O.reorder(P.refs, P.table, P.lens, [rng.randrange(heads) for _ in range(n)], page, width)
    back = [x - rng.randrange(0, (x - 1) % page + 1) if x else 0 for x in P.lens]      # within the last page
    P.refs, P.table, P.lens, _, _ = O.resize(P.refs, P.table, P.lens, back, page)
    want = [rng.choice([x, x + 1, x + rng.randrange(0, page)]) for x in P.lens]
    r, t, l, free, status = grown(P.refs, P.table, P.lens, want, page)
    er, et, el, copies, refused = O.resize(P.refs, P.table, P.lens, want, page)
    assert r == er and t == et and l == el and free == sum(c <= 0 for c in er)
    assert status == (16 if refused else 0)
    for i in range(n):
        if l[i] > P.lens[i] and P.lens[i] % page:
            assert r[t[i][(P.lens[i] - 1) // page]] == 1


def test_pages_asked_for_beyond_two_to_the_32():
    """Rows ask for 2^32 pages together in front of a last one that asks for one: it does not get what the first has."""
    D = lib()
    rows, width, page, n_pages = 4098, 1 << 20, 8, 64
    table = torch.empty((rows, width), dtype=torch.int32, device="cuda")       # (16 GiB, looked at in a few places)
    table[0, :2], table[rows - 1, :2] = -1, -1
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    want = torch.full((rows,), width * page, dtype=torch.int32, device="cuda")
    want[0], want[1], want[rows - 1] = page, (width - 1) * page, page
    assert int(((want.long() + page - 1) // page)[:-1].sum()) == 1 << 32
    refs, free, status = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), i32([-1]), i32([0])
    D.dflash_pages_resize(refs, table, lens, want, None, page_size=page, free_pages=free, status=status)
    with pytest.raises(D.DFlashError, match="free page"):
        D.dflash_status_check(status)
    assert table[0, 0].item() == 0 and table[rows - 1, 0].item() == -1
    assert lens[0].item() == page and int(lens[1:].abs().sum()) == 0
    assert refs.tolist() == [1] + [0] * (n_pages - 1) and free.item() == n_pages - 1
