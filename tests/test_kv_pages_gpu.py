"""Fork, trim and compact of the cache's pages on the GPU against the oracle: whole numbers
and bytes, which have to be equal."""
import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import kv_cache as okv
from oracle import kv_pages as opg
from rmsnorm_fp4_quant_gb300 import build as fbuild
from test_kv_masks_gpu import tolerances

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


def random_cache(pages, heads, page, D, seed):
    g = np.random.default_rng(seed)
    r = lambda *s: g.integers(0, 256, (pages, heads, *s), dtype=np.uint8)     # noqa: E731
    return [r(page, D // 2), r(page, D // 16), r(page, D // 2), r(D // 16, page)]


def scene(B, longest, page, seed, spare=8, most=None, bad=True):
    """Tables of B sequences in a pool: some share their first pages, some pages are held from
    outside, some entries hold none."""
    g = np.random.default_rng(seed)
    lens = g.integers(0, longest + 1, B)
    lens[g.integers(0, B)] = longest
    if B > 2:
        lens[1] = longest // page * page                       # ends with its page
    most = -(-longest // page) + 2 if most is None else most
    used = [-(-int(n) // page) for n in lens]
    pages = sum(used) + spare
    order = list(g.permutation(pages))
    refs = np.zeros(pages, np.int64)
    tables = np.full((B, most), -3, np.int64)
    for b in range(B):
        for i in range(used[b]):
            if b and i < used[b - 1] - 1 and i < used[b] - 1 and g.random() < 0.4:
                tables[b, i] = tables[b - 1, i]                # a page of the sequence before it
            else:
                tables[b, i] = order.pop()
            if tables[b, i] >= 0:
                refs[tables[b, i]] += 1
    for p in range(pages):
        if refs[p] and g.random() < 0.1:
            refs[p] += 1                                       # held from outside
    for _ in range(2):
        if order and len(order) > spare:
            refs[order.pop()] = 1
    if bad and longest > 3 * page:
        b = int(np.argmax(lens))
        if refs[tables[b, 0]] == 1:
            refs[tables[b, 0]] = 0
            tables[b, 0] = -1                                  # given up
    return refs, tables, lens, g


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def same(name, got, want):
    assert np.array_equal(got.cpu().numpy(), want), name


def check_fork(heads, D, page, refs, tables, lens, parents, new, new_lens=None, seed=0, repeat=True, **kw):
    cache = random_cache(len(refs), heads, page, D, seed)
    want = opg.fork(cache, refs, tables, lens, np.arange(len(lens)) if parents is None else parents, new, new_lens)
    c = [torch.from_numpy(x).cuda() for x in cache]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (c, dev(refs), dev(tables), dev(lens), None if parents is None else dev(parents))
    for _ in range(2 if repeat else 1):                        # the second call does the same again
        got = fq.kv_fork_nvfp4(*args, new_tokens=new, new_lens=None if new_lens is None else dev(new_lens),
                               status=status, **kw)
        torch.cuda.synchronize()
        for name, a, b in zip(("tables", "lens", "refs", "slots"), got, want):
            same(name, a, b)
        for a, b in zip(c, want[4]):
            same("cache", a, b)
        assert fq.read_device_status(status) == (fq.FP4_ERR_NO_PAGES if want[5] else fq.FP4_OK)
    return got


FORKS = [
    # B, longest, page, N, new tokens, heads, D, spare pages
    (1, 1, 16, 1, 1, 1, 64, 4),
    (1, 0, 16, 3, 1, 2, 128, 4),
    (1, 1003, 16, 4, 1, 2, 128, 9),
    (4, 64, 16, 4, 1, 3, 64, 12),
    (5, 63, 32, 9, 0, 2, 64, 3),
    (3, 100, 48, 40, 1, 1, 128, 50),
    (7, 333, 64, 7, 5, 2, 64, 20),
    (2, 129, 128, 5, 300, 1, 64, 40),
    (33, 700, 16, 33, 1, 1, 64, 60),
    (64, 1500, 16, 64, 2, 1, 64, 200),
    (130, 900, 32, 257, 1, 1, 64, 400),
    (6, 40000, 16, 17, 1, 1, 64, 30),
    (3, 50, 16, 1100, 1, 1, 64, 1200),
    (5, 40, 16, 3000, 1, 1, 64, 3100),                          # more children than shared memory keeps,
    (2200, 30, 16, 2200, 1, 1, 64, 2300),                       # and more sequences
]


@pytest.mark.parametrize("B,longest,page,N,new,heads,D,spare", FORKS)
def test_fork(B, longest, page, N, new, heads, D, spare):
    refs, tables, lens, g = scene(B, longest, page, seed=B + N, spare=spare,
                                  most=-(-(longest + new) // page) + 1)
    parents = g.integers(-1, B, N)
    check_fork(heads, D, page, refs, tables, lens, parents, new, seed=N)


def test_fork_into_itself():
    """parents None: one more token of every sequence; only pages that are shared are copied."""
    refs, tables, lens, g = scene(9, 150, 16, seed=3, spare=12)
    check_fork(2, 64, 16, refs, tables, lens, None, 1)
    check_fork(2, 64, 16, refs, tables, lens, None, 33, new_lens=g.integers(-2, 40, 9))


def test_parents_outside_and_lengths_beyond_the_table():
    refs, tables, lens, _ = scene(4, 200, 16, seed=4, spare=30)
    lens[0], lens[2] = 10 ** 9, -5
    check_fork(1, 64, 16, refs, tables, lens, [3, -1, 4, 2 ** 31 - 1, -2 ** 31, 0, 2, 3], 1)


def test_pages_run_out_in_the_childrens_order():
    for spare in (0, 1, 2, 5):
        refs, tables, lens, _ = scene(3, 70, 16, seed=5, spare=spare, bad=False)
        lens = np.array([70, 64, 33])
        got = check_fork(1, 64, 16, refs, tables, lens, [0, 0, 1, 1, 2, 2, 0], 1)
        del got
    # and where a table's entries do
    refs, tables, lens, _ = scene(2, 64, 16, seed=6, spare=9, most=4, bad=False)
    check_fork(1, 64, 16, refs, tables, np.array([64, 60]), [0, 1, 1], 6)


def test_a_last_page_held_elsewhere_is_copied_for_every_child():
    tables, lens = np.array([[2, 5, -1]]), np.array([20])
    refs = np.zeros(9, np.int64)
    refs[2], refs[5] = 1, 2                                     # page 5: somebody else's too
    got = check_fork(1, 64, 16, refs, tables, lens, [0, 0], 1)
    assert got[0].tolist() == [[2, 0, -1], [2, 1, -1]] and got[2].tolist()[5] == 1
    # two old sequences that share a last page: it stays with the first child of either
    got = check_fork(1, 64, 16, refs, np.array([[2, 5, -1], [2, 5, -1]]), np.array([20, 20]), [1, 0], 1)
    assert got[0].tolist() == [[2, 5, -1], [2, 0, -1]]
    # without new tokens nothing is about to be written, and nothing copied
    got = check_fork(1, 64, 16, refs, tables, lens, [0, 0], 0)
    assert got[0].tolist() == [[2, 5, -1]] * 2 and got[2].tolist()[5] == 3


def test_everything_ends():
    refs, tables, lens, _ = scene(5, 100, 16, seed=7)
    check_fork(1, 64, 16, refs, tables, lens, [], 1)
    check_fork(1, 64, 16, refs, tables, lens, [-1, -1], 1)


def test_nothing_to_do():
    """No sequences, no children, no room in a table."""
    z = lambda *s: np.zeros(s, np.int64)                                     # noqa: E731
    check_fork(1, 64, 16, z(5), z(0, 3), z(0), [-1, 0], 1)
    check_fork(1, 64, 16, z(5), z(2, 0), z(2), [1, 0], 2)
    check_fork(1, 64, 16, z(5), z(0, 3), z(0), None, 1)
    check_fork(1, 64, 16, np.array([0, 1, 0]), np.array([[1]]), np.array([16]), [0], 0)
    for refs, tables, lens in ((z(4), z(0, 3), z(0)), (np.array([0, 2, 0]), z(1, 0), z(1))):
        cache = [torch.from_numpy(x).cuda() for x in random_cache(len(refs), 1, 16, 64, 1)]
        got = fq.kv_trim_nvfp4(cache, dev(refs), dev(tables), dev(lens))
        for a, b in zip(got, opg.trim(16, refs, tables, lens)):
            same("trim", a, b)
        want = opg.compact([x.cpu().numpy() for x in cache], refs, tables, lens)
        got = fq.kv_compact_nvfp4(cache, dev(refs), dev(tables), dev(lens))
        for a, b in zip(got[:3], want):
            same("compact", a, b)
        assert got[3].item() == want[3]


def test_many_pages():
    """Pages enough for every size of the plan, free ones at the end of the pool."""
    for pages in (3000, 40000, 300000):
        refs = np.ones(pages, np.int64)
        refs[pages - 5:] = 0
        tables = np.arange(200).reshape(2, 100)
        got = check_fork(1, 64, 16, refs, tables, np.array([1599, 1585]), [0, 0, 1, 1, 1], 1, repeat=False)
        assert got[0][1, 99].item() == pages - 5


TRIMS = [(1, 1, 16), (4, 200, 16), (9, 333, 48), (40, 1000, 64), (300, 700, 16), (2, 60000, 16)]


@pytest.mark.parametrize("B,longest,page", TRIMS)
def test_trim(B, longest, page):
    refs, tables, lens, g = scene(B, longest, page, seed=B)
    cache = [torch.from_numpy(x).cuda() for x in random_cache(len(refs), 1, page, 64, 1)]
    first, end = g.integers(-3, longest + 3, B), g.integers(-3, longest + 3, B)
    end[:: 3] = 0
    for f, e in ((first, end), (None, end), (first, None), (None, None)):
        want = opg.trim(page, refs, tables, lens, f, e)
        got = fq.kv_trim_nvfp4(cache, dev(refs), dev(tables), dev(lens), None if f is None else dev(f),
                               None if e is None else dev(e))
        for name, a, b in zip(("tables", "lens", "refs"), got, want):
            same(name, a, b)


@pytest.mark.parametrize("B,longest,page,heads,D", [(1, 1, 16, 1, 64), (5, 200, 16, 3, 128), (12, 700, 48, 2, 64),
                                                    (90, 1500, 64, 1, 128), (300, 900, 16, 1, 64)])
@pytest.mark.parametrize("share", [0.0, 0.5, 1.0])
def test_compact(B, longest, page, heads, D, share):
    refs, tables, lens, g = scene(B, longest, page, seed=B)
    cache = random_cache(len(refs), heads, page, D, 2)
    ended = g.random(B) < share
    tables, lens, refs = opg.trim(page, refs, tables, lens, None, np.where(ended, 0, lens))
    want = opg.compact(cache, refs, tables, lens)
    c = [torch.from_numpy(x).cuda() for x in cache]
    for _ in range(2):
        got = fq.kv_compact_nvfp4(c, dev(refs), dev(tables), dev(lens))
        same("tables", got[0], want[0])
        same("refs", got[1], want[1])
        same("map", got[2], want[2])
        assert got[3].item() == want[3]
        for a, b in zip(c, want[4]):
            same("cache", a, b)


def test_compacting_a_large_pool():
    g = np.random.default_rng(1)
    pages = 50000
    refs = (g.random(pages) < 0.3).astype(np.int64) * g.integers(1, 5, pages)
    cache = random_cache(pages, 1, 16, 64, 3)
    live = np.flatnonzero(refs)
    tables = live[:4000].reshape(40, 100)
    want = opg.compact(cache, refs, tables, [1600] * 40)
    c = [torch.from_numpy(x).cuda() for x in cache]
    got = fq.kv_compact_nvfp4(c, dev(refs), dev(tables), dev([1600] * 40))
    for name, a, b in zip(("tables", "refs", "map"), got, want):
        same(name, a, b)
    for a, b in zip(c, want[4]):
        same("cache", a, b)


def test_pages_beyond_32_bit_offsets():
    """Page copies that lie behind 2^32 bytes of a buffer."""
    heads, page, D = 64, 128, 128
    pages = (1 << 32) // (heads * page * D // 2) + 40          # 8232 pages of 512 KiB
    c = fq.kv_cache_nvfp4(pages, page, heads, D)
    for t in c:
        t[pages - 3].random_(0, 256)
    src = [t[pages - 3].clone() for t in c]
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[pages - 1] = refs[pages - 2] = 0
    got = fq.kv_fork_nvfp4(c, refs, torch.full((1, 2), pages - 3, dtype=torch.int32, device="cuda"),
                           dev([100]), dev([0, 0]))
    assert got[0][:, 0].tolist() == [pages - 3, pages - 2] and got[3].tolist() == [[(pages - 3) * page + 100],
                                                                                 [(pages - 2) * page + 100]]
    for i, t in enumerate(c):                                   # 112 tokens of the page
        a, b = (t[pages - 2], src[i]) if i < 3 else (t[pages - 2].transpose(-1, -2), src[i].transpose(-1, -2))
        assert torch.equal(a[:, :112], b[:, :112]) and not torch.any(a[:, 112:])
    refs.zero_()
    refs[pages - 3] = 1
    got = fq.kv_compact_nvfp4(c, refs, torch.full((1, 1), pages - 3, dtype=torch.int32, device="cuda"), dev([100]))
    assert got[3].item() == 1 and got[0].item() == 0
    for t, s in zip(c, src):
        assert torch.equal(t[0], s)


def test_a_window_moves_on():
    """Pages behind a window are given up, taken by others, and attention does not miss them."""
    page, D, window = 16, 64, 40
    g = torch.Generator().manual_seed(1)
    cache = fq.kv_cache_nvfp4(12, page, 1, D)
    refs = torch.zeros(12, dtype=torch.int32, device="cuda")
    tables = torch.full((2, 16), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    kept = [[], []]
    q = torch.randn(2, 4, D, generator=g).bfloat16()
    for step in range(9):
        tables, lens, refs, slots = fq.kv_fork_nvfp4(cache, refs, tables, lens, new_tokens=13)
        k, v = (torch.randn(26, 1, D, generator=g).bfloat16() for _ in range(2))
        fq.kv_append_nvfp4(cache, k.cuda(), v.cuda(), slots.flatten())
        assert torch.all(slots >= 0)
        for b in range(2):
            kept[b] += [(k[13 * b + i], v[13 * b + i]) for i in range(13)]
        out = fq.attention_nvfp4(q.cuda(), cache, tables, lens, window=window)
        # the same over a cache that holds the window's tokens alone
        n = min(window, 13 * (step + 1))
        ref = [np.zeros(s, np.uint8) for s in ((6, 1, page, D // 2), (6, 1, page, D // 16), (6, 1, page, D // 2), (6, 1, D // 16, page))]
        for b in range(2):
            kk, vv = (torch.stack([t[j] for t in kept[b][-n:]]).float().numpy() for j in range(2))
            okv.append(ref, kk, vv, np.arange(n) + 48 * b)
        want = okv.attention(q.double().numpy(), ref, np.arange(6).reshape(2, 3), [n, n], sm_scale=D ** -0.5)
        err = np.abs(out.double().cpu().numpy() - want.out)
        assert np.all(err <= tolerances(want, D, "bf16", 0.0)[0])
        tables, lens, refs = fq.kv_trim_nvfp4(cache, refs, tables, lens, first=(lens + 1 - window).int())
        assert int((refs > 0).sum()) == int((tables >= 0).sum()) <= 8


def test_a_captured_beam_search():
    """Selection, fork, append and attention as one captured step, back and forth between two sets
    of buffers, against the same steps of the oracles."""
    B, K, V, page, D, Hq, Hkv = 2, 3, 1500, 16, 64, 4, 2
    N, most, pages, prompt = B * K, 8, 60, 37
    g = torch.Generator().manual_seed(11)
    cache = fq.kv_cache_nvfp4(pages, page, Hkv, D)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    tables, lens, refs, slots = fq.kv_fork_nvfp4(cache, refs, torch.full((B, most), -1, dtype=torch.int32, device="cuda"),
                                                 dev([0] * B), new_tokens=prompt)
    k, v = (torch.randn(B * prompt, Hkv, D, generator=g).bfloat16() for _ in range(2))
    fq.kv_append_nvfp4(cache, k.cuda(), v.cuda(), slots.flatten())
    tables, lens, refs, _ = fq.kv_fork_nvfp4(cache, refs, tables, lens, dev(np.repeat(np.arange(B), K)), new_tokens=0)
    host = [t.cpu().numpy().copy() for t in cache]
    h_refs, h_tables, h_lens = (t.cpu().numpy().astype(np.int64) for t in (refs, tables, lens))
    h_scores = np.full((B, K), -np.inf)
    h_scores[:, 0] = 0.0
    h_done = np.zeros((B, K), bool)

    logits = torch.zeros(B, K, V, dtype=torch.bfloat16, device="cuda")
    qkv = [torch.zeros(N, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
    sets = []
    for s in range(2):
        e = lambda *shape, t=torch.int32: torch.zeros(*shape, dtype=t, device="cuda")    # noqa: E731
        sets.append(dict(tables=e(N, most), lens=e(N), refs=e(pages), slots=e(N, 1, t=torch.int64),
                         out=[e(B, K, t=torch.float32), e(B, K), e(B, K), e(B, K, t=torch.bool)],
                         att=e(N, Hq, D, t=torch.bfloat16)))
    sets[0]["tables"].copy_(tables), sets[0]["lens"].copy_(lens), sets[0]["refs"].copy_(refs)
    sets[0]["out"][0].copy_(torch.from_numpy(h_scores).float())

    def step(a, b):
        fq.beam_select(logits, a["out"][0], K, finished=a["out"][3], end_token=5, out=b["out"])
        fq.kv_fork_nvfp4(cache, a["refs"], a["tables"], a["lens"], b["out"][1].view(-1), out_tables=b["tables"],
                         out_seq_lens=b["lens"], out_refs=b["refs"], out_slots=b["slots"])
        fq.kv_append_nvfp4(cache, qkv[1], qkv[2], b["slots"].view(-1))
        fq.attention_nvfp4(qkv[0], cache, b["tables"], b["lens"], out=b["att"], softcap=20.0)
    graphs = []
    side = torch.cuda.Stream()
    for a, b in ((0, 1), (1, 0)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(sets[a], sets[b])
        graphs.append(graph)
    from oracle import beam as obeam
    for i in range(7):
        x = (torch.randn(B, K, V, generator=g) * 3).bfloat16()
        q, k, v = (torch.randn(N, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        logits.copy_(x)
        for t, src in zip(qkv, (q, k, v)):
            t.copy_(src)
        graphs[i & 1].replay()
        torch.cuda.synchronize()
        b = sets[(i + 1) & 1]
        want = obeam.select(x.double().numpy(), h_scores, K, h_done, 5)
        assert want[4].min() > 7e-5
        h_scores, h_done = b["out"][0].double().cpu().numpy(), want[3]
        same("parents", b["out"][1], want[1])
        same("tokens", b["out"][2], want[2])
        h_tables, h_lens, h_refs, h_slots, host, short = opg.fork(host, h_refs, h_tables, h_lens, want[1].reshape(-1), 1)
        assert not short
        okv.append(host, k.float().numpy(), v.float().numpy(), h_slots[:, 0])
        same("tables", b["tables"], h_tables)
        same("refs", b["refs"], h_refs)
        for a, c in zip(cache, host):
            same("cache", a, c)
        ref = okv.attention(q.double().numpy(), host, h_tables, h_lens, sm_scale=D ** -0.5, softcap=20.0)
        err = np.abs(b["att"].double().cpu().numpy() - ref.out)
        assert np.all(err <= tolerances(ref, D, "bf16", 20.0)[0])


def test_streams_and_workspaces():
    refs, tables, lens, g = scene(9, 400, 16, seed=9, spare=40)
    parents = g.integers(0, 9, 12)
    cache = [torch.from_numpy(x).cuda() for x in random_cache(len(refs), 2, 16, 64, 1)]
    args = (dev(refs), dev(tables), dev(lens), dev(parents))
    first = fq.kv_fork_nvfp4(cache, *args)
    size = fq.fp4_kv_pages_workspace_bytes(len(refs), 12)
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(workspace=ws), dict(workspace=ws, pdl=True), dict(stream=side)):
        again = fq.kv_fork_nvfp4(cache, *args, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    a = fq.kv_compact_nvfp4(cache, *args[:3])
    b = fq.kv_compact_nvfp4(cache, *args[:3], workspace=ws, pdl=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals():
    refs, tables, lens, _ = scene(3, 100, 16, seed=1)
    cache = [torch.from_numpy(x).cuda() for x in random_cache(len(refs), 1, 16, 64, 1)]
    r, t, l = dev(refs), dev(tables), dev(lens)
    p = dev([0, 1])
    for call in (lambda: fq.kv_fork_nvfp4(cache, r[1:], t, l, p), lambda: fq.kv_fork_nvfp4(cache, r, t[0], l, p),
                 lambda: fq.kv_fork_nvfp4(cache, r, t, l[:2], p), lambda: fq.kv_fork_nvfp4(cache, r, t, l, p.long()),
                 lambda: fq.kv_fork_nvfp4(cache, r, t, l, p[None]), lambda: fq.kv_fork_nvfp4(cache, r, t, l, p, new_tokens=-1),
                 lambda: fq.kv_fork_nvfp4(cache, r.cpu(), t, l, p), lambda: fq.kv_fork_nvfp4([c.cpu() for c in cache], r, t, l, p),
                 lambda: fq.kv_fork_nvfp4(cache, r, t, l, p, out_slots=torch.zeros(2, 2, dtype=torch.int64, device="cuda")),
                 lambda: fq.kv_fork_nvfp4(cache, r, t, l, p, new_lens=l), lambda: fq.kv_trim_nvfp4(cache, r, t, l, first=p),
                 lambda: fq.kv_trim_nvfp4(cache, r, t.t(), l), lambda: fq.kv_compact_nvfp4(cache, r, t, l, out_live=r)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fq.kv_fork_nvfp4(cache, r, t, l, out_tables=t), lambda: fq.kv_fork_nvfp4(cache, r, t, l, out_refs=r),
                 lambda: fq.kv_trim_nvfp4(cache, r, t, l, out_tables=t), lambda: fq.kv_compact_nvfp4(cache, r, t, l, out_map=r),
                 lambda: fq.kv_compact_nvfp4(cache, r, t, l, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fq.Fp4Error):
            call()


def test_debug_build_finds_no_access_out_of_bounds():
    fbuild.build(debug=True)
    L = fq.debug_lib()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, bad.data_ptr()) == 0
    try:
        with fq.using_library(L):
            for args in FORKS:
                test_fork(*args)
            test_fork_into_itself()
            test_parents_outside_and_lengths_beyond_the_table()
            test_pages_run_out_in_the_childrens_order()
            for args in TRIMS[:5]:
                test_trim(*args)
            test_compact(12, 700, 48, 2, 64, 0.5)
            test_compact(300, 900, 16, 1, 64, 0.5)
            assert bad.item() == 0
            refs, tables, lens, _ = scene(5, 100, 16, seed=7)
            c = [torch.from_numpy(x).cuda() for x in random_cache(len(refs), 1, 16, 64, 1)]
            calls = (lambda: fq.kv_fork_nvfp4(c, dev(refs), dev(tables), dev(lens)),
                     lambda: fq.kv_trim_nvfp4(c, dev(refs), dev(tables), dev(lens)),
                     lambda: fq.kv_compact_nvfp4(c, dev(refs), dev(tables), dev(lens)))
            for call in calls:
                assert L.fp4_debug_configure(2_000_000_000, 1, 0, -1, -1, bad.data_ptr()) == 0
                before = bad.item()
                call()
                torch.cuda.synchronize()
                assert bad.item() > before
    finally:
        L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, None)
