"""Attention over the NVFP4 cache with capped logits, distance biases, windows and prefixes,
against the oracle.

Tolerance (h = half a step of the output type, n = keys of the row, w = sum of p |v|,
L = largest sum of |scale q k|, b = sum of p |bias|, bw = sum of p |bias| |v|, V = largest |v|):
  * a product is off by at most D * 2^-23 * L, its factor and its rounding by 2^-22 * L more, and
    the cap's tanh does not make that larger; the cap's own steps (an exponential, 2^-22, a
    reciprocal of a product, 2^-23 and five roundings of 2^-24, times twice the cap, and the last
    sum) add 2^-20 * cap: e_s in all;
  * a bias, the start of its line (with the reference in it, which is a logit of the row; it begins
    anew for every 16 keys) and its value there are a few roundings of 2^-24 each of at most
    |bias| + 16 |slope| + |lse| + L + cap: 2^-20 of that for every key is more than these;
  * p is off by the factor exp of these, and so is the sum: 2 e_s w + 2^-20 (bw + b |out|) + ...;
  * each p is rounded to 11 bits for the product with v, and where it is 2^14 times smaller than
    the largest, to 2^-25 of that: 2^-11 w + n 2^-25 V;
  * the fp32 sums over n keys: n * 2^-23 * w, twice; the output's rounding: h * |out|.
lse: the same of its logits, n * 2^-23 and 2^-22 (|lse| + 1).
"""
import itertools

import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import kv_cache as okv
from rmsnorm_fp4_quant_gb300 import build as fbuild
from test_kv_cache_gpu import DT, HALF_STEP, fill_sequences, for_even_split, for_ranges, gen, queries, shape_of, times_for_items

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


def tolerances(ref, D, dtype, cap, slopes=None):
    """(out [rows, Hq, D], lse [rows, Hq]) of the oracle's rows."""
    r = ref.rows
    n = ref.keys[r][:, None]
    lse = np.where(n > 0, np.abs(np.where(np.isfinite(ref.lse[r]), ref.lse[r], 0.0)), 0.0)
    e_s = (D * 2.0 ** -23 + 2.0 ** -22) * ref.logit[r] + 2.0 ** -20 * cap + 2.0 ** -20 * (lse + ref.logit[r])
    if slopes is not None:
        e_s = e_s + 2.0 ** -20 * 16 * np.abs(slopes.numpy())
    e_b = 2.0 ** -20 * ref.bias[r]
    out = np.abs(ref.out[r])
    tol = HALF_STEP[dtype] * out + (2.0 ** -11 + 2 * e_s + n * 2.0 ** -22)[..., None] * ref.weight[r] + \
        2.0 ** -20 * ref.bias_weight[r] + e_b[..., None] * out + (n * 2.0 ** -25)[..., None] * ref.largest[r] + 2.0 ** -24
    return tol, e_s + e_b + n * 2.0 ** -23 + 2.0 ** -22 * (lse + 1)


def compare(out, lse, ref, D, dtype, cap=0.0, slopes=None):
    o, s = out.double().cpu().numpy(), lse.double().cpu().numpy()
    r = ref.rows
    assert np.all(o[~r] == 5.0) and np.all(s[~r] == 6.0)                    # rows of no sequence
    o, s = o[r], s[r]
    tol, ltol = tolerances(ref, D, dtype, cap, slopes)
    assert np.all(np.isfinite(o))
    err = np.abs(o - ref.out[r])
    assert np.all(err <= tol), (err / tol).max()
    empty = np.broadcast_to(ref.keys[r][:, None] == 0, s.shape)
    assert np.all(np.isneginf(s[empty])) and np.all(o[empty] == 0)
    assert np.all(np.abs(s[~empty] - ref.lse[r][~empty]) <= ltol[~empty])


def run(q, dev, tables, lens, cu, causal, Hq, D, dtype, cap, slopes, window, prefix, **kw):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")      # noqa: E731
    out = torch.full((q.shape[0], Hq, D), 5.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((q.shape[0], Hq), 6.0, device="cuda")
    fq.attention_nvfp4(q.cuda(), dev, i32(tables), i32(lens), None if cu is None else i32(cu), causal=causal, out=out,
                       return_lse=True, lse=lse, softcap=cap or None, window=window or None,
                       alibi_slopes=None if slopes is None else slopes.cuda(),
                       prefix_lens=None if prefix is None else i32(prefix), **kw)
    torch.cuda.synchronize()
    return out, lse


def check(q, cache, tables, lens, cu, dtype, causal=True, cap=0.0, slopes=None, window=0, prefix=None, shapes=True, **kw):
    T, Hq, D = q.shape
    B, page, Hkv = len(lens), cache[0].shape[2], cache[0].shape[1]
    ref = okv.attention(q.double().numpy(), cache, tables, lens, cu, causal, D ** -0.5, softcap=cap,
                        slopes=None if slopes is None else slopes.numpy(), window=window, prefix=prefix)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    args = (causal, Hq, D, dtype, cap, slopes, window, prefix)
    out, lse = run(q, dev, tables, lens, cu, *args, **kw)
    compare(out, lse, ref, D, dtype, cap, slopes)
    if not shapes:
        return out, lse
    # the other ways of the work: wider tables (an even split of the keys, ranges of them) where no
    # window holds the keys down, and the batch repeated (256-row items)
    if max(lens) <= tables.shape[1] * page and not window:
        for wide in (for_even_split(tables, T, Hq, Hkv, D, page), for_ranges(tables, T, Hq, Hkv, D, page)):
            if wide is not None and wide.shape != tables.shape:
                compare(*run(q, dev, wide, lens, cu, *args), ref, D, dtype, cap, slopes)
    n = times_for_items(B, T, Hq, Hkv, D, tables.shape[1] * page)
    if n is not None and cu is not None and cu[0] == 0 and cu[-1] == T:
        starts = [i * T + c for i in range(n) for c in cu[:-1]] + [n * T]
        more = (causal, Hq, D, dtype, cap, slopes, window, None if prefix is None else list(prefix) * n)
        o, s = run(q.repeat(n, 1, 1), dev, np.tile(tables, (n, 1)), list(lens) * n, starts, *more)
        compare(o[:T], s[:T], ref, D, dtype, cap, slopes)
        body = o.view(n, T, Hq, D)
        assert torch.equal(body, body[:1].expand_as(body))
    return out, lse


def slopes_of(Hq):
    return 2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)


LENS = [1, 2, 15, 16, 17, 33, 63, 64, 65, 127, 129, 255, 0, 257, 513, 700]
PREFIX = [0, 1, 20, 5, 17, 40, -3, 64, 30, 127, 1, 300, 9, 0, 511, 650]
# what a call may ask for: cap, slopes, window, prefix
WHAT = [(c, s, w, p) for c, s, w, p in itertools.product((0.0, 3.0), (False, True), (0, 50), (False, True)) if c or s or w or p]


@pytest.mark.parametrize("cap,slopes,window,prefix", WHAT)
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(12, 2, 128, 16, "bf16"), (4, 4, 64, 48, "fp16"), (10, 1, 64, 32, "bf16"),
                                                 (16, 1, 128, 64, "fp16")])
def test_decode(Hq, Hkv, D, page, dtype, cap, slopes, window, prefix):
    cache, tables = fill_sequences(LENS, Hkv, D, page, seed=Hq)
    check(queries(len(LENS), Hq, D, dtype, 1, size=6.0 if cap else 1.5), cache, tables, LENS, None, dtype, cap=cap,
          slopes=slopes_of(Hq) if slopes else None, window=window, prefix=PREFIX if prefix else None)


# (lengths, query rows): rows before a sequence's first key, one, none, tile edges, ends inside pages
VARLEN = [([5, 3, 40, 0, 64, 7], [7, 3, 17, 2, 0, 1]), ([130, 300, 128], [130, 45, 128]), ([513, 90], [260, 95]),
          ([700], [31])]


@pytest.mark.parametrize("lens,q_lens", VARLEN)
@pytest.mark.parametrize("cap,slopes,window,prefix", WHAT)
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, "bf16"), (3, 3, 64, 48, "fp16")])
def test_many_rows(lens, q_lens, Hq, Hkv, D, page, dtype, cap, slopes, window, prefix):
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=len(lens))
    cu = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    check(queries(cu[-1], Hq, D, dtype, 2, size=6.0 if cap else 1.5), cache, tables, lens, cu, dtype, cap=cap,
          slopes=slopes_of(Hq) if slopes else None, window=window,
          prefix=[n // 2 if i % 2 else n + 3 for i, n in enumerate(lens)] if prefix else None)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 129, 10 ** 12])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 128)])
def test_windows(window, D, page):
    lens, q_lens = [300, 129, 64, 1], [150, 129, 3, 1]
    cache, tables = fill_sequences(lens, 1, D, page, seed=window % 97)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    check(queries(cu[-1], 4, D, "bf16", 3), cache, tables, lens, cu, "bf16", window=window)
    check(queries(4, 4, D, "fp16", 4), cache, tables, lens, None, "fp16", window=window)


@pytest.mark.parametrize("cap,slopes", [(5.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_not_causal(D, cap, slopes):
    lens, q_lens = [100, 333, 0, 17], [70, 20, 5, 140]
    cache, tables = fill_sequences(lens, 2, D, 32, seed=1)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    for Hq in (2, 10):
        check(queries(cu[-1], Hq, D, "bf16", 3, size=3.0), cache, tables, lens, cu, "bf16", causal=False, cap=cap,
              slopes=slopes_of(Hq) if slopes else None)


@pytest.mark.parametrize("cap,slopes,window,prefix", [(0.0, False, 200, False), (0.0, True, 0, True), (7.0, False, 900, True),
                                                      (7.0, True, 0, False)])
@pytest.mark.parametrize("lens,q_lens,Hq,Hkv,D", [([2500, 1200], [300, 515], 4, 1, 128), ([1900, 700], [90, 257], 2, 2, 64)])
def test_long_prompts(lens, q_lens, Hq, Hkv, D, cap, slopes, window, prefix):
    cache, tables = fill_sequences(lens, Hkv, D, 48, seed=3)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    check(queries(cu[-1], Hq, D, "fp16", 5, size=4.0 if cap else 1.5), cache, tables, lens, cu, "fp16", cap=cap,
          slopes=slopes_of(Hq) if slopes else None, window=window, prefix=[1000, 60] if prefix else None)


@pytest.mark.parametrize("cap,slopes,window", [(0.0, False, 3000), (20.0, False, 0), (0.0, True, 0), (20.0, True, 5000)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (24, 2, 64)])
def test_long_sequences(Hq, Hkv, D, cap, slopes, window):
    lens = [9001, 64, 12345, 4097]
    cache, tables = fill_sequences(lens, Hkv, D, 64, seed=9)
    check(queries(4, Hq, D, "bf16", 5, size=6.0 if cap else 1.5), cache, tables, lens, None, "bf16", cap=cap,
          slopes=slopes_of(Hq) if slopes else None, window=window)


@pytest.mark.parametrize("slope", [-0.02, 0.0, 3.0, 40.0])
@pytest.mark.parametrize("q_lens", [[1, 1], [140, 3]])
def test_slopes_of_any_size(slope, q_lens):
    """Of either sign, and so steep that a row's own key is all it sees in fp32."""
    lens = [700, 260]
    cache, tables = fill_sequences(lens, 1, 64, 16, seed=4)
    cu = [0, q_lens[0], sum(q_lens)]
    check(queries(cu[-1], 3, 64, "bf16", 6), cache, tables, lens, cu, "bf16", slopes=torch.tensor([slope, 0.1, -slope / 2]))


@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("size", [1e-3, 30.0, 2000.0])
@pytest.mark.parametrize("cap", [1e-2, 50.0, 1048576.0])
def test_caps_of_any_size(size, cap, T):
    """From logits that all meet the cap to those that never do."""
    cache, tables = fill_sequences([300], 1, 128, 16, seed=5)
    q = queries(T, 4, 128, "fp16", 7, size=size)
    check(q, cache, tables, [300], [0, T], "fp16", cap=cap)


@pytest.mark.parametrize("T", [1, 200])
def test_tiny_caps_and_huge_queries(T):
    """Where the product's factor leaves fp32: every logit meets the cap, products of 0 stay 0."""
    cache, tables = fill_sequences([200], 1, 64, 16, seed=5)
    q = queries(T, 4, 64, "bf16", 7, size=1e30)
    q[0, 1] = 0
    check(q, cache, tables, [200], [0, T], "bf16", cap=1e-30, shapes=False)


def test_large_logits_with_windows_and_biases():
    """References beyond 2^22, where products are rounded before a reference is taken from them."""
    cache, tables = fill_sequences([200, 77], 1, 64, 16, seed=6)
    q = queries(100, 4, 64, "bf16", 8, size=1e6)
    check(q, cache, tables, [200, 77], [0, 90, 100], "bf16", window=120)
    check(q, cache, tables, [200, 77], [0, 90, 100], "bf16", slopes=torch.full((4,), 0.5))


@pytest.mark.parametrize("cap,slopes,window,prefix", [(0.0, False, 40, False), (0.0, True, 0, True), (4.0, False, 0, True),
                                                      (4.0, True, 30, False)])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [1, 40, 150]])
def test_bad_pages_are_masked(q_lens, cap, slopes, window, prefix):
    lens = [150, 170, 150]
    cache, tables = fill_sequences(lens, 2, 128, 16, seed=7, bad=[(0, 0, -1), (1, 3, 1 << 30), (2, 9, -5), (1, 10, -1)])
    cu = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    check(queries(cu[-1], 4, 128, "bf16", 9), cache, tables, lens, cu, "bf16", cap=cap, slopes=slopes_of(4) if slopes else None,
          window=window, prefix=[20, 170, 3] if prefix else None)


@pytest.mark.parametrize("T", [1, 150])
@pytest.mark.parametrize("kw", [dict(cap=5.0), dict(window=70), dict(slopes=True), dict(cap=5.0, slopes=True)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_row_stays_alone(T, kw, bad):
    kw = dict(kw, slopes=slopes_of(4) if kw.get("slopes") else None)
    cache, tables = fill_sequences([200], 1, 128, 16, seed=8)
    q = queries(T, 4, 128, "bf16", 9)
    ref, _ = check(q, cache, tables, [200], [0, T], "bf16", shapes=False, **kw)
    q[T // 2, 2, 77] = bad
    dev = [torch.from_numpy(c).cuda() for c in cache]
    out, lse = run(q, dev, tables, [200], [0, T], True, 4, 128, "bf16", kw.get("cap", 0.0), kw["slopes"], kw.get("window", 0), None)
    assert torch.all(torch.isnan(out[T // 2, 2])) and torch.isnan(lse[T // 2, 2])
    keep = torch.ones(T, 4, dtype=torch.bool)
    keep[T // 2, 2] = False
    assert torch.equal(out.cpu()[keep], ref.cpu()[keep])


def test_nothing_asked_for_is_the_plain_call():
    cache, tables = fill_sequences([300, 40], 2, 128, 16, seed=1)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    t, l = torch.from_numpy(tables.astype(np.int32)).cuda(), torch.tensor([300, 40], dtype=torch.int32, device="cuda")
    q = queries(2, 8, 128, "bf16", 1).cuda()
    plain = fq.attention_nvfp4(q, dev, t, l)
    # a window longer than the sequences, slopes of 0, prefixes of 0 change nothing but roundings
    for kw in (dict(window=5000), dict(alibi_slopes=torch.zeros(8, device="cuda")), dict(prefix_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        assert torch.allclose(fq.attention_nvfp4(q, dev, t, l, **kw).float(), plain.float(), rtol=2.0 ** -7, atol=2.0 ** -9)


@pytest.mark.parametrize("T,kw", [(3, dict(cap=5.0, window=60)), (200, dict(slopes=True, prefix=[50, 8])), (200, dict(cap=5.0))])
def test_strides_graphs_streams_and_workspaces(T, kw):
    lens = [300, 90]
    cache, tables = fill_sequences(lens, 2, 64, 16, seed=2)
    cu = [0, T - 1, T]
    kw = dict(kw, slopes=slopes_of(6) if kw.get("slopes") else None)
    wide = torch.zeros(T, 6 * 64 + 32, dtype=torch.bfloat16)
    wide[:, 16:16 + 384] = queries(T, 6, 64, "bf16", 3).view(T, 384)
    q = wide.cuda()[:, 16:16 + 384].unflatten(-1, (6, 64))
    dense = q.contiguous().cpu()
    want, _ = check(dense, cache, tables, lens, cu, "bf16", **kw)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    t, l = torch.from_numpy(tables.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    opts = dict(softcap=kw.get("cap"), window=kw.get("window"), alibi_slopes=None if kw["slopes"] is None else kw["slopes"].cuda(),
                prefix_lens=None if kw.get("prefix") is None else torch.tensor(kw["prefix"], dtype=torch.int32, device="cuda"))
    assert torch.equal(fq.attention_nvfp4(q, dev, t, l, c, **opts), want)
    bound = fq.fp4_attention_workspace_bound(2, T, 6, 2, 64, tables.shape[1] * 16)
    ws = torch.full((max(bound, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(fq.attention_nvfp4(q, dev, t, l, c, workspace=ws, pdl=True, **opts), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = fq.attention_nvfp4(q, dev, t, l, c, stream=side, **opts)
    side.synchronize()
    assert torch.equal(on_side, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        fq.attention_nvfp4(q, dev, t, l, c, out=out, workspace=ws, **opts)
    l.copy_(torch.tensor([120, 33]))
    graph.replay()
    torch.cuda.synchronize()
    ref = okv.attention(dense.double().numpy(), cache, tables, [120, 33], cu, True, 64 ** -0.5, softcap=kw.get("cap", 0.0),
                        slopes=None if kw["slopes"] is None else kw["slopes"].numpy(), window=kw.get("window", 0), prefix=kw.get("prefix"))
    err = np.abs(out.double().cpu().numpy() - ref.out)
    assert np.all(err <= tolerances(ref, 64, "bf16", kw.get("cap", 0.0), kw["slopes"])[0])


def test_refusals():
    cache, tables = fill_sequences([30, 40], 1, 64, 16, seed=2)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    t, l = torch.from_numpy(tables.astype(np.int32)).cuda(), torch.tensor([30, 40], dtype=torch.int32, device="cuda")
    q = queries(2, 2, 64, "bf16", 1).cuda()
    slopes, prefix = torch.ones(2, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    for kw in (dict(softcap=0.0), dict(softcap=-1.0), dict(softcap=float("nan")), dict(window=0), dict(window=-3),
               dict(alibi_slopes=slopes[:1]), dict(alibi_slopes=slopes.double()), dict(alibi_slopes=slopes.cpu()),
               dict(prefix_lens=prefix.long()), dict(prefix_lens=prefix[:1]), dict(window=5, causal=False),
               dict(prefix_lens=prefix, causal=False)):
        with pytest.raises(ValueError):
            fq.attention_nvfp4(q, dev, t, l, **kw)
    for kw in (dict(softcap=2.0 ** 21), dict(softcap=float("inf"))):
        with pytest.raises(fq.Fp4Error):
            fq.attention_nvfp4(q, dev, t, l, **kw)


def test_debug_build_finds_no_access_out_of_bounds():
    fbuild.build(debug=True)
    L = fq.debug_lib()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, bad.data_ptr()) == 0
    try:
        with fq.using_library(L):
            for what in WHAT[::3]:
                test_decode(12, 2, 128, 16, "bf16", *what)
                for lens, q_lens in VARLEN:
                    test_many_rows(lens, q_lens, 8, 2, 128, 16, "bf16", *what)
                    test_many_rows(lens, q_lens, 3, 3, 64, 48, "fp16", *what)
            test_windows(65, 64, 128)
            test_bad_pages_are_masked([1, 40, 150], 4.0, True, 30, False)
            assert bad.item() == 0
    finally:
        L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, None)
