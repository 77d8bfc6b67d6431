"""Beam selection on the GPU against the oracle.

Tolerance of a score, from the kernels' roundings: a term 2^(x log2(e) - M) of a row's sum is
off by 2^-22 (the exponential), and by the rounding of its exponent, which is at most 64 where
the term counts: 2 * 64 * 2^-24 * log(2); a sum has at most 9 roundings inside a group of 512,
one for each group of a part and 13 over lanes, 2^-24 each, with at most 400 groups in a row here.
That is 3.1e-5 in the logarithm; pairs of floats add nothing that shows.  Then the score's
own rounding.  What the scores of different beams are ordered by differs by twice that at most,
so every case keeps neighbouring candidates of different beams 7e-5 apart (checked).
"""
import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import beam as obeam
from rmsnorm_fp4_quant_gb300 import build as fbuild

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LOG_ERROR = 3.1e-5


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


def inputs(B, K, V, dtype, seed, finished=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, K, V, generator=g) * 2.5
    x[:, :, :: max(1, V // 7)] += 4.0
    scores = -torch.rand(B, K, generator=g) * 5 - 7
    done = torch.rand(B, K, generator=g) < 0.3 if finished else None
    return x.to(DT[dtype]), scores, done


def check(x, scores, n, done=None, end=0, device_logits=None, **kw):
    want = obeam.select(x.double().numpy(), scores.double().numpy(), n, None if done is None else done.numpy(), end)
    assert want[4].min() > 7e-5, "the case leaves the order of two beams open"
    got = fq.beam_select(x.cuda() if device_logits is None else device_logits, scores.cuda(), n,
                         finished=None if done is None else done.cuda(), end_token=end, **kw)
    torch.cuda.synchronize()
    compare(got, want, done is not None)
    return got


def compare(got, want, with_done):
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[2].cpu().numpy(), want[2])
    s, w = got[0].double().cpu().numpy(), want[0]
    assert np.array_equal(np.isneginf(s), np.isneginf(w))
    f = np.isfinite(w)
    assert np.all(np.abs(s[f] - w[f]) <= LOG_ERROR + 2.0 ** -24 * np.abs(w[f]))
    assert len(got) == (4 if with_done else 3)
    if with_done:
        assert np.array_equal(got[3].cpu().numpy(), want[3])


CASES = [
    # B, K, V, n, dtype, some beams ended
    (1, 1, 1, 1, "bf16", False),
    (1, 1, 1, 3, "fp32", False),                 # more places than candidates
    (2, 3, 2, 8, "fp16", True),
    (3, 2, 7, 4, "bf16", True),
    (1, 4, 511, 4, "fp16", False),
    (1, 4, 512, 64, "fp32", False),
    (2, 5, 513, 10, "bf16", True),
    (1, 1, 8191, 32, "fp16", False),
    (2, 1, 8200, 33, "fp32", False),
    (4, 3, 1003, 7, "bf16", True),
    (5, 8, 4097, 17, "fp32", True),
    (1, 12, 32001, 24, "fp16", False),
    (7, 2, 50001, 5, "bf16", True),
    (1, 2, 200003, 64, "fp32", False),
    (40, 9, 781, 18, "fp16", True),
    (1, 256, 301, 7, "fp32", True),
    (300, 1, 600, 2, "fp16", False),
]


@pytest.mark.parametrize("B,K,V,n,dtype,ended", CASES)
def test_selection(B, K, V, n, dtype, ended):
    x, scores, done = inputs(B, K, V, dtype, seed=B + K + V, finished=ended)
    check(x, scores, n, done, end=min(2, V - 1))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lead", [1, 3, 8])
def test_rows_of_any_alignment(dtype, lead):
    """Columns of a wider matrix: every row begins somewhere else in its 32 bytes."""
    x, scores, _ = inputs(3, 4, 1501, dtype, seed=lead)
    wide = torch.full((12, 1600 + lead), 50.0, dtype=DT[dtype], device="cuda")
    view = wide[:, lead:lead + 1501]
    view.copy_(x.view(12, 1501).cuda())
    check(x, scores, 6, device_logits=view.unflatten(0, (3, 4)))


def test_masked_tokens():
    x, scores, _ = inputs(3, 4, 3001, "fp32", seed=1)
    x[0, :, 5:2990] = -np.inf                    # whole groups without a candidate
    x[1, 1] = -np.inf                            # a row without one
    x[1, 2, 17:] = torch.finfo(torch.float32).min
    x[2, 0, 3] = np.nan                          # rows that have none
    x[2, 1, 3000] = np.inf
    x[2, 2, 7] = 1e38
    check(x, scores, 12)
    y = x.to(torch.bfloat16)
    y[1, 3] = torch.finfo(torch.bfloat16).min
    check(y, scores, 12)


def test_first_step_and_dead_beams():
    x, scores, _ = inputs(4, 5, 2000, "bf16", seed=2)
    scores[:, 1:] = -np.inf
    scores[3, 0] = np.nan
    got = check(x, scores, 10)
    assert torch.all(got[1][3] == -1) and torch.all(got[2][3] == -1)
    scores[:] = np.inf
    check(x, scores, 10)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_equal_logits(dtype, V):
    """Ties go to the lowest token, zeros of both signs among them; more ties than any list holds."""
    x = torch.zeros(2, 3, V, dtype=DT[dtype])
    x[:, :, 1::2] = -0.0
    x[1] = 2.5
    scores = torch.tensor([[-1.0, -2.13, -3.37], [-1.0, -1.41, -0.57]])
    check(x, scores, 20)
    few = (torch.arange(V) % 5).to(DT[dtype]).expand(2, 3, V).contiguous()
    check(few, scores, 64)


def test_equal_beams_come_in_order():
    g = torch.Generator().manual_seed(3)
    row = torch.randn(1, 1, 4096, generator=g)
    got = fq.beam_select(row.expand(2, 4, 4096).contiguous().cuda(), torch.full((2, 4), -3.0).cuda(), 8)
    assert torch.equal(got[1].cpu(), torch.tensor([[0, 1, 2, 3] * 2, [4, 5, 6, 7] * 2], dtype=torch.int32))
    best = row.flatten().topk(2).indices
    assert torch.equal(got[2].cpu(), torch.stack([best[0]] * 4 + [best[1]] * 4).int().expand(2, 8))


def test_large_logits_and_scores():
    """Sums whose reference moves on the way, and rows far from 0."""
    x, scores, _ = inputs(2, 3, 9000, "fp32", seed=5)
    x[0, 0] += torch.linspace(0, 60000, 9000)
    x[0, 1] -= 7000.0
    x[0, 2, 4000:] += 300.0
    x[1] *= 40.0
    want = obeam.select(x.double().numpy(), scores.double().numpy(), 9)
    got = fq.beam_select(x.cuda(), scores.cuda(), 9)
    # exponents and M up to 86625: rounding them counts 2^-24 of that; rows of spread logits
    s, w = got[0].double().cpu().numpy(), want[0]
    assert np.all(np.abs(s - w) <= LOG_ERROR + 2 * 2.0 ** -24 * 86625 * np.log(2) + 2.0 ** -24 * np.abs(w))
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])


def test_repeats_graphs_streams_and_workspaces():
    x, scores, done = inputs(3, 4, 20011, "fp16", seed=7, finished=True)
    dx, ds, dd = x.cuda(), scores.cuda(), done.cuda()
    first = fq.beam_select(dx, ds, 8, finished=dd, end_token=1)
    size = fq.fp4_beam_select_workspace_bytes(3, 4, 20011, 8, fq.FP4_DT_FP16)
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again = fq.beam_select(dx, ds, 8, finished=dd, end_token=1, workspace=ws, pdl=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = fq.beam_select(dx, ds, 8, finished=dd, end_token=1, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, on_side))
    # captured, then replayed on other inputs
    out = [torch.empty_like(t) for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.beam_select(dx, ds, 8, finished=dd, end_token=1, out=out, workspace=ws)
    y, s2, d2 = inputs(3, 4, 20011, "fp16", seed=8, finished=True)
    dx.copy_(y), ds.copy_(s2), dd.copy_(d2)
    graph.replay()
    torch.cuda.synchronize()
    want = obeam.select(y.double().numpy(), s2.double().numpy(), 8, d2.numpy(), 1)
    assert want[4].min() > 7e-5
    compare(out, want, True)


def test_offsets_beyond_32_bits():
    """Rows that begin behind 2^31 elements."""
    V = (1 << 24) - 5
    wide = torch.zeros(140, V, dtype=torch.bfloat16, device="cuda")
    wide[139, 12345], wide[139, V - 1], wide[131, 7] = 9.0, 8.0, 7.0
    scores = torch.full((1, 140), -np.inf, device="cuda")
    scores[0, 139], scores[0, 131] = -1.0, -2.0
    s, p, t = fq.beam_select(wide.view(1, 140, V), scores, 3)
    assert p.tolist() == [[139, 139, 131]] and t.tolist() == [[12345, V - 1, 7]]
    total = np.log(V - 2 + np.exp(9.0) + np.exp(8.0))
    assert abs(s[0, 0].item() - (-1 + 9 - total)) < 2e-3          # (65536 sums of a part's 32768 groups: 2^-24 each)


def test_an_empty_batch():
    for done in (None, torch.zeros(0, 4, dtype=torch.bool, device="cuda")):
        got = fq.beam_select(torch.zeros(0, 4, 100, device="cuda"), torch.zeros(0, 4, device="cuda"), take=3, finished=done)
        torch.cuda.synchronize()
        assert len(got) == (3 if done is None else 4) and all(t.shape == (0, 3) for t in got)


def test_refusals():
    x, scores, done = inputs(2, 3, 100, "bf16", seed=1, finished=True)
    dx, ds, dd = x.cuda(), scores.cuda(), done.cuda()
    for bad in (dx[0], dx.double(), dx[:, :, ::2], dx.transpose(0, 1), x):
        with pytest.raises(ValueError):
            fq.beam_select(bad, ds, 3)
    for kw in (dict(scores=ds[:1]), dict(scores=ds.double()), dict(scores=scores), dict(finished=done),
               dict(finished=dd.int()), dict(out=[torch.empty(2, 3, device="cuda")]),
               dict(finished=dd, out=[torch.empty(2, 3, device="cuda")] * 3)):
        with pytest.raises(ValueError):
            fq.beam_select(dx, **{**dict(scores=ds, take=3), **kw})
    for kw in (dict(take=0), dict(take=65), dict(finished=dd, end_token=100), dict(finished=dd, end_token=-1),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fq.Fp4Error):
            fq.beam_select(dx, ds, **kw)


def test_debug_build_finds_no_access_out_of_bounds():
    fbuild.build(debug=True)
    L = fq.debug_lib()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, bad.data_ptr()) == 0
    try:
        with fq.using_library(L):
            for args in CASES[:12]:
                test_selection(*args)
            test_rows_of_any_alignment("fp16", 3)
            test_masked_tokens()
            test_equal_logits("bf16", 5000)
            assert bad.item() == 0
            assert L.fp4_debug_configure(2_000_000_000, 1, 0, -1, -1, bad.data_ptr()) == 0
            x, scores, done = inputs(2, 3, 640, "bf16", seed=1, finished=True)
            fq.beam_select(x.cuda(), scores.cuda(), 4, finished=done.cuda())
            torch.cuda.synchronize()
            assert bad.item() > 0
    finally:
        L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, None)
