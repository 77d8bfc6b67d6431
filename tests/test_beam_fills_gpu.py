"""Beam selection over vocabularies filled with large finite values, and over rows far from 0,
against the oracle.

Tolerance: as in test_beam_gpu; up to 2^30 an exponent may come out 86 further from 0 than the
64 counted there (M is a multiple of up to 128, and x times what log2(e)'s first float leaves, up
to 21), which two roundings of 2^-24 and log(2) make 7.2e-6, and log2(e), log(2) and the pairs of
floats are off by 2^-47 of x together: 1.5e-5 in all.  Beyond 2^30 the terms are ones and zeros.
"""
import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import beam as obeam
from rmsnorm_fp4_quant_gb300 import build as fbuild
from test_beam_gpu import DT, LOG_ERROR, check, inputs

pytestmark = pytest.mark.gpu

FAR_ERROR = LOG_ERROR + 1.5e-5
FILLS = [-1e9, -1e10, -1e12, -1e18, -1e20, -1e24, -1e30, -1e35]


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


def check_far(x, scores, n):
    want = obeam.select(x.double().numpy(), scores.double().numpy(), n)
    assert want[4].min() > 2.2 * FAR_ERROR, "the case leaves the order of two beams open"
    got = fq.beam_select(x.cuda(), scores.cuda(), n)
    torch.cuda.synchronize()
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])
    s, w = got[0].double().cpu().numpy(), want[0]
    assert np.array_equal(np.isneginf(s), np.isneginf(w))
    f = np.isfinite(w)
    assert np.all(np.abs(s[f] - w[f]) <= FAR_ERROR + 2.0 ** -24 * np.abs(w[f]))


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_filled_tokens(dtype, fill):
    """16 neighbours, a whole group, all but 40 tokens, at the row's start, end and middle."""
    x, scores, _ = inputs(4, 3, 3001, dtype, seed=21)
    x[0, 0, :16] = x[0, 1, 2985:] = x[0, 2, 600:616] = fill
    x[1, 0, :512] = x[1, 1, 2400:] = x[1, 2, 512:1024] = fill
    x[2, :, 20:2981] = fill
    x[3, :, 40:] = fill
    x[3, 1] = x[3, 1].flip(0)
    check(x, scores, 12)


@pytest.mark.parametrize("fill", [-1e4, -65504.0])
def test_filled_tokens_in_fp16(fill):
    x, scores, _ = inputs(2, 3, 3001, "fp16", seed=26)
    x[0, :, :16] = fill
    x[1, :, 40:] = fill
    check(x, scores, 12)


@pytest.mark.parametrize("fill", [-1e10, -1e30])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_vocabulary_of_a_few_tokens(dtype, fill):
    """More places than tokens that are not filled: then the filled ones follow, lowest first."""
    x = torch.full((2, 1, 50001), fill, dtype=DT[dtype])
    x[:, 0, [7, 30000, 49999]] = torch.tensor([1.0, 3.0, 2.0], dtype=DT[dtype])
    x[1, 0, 30000] = fill
    check(x, torch.tensor([[-2.0], [-3.0]]), 20)


@pytest.mark.parametrize("fill", [-1e18, -1e20, -1e30])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_filled_tokens_of_several_beams_come_in_order(dtype, fill):
    """Behind the tokens that are not filled all scores are the fill in 64 bits: lowest beam and
    token first, whatever the beams' own scores are."""
    x = torch.full((2, 3, 2003), fill, dtype=DT[dtype])
    x[:, 0, 1000], x[:, 1, [5, 6]], x[0, 2, 2002] = 1.0, torch.tensor([3.0, 1.0], dtype=DT[dtype]), 2.0
    scores = torch.tensor([[-9.0, -3.25, -1.5], [-2.0, -7.5, -float("inf")]])
    finished = torch.zeros(2, 3, dtype=torch.bool)
    total = scores.double()[..., None] + torch.log_softmax(x.double(), -1)
    value, index = torch.sort(total.flatten(1), dim=1, descending=True, stable=True)
    some = value[:, :40] > -float("inf")
    parents = torch.where(some, index[:, :40] // 2003 + 3 * torch.arange(2)[:, None], -1)
    tokens = torch.where(some, index[:, :40] % 2003, -1)
    for kw in (dict(), dict(finished=finished.cuda(), end_token=7)):
        got = fq.beam_select(x.cuda(), scores.cuda(), 40, **kw)
        assert torch.equal(got[1].cpu().long(), parents) and torch.equal(got[2].cpu().long(), tokens)
        assert torch.allclose(got[0].cpu().double(), value[:, :40], rtol=2.0 ** -23, atol=FAR_ERROR)


FAR = [v for m in (1.25e7, 1e9, 2.0 ** 30, 2.0 ** 30 + 128, 1e10, 1e20, 1e30, 4e37) for v in (m, -m)]


@pytest.mark.parametrize("value", FAR)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_of_one_far_value(dtype, value):
    """A row of equal logits is uniform wherever it lies."""
    x, _, _ = inputs(1, 3, 1003, dtype, seed=23)
    x[0, 0], x[0, 2] = value, value
    check_far(x, torch.tensor([[-1.0, -7.25, -1.5]]), 30)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("middle,step", [(2.0 ** 24, 2.0), (2.0 ** 30, 64.0), (2.0 ** 30 - 4096, 64.0), (1e10, 1024.0), (1e30, 2.0 ** 77)])
def test_rows_of_neighbouring_far_values(middle, step, sign):
    """Values a few of fp32's steps apart, on both sides of 2^30 among them."""
    g = torch.Generator().manual_seed(24)
    x = sign * (middle + step * torch.randint(-3, 4, (2, 2, 2000), generator=g).double()).float()
    x[1, 0] = torch.sort(x[1, 0])[0]                         # every step moves the reference
    x[1, 1] = torch.sort(x[1, 1], descending=True)[0]
    check_far(x, torch.tensor([[-1.0, -1.75], [-2.0, -2.5]]), 10)


def test_logits_beyond_the_range_empty_their_beam():
    x, scores, _ = inputs(1, 4, 700, "fp32", seed=25)
    x[0, 0, 9] = 4.3e37                          # above 2^125
    x[0, 1, 9] = 3e38
    x[0, 2, 9] = -4.3e37                         # below -2^125: a mask
    check(x, scores, 9)
    y = torch.full((1, 2, 700), -4.3e37)
    got = fq.beam_select(y.cuda(), torch.zeros(1, 2, device="cuda"), 3)
    assert got[1].tolist() == [[-1] * 3] and got[0].tolist() == [[float("-inf")] * 3]
