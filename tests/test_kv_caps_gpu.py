"""Attention with caps far above the logits, against the oracle.

Tolerance: as in test_kv_masks_gpu without its term of the cap.  Above a cap of 256 a logit is off
by 2^-19 of itself at most (below a quarter of the cap the series' steps, a few 2^-24 of it; above,
the exponential 2^-22 and its argument's rounding, times 2 e / (1 + e)^2 <= 1/2, a reciprocal
2^-23 and two roundings, 2^-21.3 of the cap, which is at most 4.1 times the result), and its size
is at most the sum of |scale q k|: L 2^-19 in the logits, twice that in the weights.
"""
import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import kv_cache as okv
from rmsnorm_fp4_quant_gb300 import build as fbuild
from test_kv_cache_gpu import fill_sequences, for_even_split, for_ranges, queries
from test_kv_masks_gpu import run, slopes_of, tolerances

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


def check(q, cache, tables, lens, cu, dtype, cap, oracle_cap, slopes=None, window=0, prefix=None):
    T, Hq, D = q.shape
    Hkv, page = cache[0].shape[1:3]
    ref = okv.attention(q.double().numpy(), cache, tables, lens, cu, True, D ** -0.5, softcap=oracle_cap,
                        slopes=None if slopes is None else slopes.numpy(), window=window, prefix=prefix)
    tol, ltol = tolerances(ref, D, dtype, 0.0, slopes)
    tol, ltol = tol + 2.0 ** -18 * ref.logit[..., None] * ref.weight, ltol + 2.0 ** -19 * ref.logit
    dev = [torch.from_numpy(c).cuda() for c in cache]
    wide = [] if window else [for_even_split(tables, T, Hq, Hkv, D, page), for_ranges(tables, T, Hq, Hkv, D, page)]
    for t in [tables] + [w for w in wide if w is not None]:
        out, lse = run(q, dev, t, lens, cu, True, Hq, D, dtype, cap, slopes, window, prefix)
        assert np.all(np.abs(out.double().cpu().numpy() - ref.out) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - ref.lse) <= ltol)


@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("size", [1e-3, 1.5, 30.0, 2000.0])
@pytest.mark.parametrize("cap", [256.01, 1000.0, 2.0 ** 15, 2.0 ** 20])
def test_wide_caps(cap, size, T):
    """Logits from far below the cap, where it changes nothing, to ones that meet it."""
    for D, page in ((128, 16), (64, 48)):
        cache, tables = fill_sequences([300], 1, D, page, seed=41)
        check(queries(T, 4, D, "fp16", 42, size=size), cache, tables, [300], [0, T], "fp16", cap, cap)


@pytest.mark.parametrize("slopes,window,prefix", [(True, 0, False), (False, 90, False), (True, 150, True)])
@pytest.mark.parametrize("lens,q_lens", [([300, 77, 1, 640], [1, 1, 1, 1]), ([333, 400], [120, 290])])
def test_wide_caps_with_the_rest(lens, q_lens, slopes, window, prefix):
    cache, tables = fill_sequences(lens, 2, 64, 16, seed=43)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    check(queries(cu[-1], 6, 64, "bf16", 44, size=30.0), cache, tables, lens, cu, "bf16", 500.0, 500.0,
          slopes_of(6) if slopes else None, window, [n // 3 for n in lens] if prefix else None)


def test_a_cap_below_fp32s_numbers_is_refused():
    """It is 0 in fp32, which the C call takes for no cap at all."""
    cache, tables = fill_sequences([30], 1, 64, 16, seed=47)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    t, l = torch.from_numpy(tables.astype(np.int32)).cuda(), torch.tensor([30], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        fq.attention_nvfp4(queries(1, 2, 64, "bf16", 48).cuda(), dev, t, l, softcap=1e-46)


@pytest.mark.parametrize("T", [1, 200])
def test_a_cap_far_above_the_logits_changes_nothing(T):
    """Logits x of up to some 30: x - cap tanh(x / cap) = x^3 / (3 cap^2) is below 2^-26 of that."""
    cache, tables = fill_sequences([700], 2, 128, 16, seed=45)
    check(queries(T, 8, 128, "fp16", 46, size=4.0), cache, tables, [700], [0, T], "fp16", 2.0 ** 20, 0.0)
