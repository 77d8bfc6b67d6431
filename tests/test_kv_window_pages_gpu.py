"""Attention over a window whose table still names pages before it: given away by the program,
they may hold anything, scales that are no numbers among it, and must not count.

Tolerance against the oracle: as in test_kv_masks_gpu.  Entries before the window that hold
no page give the same bits.
"""
import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from rmsnorm_fp4_quant_gb300 import build as fbuild
from test_kv_cache_gpu import fill_sequences, queries
from test_kv_masks_gpu import check, run, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


def give_away(cache, tables, lens, q_lens, window, page):
    """Other bytes in every page that lies before its sequence's first window; the tables without them."""
    without = tables.copy()
    for b, n in enumerate(lens):
        gone = max(0, n - q_lens[b] + 1 - window) // page
        for i, p in enumerate(tables[b, :gone]):
            cache[1][p], cache[3][p] = (0x7F, 0xFF)[i % 2], (0xFF, 0x7F)[i % 2]
            cache[0][p] = cache[2][p] = 0x77
        without[b, :gone] = -1
    assert np.any(without != tables)
    return without


CASES = [
    # lengths, query rows: single tokens, a few rows, 256-row items, mixed ones
    ([300, 129, 700, 64, 517], [1, 1, 1, 1, 1]),
    ([333, 150, 640], [3, 7, 2]),
    ([700, 433], [200, 290]),
    ([650, 900, 77], [1, 300, 40]),
]
KINDS = [dict(), dict(cap=5.0), dict(slopes=True), dict(prefix=True), dict(cap=5.0, slopes=True, prefix=True)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 20, 50, 100, 177])
@pytest.mark.parametrize("lens,q_lens", CASES)
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 48, "fp16"), (6, 1, 64, 32, "bf16"),
                                                 (4, 1, 128, 64, "fp16"), (2, 2, 128, 128, "bf16")])
def test_pages_before_a_window_do_not_count(Hq, Hkv, D, page, dtype, lens, q_lens, window, kind):
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=window)
    without = give_away(cache, tables, lens, q_lens, window, page)
    T = sum(q_lens)
    cu = None if T == len(lens) else np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    cap, slopes = kind.get("cap", 0.0), slopes_of(Hq) if kind.get("slopes") else None
    prefix = [n // 2 for n in lens] if kind.get("prefix") else None
    q = queries(T, Hq, D, dtype, 31, size=6.0 if cap else 1.5)
    out, lse = check(q, cache, tables, lens, cu, dtype, cap=cap, slopes=slopes, window=window, prefix=prefix)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    o, s = run(q, dev, without, lens, cu, True, Hq, D, dtype, cap, slopes, window, prefix)
    assert torch.equal(out, o) and torch.equal(lse, s)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("lens,q_lens,Hq,Hkv,D,page", [([9001, 7321, 12345, 4097], [1, 1, 1, 1], 8, 2, 128, 16),
                                                       ([6000], [200], 4, 1, 64, 32)])
def test_long_windows(lens, q_lens, Hq, Hkv, D, page, slopes):
    """Keys shared by CTAs and cut into ranges."""
    window = 3001
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=33)
    give_away(cache, tables, lens, q_lens, window, page)
    T = sum(q_lens)
    cu = None if T == len(lens) else np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    check(queries(T, Hq, D, "bf16", 34), cache, tables, lens, cu, "bf16", slopes=slopes_of(Hq) if slopes else None, window=window)
