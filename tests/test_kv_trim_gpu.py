"""Trim where no token stays (first >= end): the page that both places lie in is kept for the next
token, against the oracle and the fork that follows."""
import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import kv_pages as opg
from rmsnorm_fp4_quant_gb300 import build as fbuild
from test_kv_pages_gpu import dev, random_cache, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


@pytest.mark.parametrize("page", [16, 48])
def test_an_empty_range_keeps_the_next_tokens_page(page):
    # a sequence for each: first and end inside one page, at its edges, in different pages
    n = 3 * page + 5
    first = [page + 4, page + 4, page + 9, page, 2 * page, 2 * page, n, n + 7, 3 * page]
    end = [page + 4, page + 9, page + 4, page, 2 * page, page + 4, n, n, n]
    B = len(first)
    tables = np.arange(4 * B).reshape(B, 4)[:, ::-1].copy()
    refs = np.concatenate([np.ones(4 * B, np.int64), np.zeros(4, np.int64)])
    cache = random_cache(4 * B + 4, 1, page, 64, 1)
    c = [torch.from_numpy(x).cuda() for x in cache]
    got = fq.kv_trim_nvfp4(c, dev(refs), dev(tables), dev([n] * B), dev(first), dev(end))
    want = opg.trim(page, refs, tables, [n] * B, first, end)
    for name, a, b in zip(("tables", "lens", "refs"), got, want):
        same(name, a, b)
    kept = [[i for i, p in enumerate(t) if p >= 0] for t in want[0]]
    assert kept == [[1], [1], [1], [], [], [], [3], [3], [3]]
    after = fq.kv_fork_nvfp4(c, got[2], got[0], got[1])
    o = opg.fork(cache, want[2], want[0], want[1], np.arange(B), 1)
    for name, a, b in zip(("tables", "lens", "refs", "slots"), after, o):
        same(name, a, b)
    # the next token of a sequence whose page stays has the place of `end`; where that is a page's
    # first, the token takes a page
    slots = after[3][:, 0].tolist()
    for b in (0, 1, 2, 6, 7, 8):
        assert slots[b] == tables[b, end[b] // page] * page + end[b] % page
    assert slots[3] >= 0 and slots[4] >= 0
