"""Small weights beside a large one, one row a sequence, against the oracle: with a window, a
prefix, a bias or a cap they keep the bits that they have without.

Every warp's first tile holds a key whose logit is 17.7 above all others' and whose value is 0, so
that the output is what the many keys with weights of 2^-25.5 add up to.  Tolerance: as in
test_kv_masks_gpu, but a small weight is rounded to half of fp16's smallest step against a
reference 6 octaves below the largest, 2^-31 of that (against the largest itself 2^-25: 0).
"""
import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import kv_cache as okv
from rmsnorm_fp4_quant_gb300 import build as fbuild
from test_kv_cache_gpu import fill_sequences, shape_of
from test_kv_masks_gpu import run, tolerances

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


@pytest.mark.parametrize("what", ["none", "window", "prefix", "slopes", "cap", "wide cap"])
@pytest.mark.parametrize("D,rows", [(64, 1), (64, 12), (128, 1), (128, 12)])
def test_small_weights_count(D, rows, what):
    n, B = 1000, 400
    cache, tables = fill_sequences([n], 1, D, 16, seed=51)
    k, v = np.zeros((n, 1, D)), np.ones((n, 1, D))
    large = [0, 16, 32, 48, 944, 960, 976, 992]              # a key of every warp's first tile, from either end
    k[large, 0, 0], v[large] = 4.0, 0.0
    j = np.arange(n)
    okv.append(cache, k, v, tables[0][j // 16] * 16 + j % 16)
    key = okv.gather(cache, tables[0][:1] * 16)[0][0, 0, 0]  # what the cache made of 4
    q = torch.zeros(1, rows, D, dtype=torch.float16)
    q[..., 0] = 25.5 * np.log(2.0) / key * D ** 0.5
    cap = {"cap": 200.0, "wide cap": 5000.0}.get(what, 0.0)
    slopes = torch.full((rows,), 1e-6) if what == "slopes" else None
    window, prefix = 5000 if what == "window" else 0, [n // 2] if what == "prefix" else None
    assert shape_of(B, B, rows, 1, D, tables.shape[1] * 16) == {"kernel": "kv_decode_kernel", "parts": 1}
    ref = okv.attention(q.double().numpy(), cache, tables, [n], None, True, D ** -0.5, softcap=cap,
                        slopes=None if slopes is None else slopes.numpy(), window=window, prefix=prefix)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    out, _ = run(q.expand(B, rows, D).contiguous(), dev, np.tile(tables, (B, 1)), [n] * B, None, True, rows, D, "fp16", cap,
                 slopes, window, None if prefix is None else prefix * B)
    assert torch.equal(out, out[:1].expand_as(out))
    tol = tolerances(ref, D, "fp16", 0.0, slopes)[0] - n * (2.0 ** -25 - 2.0 ** -31) * ref.largest
    if cap:                                                  # 2^-20 of the cap, or 2^-19 of the logit
        tol = tol + 2 * (2.0 ** -20 * cap if cap <= 256 else 2.0 ** -19 * 17.7) * ref.weight
    assert np.all(ref.out > 3 * tol) and np.all(np.abs(out[:1].double().cpu().numpy() - ref.out) <= tol)
