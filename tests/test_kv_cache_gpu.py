"""The NVFP4 key/value cache on the GPU against the oracle: append (rotation,
quantization, placement), gather, attention, and a chain of them.

Attention's tolerance, from the kernels' roundings (h = half a step of the
output type, n = keys of the row, w = sum of p |v|, L = largest sum of |scale q k|):
  * a logit is an fp32 sum of D exact products: off by at most e_s = D * 2^-23 * L,
    and by 2^-22 * L more for the factor 2^x is taken with; p is off by the factor
    exp(e_s), and so is the sum of the p: 2 e_s * w in the output;
  * each p is rounded to 11 bits for the product with v: 2^-11 * w;
  * the fp32 sums over n keys: n * 2^-23 * w, twice (numerator and denominator);
  * the output's rounding: h * |out|.
lse: e_s + n * 2^-23 + 2^-22 * (|lse| + 1).
"""
import math

import numpy as np
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from oracle import kv_cache as okv
from rmsnorm_fp4_quant_gb300 import build as fbuild

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rope_table(n, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * freq
    return torch.cat((a.cos(), a.sin()), -1).float()


def random_cache(pages, heads, page, D, seed):
    """Any bytes: what earlier sequences left behind."""
    g = gen(seed)
    r = lambda *s: torch.randint(0, 256, (pages, heads, *s), dtype=torch.uint8, generator=g)  # noqa: E731
    return [r(page, D // 2), r(page, D // 16), r(page, D // 2), r(D // 16, page)]


def to_np(cache):
    return [t.cpu().numpy().copy() for t in cache]


# ---------------------------------------------------------------------------
# append and gather
# ---------------------------------------------------------------------------
APPEND = [
    # T, Hq, Hkv, D, page, rot, interleaved, dtype
    (1, 12, 2, 128, 16, 128, False, "bf16"),
    (1, 0, 1, 64, 16, 64, False, "fp16"),
    (7, 5, 1, 64, 48, 32, True, "bf16"),
    (41, 40, 8, 128, 16, 64, True, "fp16"),
    (130, 3, 3, 128, 64, 128, True, "bf16"),
    (33, 1, 24, 64, 32, 64, False, "fp16"),
    (65, 0, 7, 128, 16, 0, False, "bf16"),
    (1031, 9, 3, 64, 128, 32, False, "bf16"),
    (515, 14, 2, 128, 48, 96, False, "fp16"),
    (515, 14, 2, 128, 48, 96, True, "bf16"),
]


def append_inputs(T, Hq, Hkv, D, rot, dtype, seed, positions=4096):
    g = gen(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g) * 1.7
    qkv[:, ::29] *= 20
    if T > 3:
        qkv[2] = 0                                   # a token of zeros: scale and codes 0
        qkv[3] *= 1e-4                               # blocks that quantize to nothing
    qkv = qkv.to(DT[dtype])
    pos = torch.randint(0, positions, (T,), generator=g)
    return qkv, pos, rope_table(positions, rot) if rot else None


def split(qkv, Hq, Hkv, D):
    q, k, v = qkv.split((Hq * D, Hkv * D, Hkv * D), -1)
    return (q.unflatten(-1, (Hq, D)) if Hq else None, k.unflatten(-1, (Hkv, D)), v.unflatten(-1, (Hkv, D)))


def f32(t):
    return None if t is None else t.float().numpy()


@pytest.mark.parametrize("T,Hq,Hkv,D,page,rot,inter,dtype", APPEND)
@pytest.mark.parametrize("scales", [None, (2.5, 0.3125)])
def test_append_and_gather(T, Hq, Hkv, D, page, rot, inter, dtype, scales):
    qkv, pos, table = append_inputs(T, Hq, Hkv, D, rot, dtype, seed=T + D)
    pages = T // page + 3
    cache = random_cache(pages, Hkv, page, D, seed=5)
    slots = torch.randperm(pages * page, generator=gen(9))[:T]
    if T > 6:
        slots[1], slots[4], slots[5] = -1, pages * page, -(1 << 40)      # append nothing
        if rot:
            pos[0], pos[6] = -1, 4096                                    # tokens left out
    want = to_np(cache)
    q, k, v = split(qkv, Hq, Hkv, D)
    kg, vg = scales or (1.0, 1.0)
    rq, here = okv.append(want, f32(k), f32(v), slots.numpy(), pos.numpy(),
                          table.numpy() if rot else None, inter, kg, vg, f32(q)) if rot else \
        okv.append(want, f32(k), f32(v), slots.numpy(), k_gs=kg, v_gs=vg, q=f32(q))
    dev = [t.cuda() for t in cache]
    dq, dk, dv = split(qkv.cuda(), Hq, Hkv, D)
    gs = [torch.tensor([s], device="cuda") if scales else None for s in (kg, vg)]
    out_q = torch.full((T, Hq, D), 77.0, dtype=DT[dtype], device="cuda") if Hq else None
    got = fq.kv_append_nvfp4(dev, dk, dv, slots.cuda(), q=dq, positions=pos.cuda() if rot else None,
                             cos_sin=table.cuda() if rot else None, interleaved=inter,
                             k_global_scale=gs[0], v_global_scale=gs[1], out_q=out_q)
    torch.cuda.synchronize()
    for name, a, b in zip(("k_packed", "k_sf", "v_packed", "v_sf"), to_np(dev), want):
        assert np.array_equal(a, b), name
    if Hq:
        exp = torch.from_numpy(rq).to(DT[dtype])
        exp[torch.from_numpy(~here)] = 77.0
        assert torch.equal(got.cpu(), exp)
    # the slots read back: exact without a global scale
    valid = (slots >= 0) & (slots < pages * page)
    ok = slots[valid & torch.from_numpy(here)]
    gk, gv = okv.gather(want, ok.numpy(), kg, vg)
    rk, rv = fq.kv_gather_nvfp4(dev, ok.cuda(), dtype=DT[dtype], k_global_scale=gs[0], v_global_scale=gs[1])
    for a, b in ((rk, gk), (rv, gv)):
        a = a.double().cpu().numpy()
        if scales is None:
            assert np.array_equal(a, b)
        else:      # a division in 32 bits, then one rounding (values below the type's normals: absolute)
            assert np.all(np.abs(a - b) <= (HALF_STEP[dtype] + 2.0 ** -22) * np.abs(b) + 2.0 ** -25)


def test_append_equals_quantize_fp4():
    T, H, D, page = 64, 4, 128, 16
    k = (torch.randn(T, H, D, generator=gen(0)) * 3).bfloat16().cuda()
    v = (torch.randn(T, H, D, generator=gen(1)) * 3).bfloat16().cuda()
    c = fq.kv_cache_nvfp4(T // page, page, H, D)
    fq.kv_append_nvfp4(c, k, v, torch.arange(T, device="cuda"))
    for x, packed, sf in ((k, c.k_packed, c.k_sf), (v, c.v_packed, c.v_sf.transpose(-1, -2))):
        pk, s = fq.quantize_fp4(x.reshape(T * H, D), sf_layout="rowmajor")
        assert torch.equal(packed.transpose(1, 2).reshape(T * H, -1), pk)
        assert torch.equal(sf.transpose(1, 2).reshape(T * H, -1), s)


def test_append_in_place_and_views():
    """q rotated inside the fused projection's output; k and v beside it stay."""
    T, Hq, Hkv, D = 19, 4, 2, 64
    qkv, pos, table = append_inputs(T, Hq, Hkv, D, 64, "bf16", seed=3)
    dev = qkv.cuda()
    q, k, v = split(dev, Hq, Hkv, D)
    c = fq.kv_cache_nvfp4(4, 16, Hkv, D)
    out = fq.kv_append_nvfp4(c, k, v, torch.arange(T, device="cuda"), q=q, positions=pos.cuda(),
                             cos_sin=table.cuda(), out_q=q)
    assert out.data_ptr() == dev.data_ptr()
    want = okv.rotate(f32(split(qkv, Hq, Hkv, D)[0]), pos.numpy(), table.numpy(), False)
    assert torch.equal(q.cpu(), torch.from_numpy(want).bfloat16())
    assert torch.equal(dev[:, Hq * D:].cpu(), qkv[:, Hq * D:])
    with pytest.raises(fq.Fp4Error):           # out_q over k's columns
        fq.kv_append_nvfp4(c, k, v, torch.arange(T, device="cuda"), q=q, positions=pos.cuda(),
                           cos_sin=table.cuda(), out_q=dev[:, D:(Hq + 1) * D].unflatten(-1, (Hq, D)))


def test_gather_leaves_rows_of_slots_outside_and_repeats():
    c = [t.cuda() for t in random_cache(3, 2, 16, 64, seed=1)]
    c[1] &= 0x3F
    c[3] &= 0x3F
    slots = torch.tensor([5, -1, 47, 48, 5, 1 << 50], device="cuda")
    out_k = torch.full((6, 2, 64), 3.0, dtype=torch.float16, device="cuda")
    out_v = torch.full_like(out_k, 4.0)
    fq.kv_gather_nvfp4(c, slots, out_k=out_k, out_v=out_v)
    gk, gv = okv.gather(to_np(c), [5, 47, 5])
    live = torch.tensor([0, 2, 4])
    assert np.array_equal(out_k.cpu()[live].double().numpy(), gk)
    assert np.array_equal(out_v.cpu()[live].double().numpy(), gv)
    dead = torch.tensor([1, 3, 5])
    assert torch.all(out_k.cpu()[dead] == 3) and torch.all(out_v.cpu()[dead] == 4)


def test_append_infinities_and_nan_stay_in_their_blocks():
    T, H, D = 4, 1, 64
    k = torch.ones(T, H, D)
    k[1, 0, 3], k[2, 0, 17], k[3, 0, 40] = float("inf"), float("-inf"), float("nan")
    c = fq.kv_cache_nvfp4(1, 16, H, D)
    fq.kv_append_nvfp4(c, k.bfloat16().cuda(), k.bfloat16().cuda(), torch.arange(T, device="cuda"))
    gk, _ = fq.kv_gather_nvfp4(c, torch.arange(T, device="cuda"))
    gk = gk.float().cpu()
    assert torch.isfinite(gk).all()            # the format has no infinities: they saturate
    one = gk[0, 0, 0]
    for t, blk in ((1, 0), (2, 1), (3, 2)):
        for b in range(4):
            if b != blk:
                assert torch.all(gk[t, 0, 16 * b:16 * b + 16] == one)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def fill_sequences(lens, Hkv, D, page, seed, extra_pages=3, bad=()):
    """A cache of garbage with `lens` tokens written for each sequence by the oracle;
    (cache, tables).  bad: (sequence, page index, number) entries put into the tables
    afterwards."""
    g = gen(seed)
    used = [max(0, -(-n // page)) for n in lens]
    pages = sum(used) + extra_pages
    cache = to_np(random_cache(pages, Hkv, page, D, seed + 1))
    cache[1][:, :, ::3] = 0x7F                       # scales that are no numbers, too
    cache[3][:, :, :, 1::3] = 0xFF
    order = torch.randperm(pages, generator=g).numpy()
    tables = np.full((len(lens), max(used + [1]) + 1), -7, np.int64)
    at = 0
    for b, n in enumerate(lens):
        tables[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        j = np.arange(n)
        slots = tables[b][j // page] * page + j % page if n else j
        k = torch.randn(n, Hkv, D, generator=g).numpy()
        k[..., 3::17] *= 3
        if n:
            okv.append(cache, k, torch.randn(n, Hkv, D, generator=g).numpy(), slots)
    for b, i, number in bad:
        tables[b, i] = number
    return cache, tables


def shape_of(B, T, Hq, Hkv, D, keys):
    return fq.fp4_attention_launch_shape(B, T, Hq, Hkv, D, keys)


def widened(tables, T, Hq, Hkv, D, page, wanted):
    """The tables, widened by pages of no sequence until the call's launch shape is as
    wanted; None if no width does it."""
    B, width = tables.shape
    while width * page < 1 << 22:
        if wanted(shape_of(B, T, Hq, Hkv, D, width * page)):
            wide = np.full((B, width), -7, tables.dtype)
            wide[:, :tables.shape[1]] = tables
            return wide
        width *= 2
    return None


def for_ranges(*args):
    """256-row items whose keys are cut into ranges."""
    return widened(*args, lambda s: s["kernel"] == "kv_prefill_kernel" and s["parts"] > 1)


def for_even_split(*args):
    """The keys of all items split evenly over the CTAs."""
    return widened(*args, lambda s: s == {"kernel": "kv_decode_kernel", "parts": 0})


def times_for_items(B, T, Hq, Hkv, D, keys):
    """How often the batch has to be repeated for a call that takes 256-row items with
    all their keys; None if no number does."""
    n = 1
    while n <= 128:
        if shape_of(n * B, n * T, Hq, Hkv, D, keys) == {"kernel": "kv_prefill_kernel", "parts": 1}:
            return n
        n *= 2
    return None


def check_attention(q, cache, tables, lens, cu, causal, dtype, sm_scale=None, kg=1.0, vg=1.0, **kw):
    """Runs the call and compares every row with the oracle; returns (out, lse).  The same
    rows are run in the other launch shapes, too: over wider tables (an even split of the
    keys, 256-row items with ranges of them) and with the batch repeated (256-row items)."""
    T, Hq, D = q.shape
    B, page, Hkv = len(lens), cache[0].shape[2], cache[0].shape[1]
    scale = D ** -0.5 if sm_scale is None else sm_scale
    ref = okv.attention(q.double().numpy(), cache, tables, lens, cu, causal, scale, kg, vg)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    gs = dict(k_global_scale=torch.tensor([kg], device="cuda") if kg != 1 else None,
              v_global_scale=torch.tensor([vg], device="cuda") if vg != 1 else None)

    def run(q, tables, lens, cu):
        T = q.shape[0]
        out = torch.full((T, Hq, D), 5.0, dtype=DT[dtype], device="cuda")
        lse = torch.full((T, Hq), 6.0, device="cuda")
        fq.attention_nvfp4(q.cuda(), dev, torch.from_numpy(tables.astype(np.int32)).cuda(),
                           torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"),
                           causal=causal, sm_scale=sm_scale, out=out, return_lse=True, lse=lse, **gs, **kw)
        torch.cuda.synchronize()
        return out, lse
    out, lse = run(q, tables, lens, cu)
    compare_attention(out, lse, ref, D, dtype)
    if max(lens) <= tables.shape[1] * page:
        for wide in (for_even_split(tables, T, Hq, Hkv, D, page), for_ranges(tables, T, Hq, Hkv, D, page)):
            if wide is not None and wide.shape != tables.shape:
                compare_attention(*run(q, wide, lens, cu), ref, D, dtype)
    n = times_for_items(B, T, Hq, Hkv, D, tables.shape[1] * page)
    if n is not None and cu is not None:
        first, last = cu[0], cu[-1]
        rows = last - first
        starts = [first + i * rows + c - first for i in range(n) for c in cu[:-1]] + [first + n * rows]
        o, s = run(torch.cat([q[:first], q[first:last].repeat(n, 1, 1), q[last:]]), np.tile(tables, (n, 1)), list(lens) * n,
                   starts)
        for i in (0, n - 1):
            pick = torch.cat([torch.arange(first), first + i * rows + torch.arange(rows),
                              first + n * rows + torch.arange(T - last)]).cuda()
            compare_attention(o[pick], s[pick], ref, D, dtype)
        body = o[first:first + n * rows].view(n, rows, Hq, D)
        assert torch.equal(body, body[:1].expand_as(body))
    return out, lse


def compare_attention(out, lse, ref, D, dtype):
    o, s = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(o[~ref.rows] == 5.0) and np.all(s[~ref.rows] == 6.0)      # rows of no sequence
    o, s = o[ref.rows], s[ref.rows]
    n = ref.keys[ref.rows][:, None]
    e_s = (D * 2.0 ** -23 + 2.0 ** -22) * ref.logit[ref.rows]
    tol = HALF_STEP[dtype] * np.abs(ref.out[ref.rows]) + \
        (2.0 ** -11 + 2 * e_s + n * 2.0 ** -22)[..., None] * ref.weight[ref.rows] + 2.0 ** -24
    err = np.abs(o - ref.out[ref.rows])
    assert np.all(np.isfinite(o))
    assert np.all(err <= tol), (err / tol).max()
    empty = np.broadcast_to(n == 0, s.shape)
    assert np.all(np.isneginf(s[empty])) and np.all(o[empty] == 0)
    want = ref.lse[ref.rows][~empty]
    ltol = (e_s + n * 2.0 ** -23)[~empty] + 2.0 ** -22 * (np.abs(want) + 1)
    assert np.all(np.abs(s[~empty] - want) <= ltol), (np.abs(s[~empty] - want) / ltol).max()


def queries(T, Hq, D, dtype, seed, size=1.5):
    return (torch.randn(T, Hq, D, generator=gen(seed)) * size).to(DT[dtype])


EDGE_LENS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 0, 511, 700]


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [
    (12, 2, 128, 16, "bf16"), (4, 4, 64, 48, "fp16"), (7, 1, 128, 64, "fp16"), (6, 2, 64, 16, "bf16"),
    (8, 1, 128, 32, "bf16"), (10, 1, 64, 128, "fp16"), (17, 1, 128, 16, "bf16"), (40, 8, 128, 48, "fp16"),
    (33, 1, 64, 16, "bf16"),
])
def test_decode_lengths(Hq, Hkv, D, page, dtype):
    cache, tables = fill_sequences(EDGE_LENS, Hkv, D, page, seed=Hq)
    check_attention(queries(len(EDGE_LENS), Hq, D, dtype, 3), cache, tables, EDGE_LENS, None, True, dtype)


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,dtype", [
    ([5000], 4, 1, 128, 16, "bf16"), ([4097, 3, 0, 2050], 12, 2, 64, 64, "fp16"),
    ([9001, 1], 8, 2, 128, 128, "bf16"), ([12345], 1, 1, 64, 48, "fp16"),
])
def test_decode_long(lens, Hq, Hkv, D, page, dtype):
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=2)
    check_attention(queries(len(lens), Hq, D, dtype, 4), cache, tables, lens, None, True, dtype)


def test_decode_many_sequences():
    lens = [(i * 37) % 90 for i in range(700)]
    cache, tables = fill_sequences(lens, 1, 64, 16, seed=2)
    check_attention(queries(700, 2, 64, "bf16", 4), cache, tables, lens, None, True, "bf16")


# (more than 20000 keys in all take the oracle long)
@pytest.mark.parametrize("B,Hkv,longest", [
    (B, Hkv, n) for n in (20, 100, 200, 500, 1000, 2000, 6000)
    for B, Hkv in ((1, 1), (3, 4), (14, 5), (40, 6), (150, 8)) if B * n <= 20000])
def test_decode_items_by_length(B, Hkv, longest):
    lens = [1 + (i * 7919) % longest for i in range(B)]
    lens[B // 2] = longest
    cache, tables = fill_sequences(lens, Hkv, 64, 16, seed=B)
    check_attention(queries(B, Hkv * (2 if B > 3 else 12), 64, "bf16", 4), cache, tables, lens, None, True, "bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("parts", [0, 1, 2, 3, 4, 6, 8])
def test_every_way_to_share_an_item(D, group, parts):
    """One CTA, each size of cluster, the even split: the first sizes that lead to it."""
    B, Hkv, longest = next((B, Hkv, n) for n in (100, 400, 700, 1000, 1500, 2200, 3000, 6000, 12000)
                           for B in (1, 2, 4, 6, 9, 12, 16, 20, 26) for Hkv in (1, 2, 4, 8)
                           if shape_of(B, B, Hkv * group, Hkv, D, n + 32)["parts"] == parts)
    lens = [longest] + [(i * 131) % min(longest, 500) for i in range(1, B)]
    cache, tables = fill_sequences(lens, Hkv, D, 32, seed=parts)
    assert shape_of(B, B, Hkv * group, Hkv, D, 32 * tables.shape[1]) == {"kernel": "kv_decode_kernel", "parts": parts}
    check_attention(queries(B, Hkv * group, D, "fp16", 4), cache, tables, lens, None, True, "fp16")


VARLEN = [
    # lens, q lengths (rows before, between and behind them belong to nobody)
    ([40, 17, 0, 129, 64, 5], [1, 17, 3, 2, 0, 9]),
    ([300], [300]),
    ([301, 129], [129, 129]),
    ([700, 20, 33], [65, 1, 40]),
    ([128], [128]),
    ([1, 1, 1], [1, 5, 1]),
]


@pytest.mark.parametrize("lens,q_lens", VARLEN)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [
    (8, 2, 128, 16, "bf16"), (3, 3, 64, 48, "fp16"), (5, 1, 128, 64, "fp16"), (24, 8, 64, 32, "bf16")])
def test_varlen(lens, q_lens, causal, Hq, Hkv, D, page, dtype):
    cu = np.cumsum([2] + q_lens).tolist()                 # two rows in front of the first sequence
    T = cu[-1] + 3                                        # and three behind the last
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=11)
    check_attention(queries(T, Hq, D, dtype, 6), cache, tables, lens, cu, causal, dtype)


def test_a_mixed_batch_in_one_call_and_in_two():
    """A prompt's piece and single rows together, and apart over their rows of q, out and lse
    and their rows of the tables."""
    lens, q_lens, Hq, Hkv, D, page = [310] + [40 + 7 * i for i in range(9)], [150] + [1] * 9, 8, 2, 64, 16
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=17)
    cu = np.cumsum([0] + q_lens).tolist()
    q = queries(cu[-1], Hq, D, "bf16", 5)
    check_attention(q, cache, tables, lens, cu, True, "bf16")
    dev = [torch.from_numpy(c).cuda() for c in cache]
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qd = q.cuda()
    out = torch.full_like(qd, 5.0)
    lse = torch.full(qd.shape[:2], 6.0, device="cuda")
    fq.attention_nvfp4(qd[:150], dev, tab[:1], sl[:1], torch.tensor([0, 150], dtype=torch.int32, device="cuda"),
                       out=out[:150], return_lse=True, lse=lse[:150])
    fq.attention_nvfp4(qd[150:], dev, tab[1:], sl[1:], out=out[150:], return_lse=True, lse=lse[150:])
    compare_attention(out, lse, okv.attention(q.double().numpy(), cache, tables, lens, cu, True, D ** -0.5), D, "bf16")


# long tables and few rows: each item's keys are cut into ranges that are joined afterwards
@pytest.mark.parametrize("lens,q_lens,causal", [
    ([3000, 1500], [70, 130], True), ([2600], [300], False), ([64, 4200, 3], [64, 129, 200], True),
    ([1, 2100], [90, 40], True),
])
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [
    (4, 1, 128, 16, "bf16"), (3, 1, 64, 48, "fp16"), (2, 2, 128, 128, "fp16"), (6, 2, 64, 64, "bf16")])
def test_many_rows_over_long_sequences(lens, q_lens, causal, Hq, Hkv, D, page, dtype):
    cu = np.cumsum([1] + q_lens).tolist()
    bad = [(0, 3, -1)] if lens[0] > 1000 else [(1, 3, 10 ** 7), (1, 15, -2)]
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=13, bad=bad)
    check_attention(queries(cu[-1] + 2, Hq, D, dtype, 7), cache, tables, lens, cu, causal, dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_of_empty_and_short_sequences(causal, D):
    """Hundreds of rows per sequence, over no keys, fewer keys than rows, one key more than a step."""
    lens, q_lens = [0, 5, 129, 1], [140, 260, 130, 257]
    cu = np.cumsum([0] + q_lens).tolist()
    cache, tables = fill_sequences(lens, 2, D, 16, seed=9)
    check_attention(queries(cu[-1], 4, D, "bf16", 7), cache, tables, lens, cu, causal, "bf16")


@pytest.mark.parametrize("group,q_len", [(1, 63), (1, 64), (1, 65), (3, 21), (3, 22), (64, 1), (80, 1), (9, 7), (128, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_around_the_change_of_kernels(group, q_len, D):
    """Rows per sequence and key/value head on both sides of each choice by their number."""
    lens = [200, 77]
    cache, tables = fill_sequences(lens, 1, D, 16, seed=group)
    cu = [0, q_len, 2 * q_len]
    check_attention(queries(2 * q_len, group, D, "bf16", 3), cache, tables, lens, cu, True, "bf16")


def test_a_reference_that_keeps_moving():
    """Keys whose logits grow along the sequence: the running reference moves in every
    step of every kernel, and everything before it is scaled down."""
    D, page, n = 64, 16, 1200
    cache = to_np(random_cache(n // page, 1, page, D, 3))
    k = np.zeros((n, 1, D), np.float32)
    k[:, 0, 0] = np.linspace(0, 300, n)
    v = torch.randn(n, 1, D, generator=gen(5)).numpy()
    okv.append(cache, k, v, np.arange(n))
    tables = np.arange(n // page, dtype=np.int64)[None]
    for cu, T in ((None, 1), ([0, 100], 100)):
        for sign in (1.0, -1.0):
            q = torch.zeros(T, 2, D)
            q[..., 0] = sign * torch.linspace(1, 9, T)[:, None]
            check_attention(q.bfloat16(), cache, tables, [n], cu, True, "bf16", sm_scale=1.0)


@pytest.mark.parametrize("q_lens", [None, [1, 40, 150]])
@pytest.mark.parametrize("D", [64, 128])
def test_bad_pages_are_masked(q_lens, D):
    lens = [200, 100, 160]
    cache, tables = fill_sequences(lens, 2, D, 16, seed=21,
                                   bad=[(0, 2, -1), (0, 12, 10 ** 6), (2, 0, 2 ** 31 - 1), (2, 9, -2 ** 31)]
                                   + [(1, i, -1) for i in range(7)])        # sequence 1 sees nothing
    cu = None if q_lens is None else np.cumsum([0] + q_lens).tolist()
    T = 3 if cu is None else cu[-1]
    check_attention(queries(T, 4, D, "bf16", 2), cache, tables, lens, cu, True, "bf16")


@pytest.mark.parametrize("varlen", [False, True])
def test_lengths_beyond_the_table_are_clamped(varlen):
    cache, tables = fill_sequences([64, 64], 1, 64, 16, seed=1)
    tables = tables[:, :4]
    cu = [0, 20, 40] if varlen else None
    T = 40 if varlen else 2
    check_attention(queries(T, 4, 64, "fp16", 1), cache, np.ascontiguousarray(tables), [1000, 64], cu, False, "fp16")
    check_attention(queries(T, 4, 64, "fp16", 1), cache, np.ascontiguousarray(tables), [-5, 64], cu, False, "fp16")


@pytest.mark.parametrize("dtype,size", [("bf16", 1e-3), ("bf16", 60.0), ("fp16", 60.0), ("bf16", 1e6), ("fp16", 300.0),
                                        ("bf16", 0.0)])
@pytest.mark.parametrize("varlen", [False, True])
def test_query_sizes(dtype, size, varlen):
    lens = [90, 300]
    cache, tables = fill_sequences(lens, 2, 128, 16, seed=31)
    cu = [0, 30, 170] if varlen else None
    check_attention(queries(170 if varlen else 2, 4, 128, dtype, 8, size), cache, tables, lens, cu, True, dtype)


@pytest.mark.parametrize("varlen", [False, True])
def test_global_scales_and_softmax_scale(varlen):
    lens = [90, 300]
    cache, tables = fill_sequences(lens, 2, 128, 16, seed=31)
    cu = [0, 30, 170] if varlen else None
    check_attention(queries(170 if varlen else 2, 4, 128, "fp16", 8), cache, tables, lens, cu, True, "fp16",
                    sm_scale=0.21, kg=1.75, vg=0.4)


@pytest.mark.parametrize("varlen", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_row_stays_alone(varlen, bad):
    lens = [90, 300]
    cache, tables = fill_sequences(lens, 2, 64, 16, seed=31)
    cu = [0, 30, 170] if varlen else None
    T = 170 if varlen else 2
    if varlen:
        tables = for_ranges(tables, T, 4, 2, 64, 16)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    q = queries(T, 4, 64, "bf16", 8).cuda()
    a = fq.attention_nvfp4(q, dev, tab, sl, cud)
    q2 = q.clone()
    q2[T // 2, 1, 5] = bad
    b = fq.attention_nvfp4(q2, dev, tab, sl, cud)
    same = torch.ones(T, 4, dtype=torch.bool)
    same[T // 2, 1] = False
    assert torch.equal(a.cpu()[same], b.cpu()[same])
    assert torch.isnan(b[T // 2, 1]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 150])
def test_a_row_whose_logits_are_all_minus_infinity(T, D):
    """-inf - -inf: NaN, as from the formula; a row that sees no key is 0 all the same."""
    n = 40
    cache = to_np(random_cache(3, 1, 16, D, 3))
    okv.append(cache, np.ones((n, 1, D), np.float32), torch.randn(n, 1, D, generator=gen(5)).numpy(), np.arange(n))
    tables = np.arange(3, dtype=np.int64)[None]
    cu = None if T == 1 else [0, T]
    for tab in [tables] + ([] if T == 1 else [for_ranges(tables, T, 4, 1, D, 16)]):
        q = queries(T, 4, D, "bf16", 2).cuda()
        q[:, 1] = -float("inf")
        out, lse = fq.attention_nvfp4(q, [torch.from_numpy(c).cuda() for c in cache],
                                      torch.from_numpy(tab.astype(np.int32)).cuda(),
                                      torch.tensor([n], dtype=torch.int32, device="cuda"),
                                      None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                      return_lse=True)
        seen = torch.arange(T) >= T - n
        assert torch.isnan(out.cpu()[seen, 1]).all() and torch.isnan(lse.cpu()[seen, 1]).all()
        assert torch.all(out.cpu()[~seen] == 0) and torch.all(torch.isneginf(lse.cpu()[~seen]))
        keep = [0, 2, 3]
        assert torch.isfinite(out.cpu()[seen][:, keep]).all()


# what one element of channel 0 makes of a logit: queries up to the ends of their types
LOGIT_SIZES = [("bf16", x) for x in (3e4, 1e7, 1e9, 3e13, 1e20, 2e30, 1e33)] + [("fp16", 3e4)]


@pytest.mark.parametrize("dtype,size", LOGIT_SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 150])
@pytest.mark.parametrize("zeros", [False, True])
def test_logits_of_any_size(dtype, size, D, T, zeros):
    """Keys and queries with one channel: a logit is one exact product, so equal keys share
    a row's weight equally and the next smaller logit is more than 1000 below.  Rows of
    either sign; the largest logit is in a first, a middle and the last key; the last row
    of all sees one key of the largest negative logit; with zeros, 100 keys further on have
    logits of 0, which are a negative row's largest.  In every launch shape."""
    n, page = 500, 16
    scale = 1.0 if dtype == "bf16" else 2.0 ** 13
    cache = to_np(random_cache(-(-n // page), 1, page, D, 3))
    k = np.zeros((n, 1, D), np.float32)
    k[:, 0, 0] = np.where(np.arange(n) % 2, 2, 4)        # times +-size: the rows want 4 or 2
    for j in (0, 201, 203, n - 1):
        k[j, 0, 0] = 6 if j != 203 else 1
    if zeros:
        k[300:400] = 0
    v = torch.randn(n, 1, D, generator=gen(5)).numpy()
    okv.append(cache, k, v, np.arange(n))
    values = okv.gather(cache, np.arange(n))[1][:, 0]
    keys = okv.gather(cache, np.arange(n))[0][:, 0, 0]
    q = torch.zeros(T, 4, D, dtype=torch.float64)
    q[:, :, 0] = torch.tensor([1.0, -1.0, 0.25, -0.25]) * size
    q = q.to(DT[dtype])
    slim = np.arange(-(-n // page), dtype=np.int64)[None]
    calls = [(1, t) for t in (slim, for_even_split(slim, T, 4, 1, D, page), for_ranges(slim, T, 4, 1, D, page))]
    calls.append((times_for_items(1, T, 4, 1, D, slim.size * page) or 1, slim))
    dev = [torch.from_numpy(c).cuda() for c in cache]
    for seen_last in (n, 1):
        for copies, tables in calls:
            if tables is None:
                continue
            i32 = dict(dtype=torch.int32, device="cuda")
            out, lse = fq.attention_nvfp4(q.repeat(copies, 1, 1).cuda(), dev,
                                          torch.from_numpy(np.tile(tables, (copies, 1))).to(**i32),
                                          torch.tensor([seen_last] * copies, **i32),
                                          None if T == 1 else torch.arange(0, copies * T + 1, T, **i32),
                                          sm_scale=scale, return_lse=True)
            out, lse = out.double().cpu().numpy()[-T:], lse.double().cpu().numpy()[-T:]
            for t in range(T):
                seen = seen_last - T + t + 1
                for h in range(4):
                    if seen <= 0:
                        assert np.all(out[t, h] == 0) and np.isneginf(lse[t, h])
                        continue
                    x = scale * float(q[t, h, 0]) * keys[:seen]
                    best = x == x.max()
                    assert np.max(x[~best], initial=-np.inf) < x.max() - 1000
                    want = values[:seen][best].mean(0)
                    # equal weights 1 / m in 11 bits and their fp32 sum, then the output's rounding
                    tol = HALF_STEP[dtype] * np.abs(want) + \
                        (2.0 ** -11 + best.sum() * 2.0 ** -22) * np.abs(values[:seen][best]).mean(0) + 2.0 ** -24
                    assert np.all(np.abs(out[t, h] - want) <= tol), (t, h, seen_last)
                    want = x.max() + np.log(best.sum())
                    # 8 roundings of 2^-24: the factor's three, the product, the reference, the sum
                    # with the logarithm, and the factor back
                    assert abs(lse[t, h] - want) <= 2.0 ** -21 * (abs(want) + 1), (t, h, seen_last)


@pytest.mark.parametrize("varlen", [False, True])
def test_strided_queries_graphs_streams_and_repeats(varlen):
    """A column slice of a wider matrix as q; the same bits on repeats, on another
    stream and from a captured graph, which follows the lengths; two graphs."""
    lens = [90, 300, 40]
    Hq, D = 4, 128
    cache, tables = fill_sequences(lens, 2, D, 16, seed=31)
    cu = [0, 30, 170, 180] if varlen else None
    T = 180 if varlen else 3
    if varlen:
        tables = for_ranges(tables, T, Hq, 2, D, 16)
    wide = torch.randn(T, (Hq + 3) * D, generator=gen(0)).bfloat16().cuda()
    q = wide[:, D:(Hq + 1) * D].unflatten(-1, (Hq, D))
    dev = [torch.from_numpy(c).cuda() for c in cache]
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")

    def call(**kw):
        return fq.attention_nvfp4(q, dev, tab, sl, cud, return_lse=True, **kw)
    a, la = call()
    assert torch.equal(a, fq.attention_nvfp4(q.contiguous(), dev, tab, sl, cud))
    for _ in range(3):
        b, lb = call()
        assert torch.equal(a, b) and torch.equal(la, lb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, lb = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b) and torch.equal(la, lb)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1, l1 = call()
    with torch.cuda.graph(g2):
        o2, l2 = call()
    for t in (o1, l1, o2, l2):
        t.fill_(9)
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, a) and torch.equal(o2, a) and torch.equal(l1, la) and torch.equal(l2, la)
    sl.copy_(torch.tensor([10, 299, 0], dtype=torch.int32))
    g1.replay()
    torch.cuda.synchronize()
    c, lc = call()
    assert torch.equal(o1, c) and torch.equal(l1, lc)
    assert not torch.equal(c, a)


def test_offsets_beyond_32_bits():
    """Pages behind 4 GiB of codes."""
    pages, Hkv, page, D = 70000, 8, 128, 128
    kp = torch.empty(pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
    assert kp.numel() > 1 << 32
    vp = torch.empty_like(kp)
    ks = torch.empty(pages, Hkv, page, D // 16, dtype=torch.uint8, device="cuda")
    vs = torch.empty(pages, Hkv, D // 16, page, dtype=torch.uint8, device="cuda")
    c = (kp, ks, vp, vs)
    T = 300
    k, v = torch.randn(2, T, Hkv, D, generator=gen(0)).bfloat16().cuda()
    tab = torch.tensor([[69999, 3, 68001]], dtype=torch.int32, device="cuda")
    j = torch.arange(T, device="cuda")
    slots = tab[0].long()[j // page] * page + j % page
    fq.kv_append_nvfp4(c, k, v, slots)
    small = fq.kv_cache_nvfp4(3, page, Hkv, D)
    fq.kv_append_nvfp4(small, k, v, j)
    for a, b in zip(fq.kv_gather_nvfp4(c, slots), fq.kv_gather_nvfp4(small, j)):
        assert torch.equal(a, b)
    sl = torch.tensor([T], dtype=torch.int32, device="cuda")
    tab2 = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    q = queries(200, 16, D, "bf16", 1).cuda()
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    assert torch.equal(fq.attention_nvfp4(q, c, tab, sl, cu), fq.attention_nvfp4(q, small, tab2, sl, cu))
    assert torch.equal(fq.attention_nvfp4(q[:1], c, tab, sl), fq.attention_nvfp4(q[:1], small, tab2, sl))


# ---------------------------------------------------------------------------
# every key counts: equal weights
# ---------------------------------------------------------------------------
def equal_cache(lens, Hkv, D, page, seed):
    """Values of +-6 at random (one code, scale 1), keys of any finite bytes, garbage behind
    the ends; (cache, tables, running sums of the signs per sequence: [n + 1, Hkv, D])."""
    rng = np.random.default_rng(seed)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 2
    bits = lambda *s: rng.integers(0, 256, (pages, Hkv, *s), dtype=np.uint8)  # noqa: E731
    cache = [bits(page, D // 2), bits(page, D // 16) & 0x77, bits(page, D // 2), np.full((pages, Hkv, D // 16, page), 0xFF, np.uint8)]
    order = rng.permutation(pages)
    tables = np.full((len(lens), max(used + [1])), -1, np.int64)
    sums, at = [], 0
    for b, n in enumerate(lens):
        tables[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        minus = rng.integers(0, 2, (n, Hkv, D), dtype=np.uint8)
        code = 7 + 8 * minus
        pg, i = tables[b][np.arange(n) // page], np.arange(n) % page
        cache[2][pg, :, i] = code[..., 0::2] | code[..., 1::2] << 4
        cache[3][pg, :, :, i] = 0x38
        if n % page:                                        # keys behind the end: scales that are no numbers
            cache[1][tables[b, used[b] - 1], :, n % page:] = 0x7F
        sums.append(np.concatenate([np.zeros((1, Hkv, D), np.int32), (1 - 2 * minus.astype(np.int32)).cumsum(0, dtype=np.int32)]))
    return cache, tables, sums


def check_equal(lens, q_lens, causal, Hq, Hkv, D, page, shape, seed):
    """Queries of 0: every logit is 0 and every weight 2^6, exact in 16 bits as in the sums,
    which stay below 2^24.  So lse is log(n) but for log2, a sum and a product in 32 bits, and
    out the mean of the values but for a reciprocal, a product and its rounding: one key lost
    or taken twice moves all channels of a row by more."""
    cache, tables, sums = equal_cache(lens, Hkv, D, page, seed)
    cu = None if q_lens is None else np.cumsum([0] + q_lens)
    T = len(lens) if cu is None else int(cu[-1])
    tables = widened(tables, T, Hq, Hkv, D, page, shape)
    out, lse = fq.attention_nvfp4(torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda"),
                                  [torch.from_numpy(c).cuda() for c in cache],
                                  torch.from_numpy(tables.astype(np.int32)).cuda(),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  None if cu is None else torch.from_numpy(cu.astype(np.int32)).cuda(),
                                  causal=causal, return_lse=True)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        rows = np.arange(b, b + 1) if cu is None else np.arange(cu[b], cu[b + 1])
        seen = np.clip(n - len(rows) + 1 + np.arange(len(rows)), 0, n) if causal else np.full(len(rows), n)
        some = seen > 0
        assert np.all(out[rows[~some]] == 0) and np.all(np.isneginf(lse[rows[~some]]))
        rows, seen = rows[some], seen[some].astype(np.float64)
        want = np.repeat(6 * sums[b][seen.astype(int)] / seen[:, None, None], Hq // Hkv, 1)
        # the rounding to 16 bits (below its normals: absolute) and two of 2^-24, doubled
        tol = (2.0 ** -11 + 2.0 ** -22) * np.abs(want) + 2.0 ** -25
        assert np.all(np.abs(out[rows] - want) <= tol), b
        assert np.all(tol < 0.5 * (6 - np.abs(want)) / seen[:, None, None], where=np.abs(want) < 5.9)
        # log2 of 64 n: a unit (2^-19 up to 32), the sum with the reference half of one, the product
        ltol = 1.5 * 2.0 ** -19 + 2.0 ** -23 * np.log(seen)
        assert np.all(np.abs(lse[rows] - np.log(seen)[:, None]) <= ltol[:, None]), b
        assert np.all(ltol < 0.5 * np.log1p(1 / seen))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("parts", [0, 1, 2, 3, 4, 6, 8])
def test_every_key_counts_once_in_each_share(D, group, parts):
    """Lengths around the edges of tiles, units and shares, for every way to share an item."""
    B, Hkv, longest = next((B, Hkv, n) for n in (400, 700, 1000, 1500, 2200, 3000, 6000, 12000)
                           for B in (1, 2, 4, 6, 9, 12, 16, 20, 26) for Hkv in (1, 2, 4, 8)
                           if shape_of(B, B, Hkv * group, Hkv, D, n)["parts"] == parts)
    for shift in (0, 1, 63):
        less = [0, 1, 15, 16, 17, 31, 33, 47, 63, 64, 65, 79, 127, 128, 129, 191, 193, 255, 256, 257, 300, 320, 350, 399]
        lens = [max(0, longest - shift - x) for x in less][:B] + [longest // 2] * (B - len(less))
        check_equal(lens, None, True, Hkv * group, Hkv, D, 16, lambda s: s["parts"] == parts, seed=shift)


@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([40001], 4, 1, 128, 16), ([12345], 12, 1, 64, 48), ([5000, 9001, 3, 0, 20050], 12, 2, 64, 64),
    ([30000 - 13 * i for i in range(7)], 3, 3, 128, 128), ([17 * i for i in range(400)], 2, 1, 64, 16),
])
def test_every_key_counts_once_in_the_even_split(lens, Hq, Hkv, D, page):
    check_equal(lens, None, True, Hq, Hkv, D, page, lambda s: s == {"kernel": "kv_decode_kernel", "parts": 0}, seed=1)


@pytest.mark.parametrize("lens,q_lens,Hq,Hkv,D,page,ranges", [
    ([5000, 2049, 127], [300, 129, 300], 4, 1, 128, 16, True), ([12801], [257], 3, 1, 64, 48, True),
    ([4096, 4095, 4097, 128], [128, 129, 127, 200], 6, 2, 128, 128, True),
    ([1024, 1023, 1025, 1000], [600, 513, 1025, 64], 48, 24, 64, 16, False),
    ([2000, 1921], [700, 650], 48, 12, 128, 64, False),
])
@pytest.mark.parametrize("causal", [True, False])
def test_every_key_counts_once_for_many_rows(lens, q_lens, Hq, Hkv, D, page, ranges, causal):
    check_equal(lens, q_lens, causal, Hq, Hkv, D, page,
                lambda s: s["kernel"] == "kv_prefill_kernel" and (s["parts"] > 1) == ranges, seed=2)


# ---------------------------------------------------------------------------
# together, as a serving step uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 3)])
def test_prefill_then_decode_steps(pdl, D, Hq, Hkv):
    """A prompt, then single tokens: append, attention, the output quantized for the
    next product and multiplied; every attention row against the oracle on the oracle's
    own cache bytes, which the GPU's equal."""
    dtype, page, prompt, steps, B = "bf16", 16, 37, 5, 2
    pages = 16
    table = rope_table(256, D)
    dev = fq.kv_cache_nvfp4(pages, page, Hkv, D)
    ref = to_np(dev)
    tables = np.arange(pages, dtype=np.int64)[::-1].reshape(B, -1).copy()
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    g = gen(77)
    wmat = torch.randn(64, Hq * D, generator=g).bfloat16().cuda()
    wp, wsf = fq.quantize_fp4(wmat)
    lens = [0] * B
    for step in range(1 + steps):
        new = [prompt, prompt - 9] if step == 0 else [1] * B
        cu = np.cumsum([0] + new)
        T = int(cu[-1])
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).bfloat16()
        pos = torch.cat([torch.arange(lens[b], lens[b] + new[b]) for b in range(B)])
        slots = torch.cat([torch.from_numpy(tables[b])[torch.arange(lens[b], lens[b] + new[b]) // page] * page
                           + torch.arange(lens[b], lens[b] + new[b]) % page for b in range(B)])
        q, k, v = split(qkv, Hq, Hkv, D)
        rq, _ = okv.append(ref, f32(k), f32(v), slots.numpy(), pos.numpy(), table.numpy(), False, q=f32(q))
        lens = [lens[b] + new[b] for b in range(B)]
        dq, dk, dv = split(qkv.cuda(), Hq, Hkv, D)
        oq = fq.kv_append_nvfp4(dev, dk, dv, slots.cuda(), q=dq, positions=pos.cuda(), cos_sin=table.cuda(), pdl=pdl)
        out, lse = fq.attention_nvfp4(oq, dev, tab, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                      None if step else torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                      return_lse=True, pdl=pdl)
        pk, sf = fq.quantize_fp4(out.reshape(T, Hq * D), pdl=pdl)
        y = fq.gemm_nvfp4_bf16(pk, wp, sf, wsf, pdl=pdl)
        torch.cuda.synchronize()
        for a, b in zip(to_np(dev), ref):
            assert np.array_equal(a, b)
        q16 = torch.from_numpy(rq).bfloat16()
        assert torch.equal(oq.cpu(), q16)
        r = okv.attention(q16.double().numpy(), ref, tables, lens, cu, True, D ** -0.5)
        compare_attention(out, lse, r, D, dtype)
        a = fq.dequant(pk, sf, T, Hq * D, sf_layout="swizzled").double()
        b = fq.dequant(wp, wsf, 64, Hq * D, sf_layout="swizzled").double()
        exact = a @ b.T
        bound = a.abs() @ b.abs().T
        assert torch.all((y.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + 2.0 ** -22 * Hq * D * bound)


def test_cross_attention_to_encoder_states():
    """Keys and values of an encoder appended without rotation; every decoder row sees all of them."""
    Hq, Hkv, D, page = 6, 6, 64, 16
    enc = [50, 77]
    cache, tables = fill_sequences(enc, Hkv, D, page, seed=5)
    check_attention(queries(9, Hq, D, "fp16", 5), cache, tables, enc, [0, 5, 9], False, "fp16")


def test_status_word_is_left_alone():
    cache, tables = fill_sequences([90, 300], 2, 128, 16, seed=31)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu, T in ((None, 2), ([0, 30, 170], 170)):
        check_attention(queries(T, 4, 128, "bf16", 8), cache, tables, [90, 300], cu, True, "bf16", status=status)
        assert fq.read_device_status(status) == fq.FP4_OK


def test_one_workspace_for_calls_in_a_row():
    """A workspace of the caller's, any contents, used by calls one after the other, each
    launched beside the tail of the one before it."""
    D, Hq, Hkv = 128, 8, 2
    lens = [2000, 300]
    cache, tables = fill_sequences(lens, Hkv, D, 16, seed=3)
    tables = for_ranges(tables, 120, Hq, Hkv, D, 16)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40, 120], dtype=torch.int32, device="cuda")
    keys = tab.shape[1] * 16
    need = max(fq.fp4_attention_workspace_bytes(2, T, Hq, Hkv, D, keys) for T in (2, 120))
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    qs = [queries(2 if i % 2 else 120, Hq, D, "bf16", i).cuda() for i in range(6)]
    torch.cuda.synchronize()
    got = [fq.attention_nvfp4(q, dev, tab, sl, None if q.shape[0] == 2 else cu, workspace=ws, pdl=True) for q in qs]
    want = [fq.attention_nvfp4(q, dev, tab, sl, None if q.shape[0] == 2 else cu) for q in qs]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with pytest.raises(fq.Fp4Error):
        fq.attention_nvfp4(qs[0], dev, tab, sl, cu, workspace=ws[:16])


def test_without_the_private_calls_of_torch(monkeypatch):
    """The short cuts to the allocator and the current stream have a public way beside them."""
    cache, tables = fill_sequences([300], 1, 64, 16, seed=3)
    tables = for_even_split(tables, 1, 4, 1, 64, 16)
    dev = [torch.from_numpy(c).cuda() for c in cache]
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    assert fq.fp4_attention_workspace_bytes(1, 1, 4, 1, 64, tab.shape[1] * 16) > 0
    sl = torch.tensor([300], dtype=torch.int32, device="cuda")
    q = queries(1, 4, 64, "bf16", 1).cuda()
    want = fq.attention_nvfp4(q, dev, tab, sl)
    for name in ("_cuda_cudaCachingAllocator_raw_alloc", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.default_stream())
    got = [fq.attention_nvfp4(q, dev, tab, sl), fq.attention_nvfp4(q, dev, tab, sl, stream=side)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)


def test_one_workspace_of_the_largest_size():
    """A workspace for the largest call takes the smaller ones that need more than it."""
    D, Hq, Hkv, page = 64, 8, 1, 16
    lens = [2000]
    cache, tables = fill_sequences(lens, Hkv, D, page, seed=3)
    wide = np.full((1, 2048), -7, tables.dtype)
    wide[:, :tables.shape[1]] = tables
    dev = [torch.from_numpy(c).cuda() for c in cache]
    tab = torch.from_numpy(wide.astype(np.int32)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    size = [fq.fp4_attention_workspace_bytes(1, T, Hq, Hkv, D, 2048 * page) for T in (20000, 300, 1)]
    assert size[0] < size[1]
    ws = torch.full((fq.fp4_attention_workspace_bound(1, 20000, Hq, Hkv, D, 2048 * page),), 255, dtype=torch.uint8,
                    device="cuda")
    for T in (20000, 300, 1):
        q = queries(T, Hq, D, "bf16", T).cuda()
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        got = fq.attention_nvfp4(q, dev, tab, sl, cu, workspace=ws, causal=False)
        assert torch.equal(got, fq.attention_nvfp4(q, dev, tab, sl, cu, causal=False))


def test_tensor_calls_refuse_what_they_cannot_take():
    T, Hq, Hkv, D = 3, 4, 2, 64
    c = fq.kv_cache_nvfp4(4, 16, Hkv, D)
    k = torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(T, device="cuda")
    tab = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    sl = torch.ones(T, dtype=torch.int32, device="cuda")
    cs = torch.zeros(8, 64, device="cuda")
    for bad in [dict(k=k.half()), dict(k=k[:2]), dict(slots=slots.int()), dict(slots=slots[:2]), dict(q=q.float()),
                dict(k=k[:1].expand(T, Hkv, D)), dict(k=k.transpose(1, 2)), dict(cos_sin=cs), dict(positions=slots),
                dict(cos_sin=cs.double(), positions=slots), dict(cos_sin=cs, positions=slots.int()),
                dict(out_q=q), dict(q=q, out_q=q[:2]), dict(slots=slots.cpu()), dict(k=k.cpu()),
                dict(cache=c[:3]), dict(cache=(c[0], c[1], c[2], c[3].transpose(2, 3))), dict(v=k.float())]:
        a = dict(cache=c, k=k, v=k.clone(), slots=slots)
        a.update(bad)
        with pytest.raises(ValueError):
            fq.kv_append_nvfp4(a.pop("cache"), a.pop("k"), a.pop("v"), a.pop("slots"), **a)
    with pytest.raises(fq.Fp4Error):                      # rotated channels in multiples of 32
        fq.kv_append_nvfp4(c, k, k.clone(), slots, positions=slots, cos_sin=torch.zeros(8, 16, device="cuda"))
    for bad in [dict(q=q[0]), dict(q=q[:, :3]), dict(q=q.float()), dict(block_tables=tab.long()), dict(block_tables=tab[:2]),
                dict(seq_lens=sl.long()), dict(seq_lens=sl[:2]), dict(cu_seqlens_q=sl), dict(out=q.half()),
                dict(lse=torch.zeros(T, Hq, dtype=torch.float64, device="cuda")), dict(q=q[:2]), dict(seq_lens=sl.cpu()),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(block_tables=tab[0]),
                dict(k_global_scale=torch.ones(1)), dict(v_global_scale=torch.ones(2, device="cuda"))]:
        a = dict(q=q, cache=c, block_tables=tab, seq_lens=sl)
        a.update(bad)
        with pytest.raises(ValueError):
            fq.attention_nvfp4(a.pop("q"), a.pop("cache"), a.pop("block_tables"), a.pop("seq_lens"), **a)
    with pytest.raises(fq.Fp4Error):
        fq.attention_nvfp4(q, c, tab, sl, sm_scale=0.0)
    # nothing to do: no rows, no sequences, no pages
    e = torch.empty(0, Hq, D, dtype=torch.bfloat16, device="cuda")
    assert fq.attention_nvfp4(e, c, tab[:0], sl[:0]).shape == e.shape
    assert fq.kv_append_nvfp4(c, k[:0], k[:0].clone(), slots[:0]) is None
    out, lse = fq.attention_nvfp4(q, c, torch.empty(T, 0, dtype=torch.int32, device="cuda"), sl, return_lse=True)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_tensor_calls_refuse_too_few_dimensions():
    c = fq.kv_cache_nvfp4(4, 16, 2, 64)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")
    one = torch.zeros((), dtype=torch.bfloat16, device="cuda")
    for a in (one, k[0], k[None]):
        with pytest.raises(ValueError):
            fq.kv_append_nvfp4(c, a, a.clone(), slots)
        with pytest.raises(ValueError):
            fq.kv_append_nvfp4(c, k, k.clone(), slots, q=a)
        with pytest.raises(ValueError):
            fq.attention_nvfp4(a, c, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), slots.int())
    with pytest.raises(ValueError):
        fq.kv_append_nvfp4(c, k, k[0], slots)
    for s in (slots[0], slots[None]):
        with pytest.raises(ValueError):
            fq.kv_gather_nvfp4(c, s)
        with pytest.raises(ValueError):
            fq.kv_append_nvfp4(c, k, k.clone(), s)


def test_waits_that_run_out_are_reported():
    """The debug build with waits cut to a microsecond: rows are NaN or right, the status
    word says so, and the next call is as ever."""
    fbuild.build(debug=True)
    L = fq.debug_lib()
    lens, cu, D, Hq = [900, 2500], [0, 200, 290], 128, 4
    cache, tables = fill_sequences(lens, 1, D, 16, seed=4)
    q = queries(290, Hq, D, "bf16", 2)
    ref = okv.attention(q.double().numpy(), cache, tables, lens, cu, True, D ** -0.5)
    tables = for_ranges(tables, 290, Hq, 1, D, 16)       # the kernel that waits
    dev = [torch.from_numpy(c).cuda() for c in cache]
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd = q.cuda()

    def call():
        out, lse = fq.attention_nvfp4(qd, dev, tab, sl, cud, return_lse=True, status=status)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.cpu().numpy()
    try:
        with fq.using_library(L):
            for limit in (500, 3000, 20000):
                assert L.fp4_debug_configure(limit, 0, 0, -1, -1, None) == 0
                status.zero_()
                out, lse = call()
                nan = np.isnan(out).any(-1)
                assert nan.any() == (fq.read_device_status(status) == fq.FP4_ERR_TIMEOUT)
                assert np.array_equal(nan, np.isnan(lse))
                assert np.all(np.abs(out - ref.out)[~nan] <= 0.02)
                if limit == 500:
                    assert nan.any()
            assert L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, None) == 0
            status.zero_()
            out, lse = call()
            assert fq.read_device_status(status) == fq.FP4_OK
            assert np.all(np.abs(out - ref.out) <= 0.02)
    finally:
        L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, None)


def test_debug_build_finds_no_access_out_of_bounds():
    fbuild.build(debug=True)
    L = fq.debug_lib()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, bad.data_ptr()) == 0
    try:
        with fq.using_library(L):
            for args in APPEND[:8]:
                test_append_and_gather(*args, None)
            test_decode_lengths(12, 2, 128, 48, "bf16")
            test_decode_lengths(4, 4, 64, 16, "fp16")
            test_decode_long([4097, 3, 0, 2050], 12, 2, 64, 64, "fp16")
            for lens, q_lens in VARLEN:
                test_varlen(lens, q_lens, True, 8, 2, 128, 16, "bf16")
                test_varlen(lens, q_lens, False, 3, 3, 64, 48, "fp16")
            test_bad_pages_are_masked([1, 40, 150], 128)
            test_many_rows_over_long_sequences([3000, 1500], [70, 130], True, 4, 1, 128, 16, "bf16")
            test_rows_around_the_change_of_kernels(9, 7, 64)
            # row limits that do not ascend, or lie outside, are held to the rows there are
            c, tables = fill_sequences([100, 50, 70], 1, 64, 16, seed=1)
            c = [torch.from_numpy(x).cuda() for x in c]
            sl = torch.tensor([100, 50, 70], dtype=torch.int32, device="cuda")
            more = for_ranges(tables, 95, 4, 1, 64, 16)
            for cu in ([0, 90, 20, 1000], [-5, 3, 2 ** 31 - 1, 7], [40, 30, 20, 10]):
                for T, tab in ((12, tables), (95, tables), (95, more)):
                    fq.attention_nvfp4(queries(T, 4, 64, "fp16", 1).cuda(), c,
                                       torch.from_numpy(tab.astype(np.int32)).cuda(), sl,
                                       torch.tensor(cu, dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()
            assert bad.item() == 0
            # with every extent one byte shorter the checks see the last accesses
            assert L.fp4_debug_configure(2_000_000_000, 1, 0, -1, -1, bad.data_ptr()) == 0
            c = fq.kv_cache_nvfp4(1, 16, 1, 64)
            k = torch.zeros(16, 1, 64, dtype=torch.bfloat16, device="cuda")
            slots = torch.arange(16, device="cuda")
            fq.kv_append_nvfp4(c, k, k, slots)
            torch.cuda.synchronize()
            n1 = bad.item()
            assert n1 > 0
            fq.kv_gather_nvfp4(c, slots)
            torch.cuda.synchronize()
            assert bad.item() > n1
    finally:
        L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, None)


def test_debug_build_checks_every_attention_kernel():
    """One CTA or cluster an item, the even split, 256-row items, ranges of keys: no access
    out of bounds, and with every extent one byte shorter the last accesses are seen (the
    lengths, the tables, queries, cache, outputs and workspace end where the call says)."""
    fbuild.build(debug=True)
    L = fq.debug_lib()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    D, page, lens = 64, 16, [300, 40, 170]
    few, many = 4, 256                                   # rows of a key/value head
    cache, tables = fill_sequences(lens, 1, D, page, seed=1)
    n = times_for_items(3, 3, many, 1, D, tables.shape[1] * page)
    calls = [(few, tables, 1), (few, for_even_split(tables, 3, few, 1, D, page), 1),
             (many, tables, n), (many, for_ranges(tables, 3, many, 1, D, page), 1)]
    assert shape_of(3, 3, few, 1, D, tables.shape[1] * page)["parts"] > 0
    dev = [torch.from_numpy(x).cuda() for x in cache]
    try:
        with fq.using_library(L):
            for shrink in (0, 1):
                for Hq, tab, copies in calls:
                    assert L.fp4_debug_configure(2_000_000_000, shrink, 0, -1, -1, bad.data_ptr()) == 0
                    before = bad.item()
                    fq.attention_nvfp4(queries(3 * copies, Hq, D, "bf16", 2).cuda(), dev,
                                       torch.from_numpy(np.tile(tab, (copies, 1)).astype(np.int32)).cuda(),
                                       torch.tensor(lens * copies, dtype=torch.int32, device="cuda"), return_lse=True)
                    torch.cuda.synchronize()
                    assert (bad.item() > before) == bool(shrink), (Hq, copies, tab.shape)
    finally:
        L.fp4_debug_configure(2_000_000_000, 0, 0, -1, -1, None)
