"""Host-side refusals of the key/value cache entry points (no GPU): every call
below fails its checks before anything is launched or read."""
import ctypes

import pytest

import rmsnorm_fp4_quant_gb300 as fq
from rmsnorm_fp4_quant_gb300 import build as fbuild

A = 0x7F0000000000


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    return fq.lib()


def at(i):
    return A + (i << 34)


def cache(**kw):
    d = dict(k_packed=at(0), k_sf=at(1), v_packed=at(2), v_sf=at(3), k_global_scale=None,
             v_global_scale=None, num_pages=64, page_size=16, num_kv_heads=2, head_dim=128)
    d.update(kw)
    return fq.KVCacheStruct(**d)


CACHE_REFUSALS = [
    (dict(k_packed=0), 1), (dict(k_sf=0), 1), (dict(v_packed=0), 1), (dict(v_sf=0), 1),
    (dict(num_pages=-1), 1), (dict(page_size=0), 1), (dict(num_kv_heads=0), 1),
    (dict(head_dim=96), 2), (dict(head_dim=32), 2), (dict(page_size=24), 2), (dict(head_dim=0), 1),
    (dict(num_pages=1 << 31), 2), (dict(num_kv_heads=5000), 2), (dict(num_pages=1 << 27), 2),
    (dict(k_packed=at(0) + 8), 3), (dict(v_sf=at(3) + 4), 3), (dict(k_global_scale=at(9) + 2), 3),
]


def append(c=None, **kw):
    a = dict(q=at(4), qs=0, oq=at(5), oqs=0, k=at(6), ks=0, v=at(7), vs=0, pos=at(8), cs=at(9),
             maxp=1024, rot=128, inter=0, slots=at(10), T=5, Hq=4, dt=0)
    a.update(kw)
    return fq.fp4_kv_append_nvfp4(a["q"], a["qs"], a["oq"], a["oqs"], a["k"], a["ks"], a["v"],
                                  a["vs"], a["pos"], a["cs"], a["maxp"], a["rot"], a["inter"],
                                  a["slots"], a["T"], a["Hq"], a["dt"], c or cache(), 0, 0)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_append_refuses_bad_caches(kw, status):
    assert append(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), 1), (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(inter=2), 1), (dict(rot=-32), 1),
    (dict(maxp=-1), 1), (dict(rot=48), 2), (dict(rot=160), 2), (dict(Hq=5000), 2), (dict(T=1 << 31), 2),
    (dict(q=0), 1), (dict(oq=0), 1), (dict(q=0, oq=0), 1), (dict(Hq=0), 1),
    (dict(k=0), 1), (dict(v=0), 1), (dict(slots=0), 1), (dict(pos=0), 1), (dict(cs=0), 1),
    (dict(qs=500), 1), (dict(ks=250), 1), (dict(vs=128), 1), (dict(oqs=256), 1),
    (dict(q=at(4) + 16), 3), (dict(k=at(6) + 2), 3), (dict(v=at(7) + 8), 3), (dict(oq=at(5) + 4), 3),
    (dict(qs=520), 3), (dict(ks=264), 3), (dict(slots=at(10) + 4), 3), (dict(pos=at(8) + 4), 3),
    (dict(cs=at(9) + 8), 3),
    (dict(oq=at(4) + 64), 1),                        # out_q shifted against q
    (dict(oq=at(4), oqs=528), 1),                    # q itself with another stride
    (dict(oq=at(6)), 1),                             # out_q over k
    (dict(oq=at(0) + 4096), 1),                      # out_q inside the cache
    (dict(k=at(2) + 32), 1),                         # k inside the cache
    (dict(slots=at(1) + 64), 1), (dict(pos=at(3) + 8), 1), (dict(cs=at(0)), 1),
    (dict(oq=at(10)), 1),
    (dict(q=at(6) + 256, qs=768, oq=at(6) + 256, oqs=768, k=at(6), ks=768), 1),   # columns shared
    (dict(T=0, q=0, oq=0, Hq=0, k=0, v=0, slots=0), 0),
])
def test_append_refusals(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(maxp=1 << 60), dict(maxp=(1 << 63) - 1), dict(ks=1 << 61), dict(vs=1 << 61), dict(qs=1 << 61),
    dict(oqs=1 << 61), dict(ks=(1 << 63) - 16)])
def test_append_refuses_extents_beyond_64_bits(kw):
    """Whose overlaps could not be told."""
    assert append(**kw) == 2
    assert append(oq=at(8) + 64, maxp=1 << 60) == 2


def test_append_refuses_shared_cache_buffers():
    assert append(cache(v_packed=at(0) + 64)) == 1
    assert append(cache(k_sf=at(2))) == 1


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_gather_refuses_bad_caches(kw, status):
    assert fq.fp4_kv_gather_nvfp4(cache(**kw), at(10), 5, 0, at(4), at(5), 0, 0) == status


@pytest.mark.parametrize("args,status", [
    ((at(10), -1, 0, at(4), at(5)), 1), ((at(10), 5, 2, at(4), at(5)), 1), ((0, 5, 0, at(4), at(5)), 1),
    ((at(10) + 4, 5, 0, at(4), at(5)), 3), ((at(10), 5, 0, at(4) + 16, at(5)), 3),
    ((at(10), 5, 0, at(4), at(4) + 32), 1), ((at(10), 5, 0, at(2), at(5)), 1),
    ((at(10), 5, 0, at(4), at(10)), 1), ((at(10), 1 << 31, 0, at(4), at(5)), 2),
    ((0, 0, 0, 0, 0), 0), ((at(10), 5, 0, 0, 0), 0),
])
def test_gather_refusals(args, status):
    assert fq.fp4_kv_gather_nvfp4(cache(), *args, 0, 0) == status


def attention(c=None, **kw):
    a = dict(q=at(4), qs=0, tab=at(6), pages=8, lens=at(7), cu=0, B=5, T=5, Hq=4, dt=0, scale=0.1,
             causal=1, out=at(5), lse=at(8), ws=at(11), wsb=1 << 33, st=0)
    a.update(kw)
    return fq.fp4_attention_nvfp4(a["q"], a["qs"], c or cache(), a["tab"], a["pages"], a["lens"],
                                  a["cu"], a["B"], a["T"], a["Hq"], a["dt"], a["scale"],
                                  a["causal"], a["out"], a["lse"], a["ws"], a["wsb"], a["st"], 0, 0)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_attention_refuses_bad_caches(kw, status):
    assert attention(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hq=3), 1),
    (dict(pages=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(qs=500), 1), (dict(T=6), 1), (dict(B=4), 1),
    (dict(pages=1 << 30), 2), (dict(Hq=5000), 2), (dict(T=1 << 31, B=1 << 31), 2),
    (dict(q=0), 1), (dict(out=0), 1), (dict(lens=0), 1), (dict(tab=0), 1),
    (dict(q=at(4) + 16), 3), (dict(qs=520), 3), (dict(out=at(5) + 8), 3), (dict(lse=at(8) + 2), 3),
    (dict(tab=at(6) + 2), 3), (dict(lens=at(7) + 1), 3), (dict(cu=at(9) + 2), 3), (dict(st=at(9) + 2), 3),
    (dict(out=at(4)), 1), (dict(out=at(0) + 64), 1), (dict(lse=at(5) + 64), 1), (dict(lse=at(4)), 1),
    (dict(out=at(6)), 1), (dict(out=at(7)), 1), (dict(cu=at(5)), 1), (dict(st=at(5)), 1),
    (dict(st=at(7)), 1), (dict(lse=at(3)), 1),
    (dict(T=0, B=0, q=0, out=0), 0),
])
def test_attention_refusals(kw, status):
    assert attention(**kw) == status


def test_attention_refuses_extents_beyond_64_bits():
    for qs in (1 << 61, (1 << 63) - 16):
        assert attention(qs=qs) == 2


def test_workspace_sizes():
    f = fq.fp4_attention_workspace_bytes
    for bad in [(-1, 4, 8, 2, 128, 512), (4, -1, 8, 2, 128, 512), (4, 4, 0, 2, 128, 512), (4, 4, 8, 3, 128, 512),
                (4, 4, 8, 2, 96, 512), (4, 4, 8, 0, 128, 512), (4, 4, 8, 2, 128, -1)]:
        assert f(*bad) == -1
    assert f(0, 0, 8, 2, 128, 512) == 0
    assert f(1, 1, 8, 2, 128, 1024) == 0                 # a cluster per item
    for bad in [(1 << 30, 4, 8, 2, 128, 512), (4, 1 << 29, 8, 2, 128, 512), (4, 4, 8, 2, 128, 1 << 30),
                (4, 4, 8192, 2, 128, 512)]:
        assert f(*bad) == -1                             # sizes the call refuses
    # tables of 2^20 keys: parts of CTAs; 100 x 100 rows over them: ranges of keys
    for a, kw in (((5, 5, 4, 2, 128), {}), ((5, 500, 4, 2, 128), dict(T=500, cu=at(12)))):
        kw["pages"] = 65536
        need = f(*a, 1 << 20)
        assert need > 0
        assert attention(wsb=need - 1, **kw) == 1 and attention(ws=0, **kw) == 1
        assert attention(ws=at(11) + 8, **kw) == 3
        assert attention(ws=at(5), **kw) == 1 and attention(ws=at(0), **kw) == 1


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (12, 2, 64), (24, 24, 64), (17, 1, 128), (1, 1, 128), (256, 2, 64)])
def test_one_workspace_for_every_smaller_call(Hq, Hkv, D):
    """The exact size is not monotone; the bound is, and covers every call below it."""
    exact, bound = fq.fp4_attention_workspace_bytes, fq.fp4_attention_workspace_bound
    sizes = [1, 2, 3, 7, 16, 17, 60, 100, 256, 300, 512, 1024, 2048, 5000]
    keys = [0, 16, 128, 144, 512, 4096, 20000, 131072, 1 << 20]
    most = {}                                    # the largest call below each size
    for i, B in enumerate(sizes):
        for j, T in enumerate(sizes):
            for k, n in enumerate(keys):
                here = [exact(B, T, Hq, Hkv, D, n)] + [most.get(x, 0) for x in ((i - 1, j, k), (i, j - 1, k), (i, j, k - 1))]
                most[i, j, k] = max(here)
                assert most[i, j, k] <= bound(B, T, Hq, Hkv, D, n), (B, T, n)
                assert bound(B, T, Hq, Hkv, D, n) <= bound(B + 1, T + 3, Hq, Hkv, D, n + 16)
    assert any(exact(1, sizes[j], Hq, Hkv, D, 131072) > exact(1, 5000, Hq, Hkv, D, 131072) for j in range(len(sizes)))
    assert bound(0, 0, Hq, Hkv, D, 512) == 0 and bound(-1, 4, Hq, Hkv, D, 512) == -1
    assert bound(4, 4, Hq, Hkv, 96, 512) == -1 and bound(4, 4, 8192, Hkv, D, 512) == -1


def test_the_struct_matches_the_header():
    assert ctypes.sizeof(fq.KVCacheStruct) == 6 * ctypes.sizeof(ctypes.c_void_p) + 4 * 8


def test_tensor_calls_refuse_cpu_tensors_and_bad_shapes():
    import torch
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    c = (u8(4, 2, 16, 64), u8(4, 2, 16, 8), u8(4, 2, 16, 64), u8(4, 2, 8, 16))
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        fq.kv_append_nvfp4(c, k, k, slots)
    with pytest.raises(ValueError, match="CUDA"):
        fq.kv_gather_nvfp4(c, slots)
    with pytest.raises(ValueError, match="CUDA"):
        fq.attention_nvfp4(k, c, torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        fq.kv_cache_nvfp4(4, 24, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        fq.kv_cache_nvfp4(4, 16, 2, 96, device="cpu")


def test_attention_launch_shape():
    """The choice of kernel: host only (152 SMs without a device)."""
    f = fq.fp4_attention_launch_shape
    decode, prefill = "kv_decode_kernel", "kv_prefill_kernel"
    assert f(1, 1, 12, 2, 128, 1000) == {"kernel": decode, "parts": 8}
    assert f(128, 128, 56, 8, 128, 16384) == {"kernel": decode, "parts": 0}
    assert f(200, 200, 32, 8, 128, 200) == {"kernel": decode, "parts": 1}
    assert f(1, 80, 32, 8, 128, 80)["kernel"] == decode          # few items of few keys
    assert f(1, 4096, 32, 8, 128, 4096) == {"kernel": prefill, "parts": 1}
    assert f(1, 64, 32, 8, 128, 60000)["kernel"] == prefill and f(1, 64, 32, 8, 128, 60000)["parts"] > 8
    for B, T, keys in [(1, 1, 0), (1, 10 ** 6, 1), (7, 3, 10 ** 6), (10 ** 6, 1, 16), (3, 100, 2 ** 30 - 16)]:
        for Hq, Hkv, D in [(1, 1, 64), (128, 1, 128), (24, 24, 64)]:
            s = f(B, T, Hq, Hkv, D, keys)
            assert 1 <= s["parts"] <= 32 if s["kernel"] == prefill else s["parts"] in (0, 1, 2, 3, 4, 6, 8)
            # only what is joined from memory has a workspace
            need = fq.fp4_attention_workspace_bytes(B, T, Hq, Hkv, D, keys)
            assert (need > 0) == (s["parts"] > 1 if s["kernel"] == prefill else s["parts"] == 0)
    for bad in [(0, 1, 8, 2, 128, 512), (1, 0, 8, 2, 128, 512), (4, 4, 8, 3, 128, 512), (4, 4, 8, 2, 96, 512),
                (1 << 30, 4, 8, 2, 128, 512)]:
        with pytest.raises(fq.Fp4Error):
            f(*bad)
