"""Host-side refusals of beam selection, page and masked attention entry points (no GPU): every
call below fails its checks before anything is launched or read."""
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


def beam(**kw):
    a = dict(x=at(4), stride=0, dt=0, s=at(5), f=at(6), end=3, B=2, K=3, V=1000, n=6, os=at(7), op=at(8), ot=at(9),
             of=at(10), ws=at(11), size=1 << 30)
    a.update(kw)
    return fq.fp4_beam_select(a["x"], a["stride"], a["dt"], a["s"], a["f"], a["end"], a["B"], a["K"], a["V"], a["n"],
                              a["os"], a["op"], a["ot"], a["of"], a["ws"], a["size"], 0, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), 1), (dict(dt=-1), 1), (dict(B=-1), 1), (dict(K=0), 1), (dict(V=0), 1), (dict(n=0), 1),
    (dict(K=257), 2), (dict(n=65), 2), (dict(V=(1 << 24) + 1), 2), (dict(B=1 << 30), 2), (dict(B=1 << 22, K=200, V=1 << 24), 2),
    (dict(stride=999), 1), (dict(stride=1 << 60), 2), (dict(end=-1), 1), (dict(end=1000), 1),
    (dict(f=0), 1), (dict(of=0), 1), (dict(x=0), 1), (dict(s=0), 1), (dict(os=0), 1), (dict(op=0), 1), (dict(ot=0), 1),
    (dict(ws=0), 1), (dict(size=100), 1), (dict(size=-1), 1),
    (dict(x=at(4) + 1), 3), (dict(x=at(4) + 2, dt=2), 3), (dict(s=at(5) + 2), 3), (dict(os=at(7) + 1), 3), (dict(ws=at(11) + 8), 3),
    (dict(op=at(7) + 8), 1), (dict(ot=at(4) + 4), 1), (dict(of=at(6) + 5), 1), (dict(os=at(5)), 1), (dict(ws=at(4)), 1),
    (dict(ws=at(7) + 32), 1),
    (dict(B=0, x=0, s=0, ws=0, size=0), 0),
])
def test_beam_refusals(kw, status):
    assert beam(**kw) == status


def test_beam_workspace():
    f = fq.fp4_beam_select_workspace_bytes
    assert f(-1, 1, 10, 1, 0) == f(1, 0, 10, 1, 0) == f(1, 1, 10, 65, 0) == f(1, 1, 10, 1, 7) == -1
    sizes = [1, 2, 3, 7, 8, 40, 200]
    for V in (1, 600, 50001, 200003):
        last = 0
        for B in sizes:
            assert f(B, 4, V, 8, 0) >= last                       # what a smaller call needs is there
            last = f(B, 4, V, 8, 0)
    for K in (1, 5, 9):
        assert f(3, K, 5000, 8, 0) <= f(3, K + 1, 5000, 8, 0) and f(3, K, 5000, 8, 0) <= f(3, K, 5600, 8, 0)


def fork(c=None, **kw):
    a = dict(r=at(4), t=at(5), most=8, l=at(6), B=3, p=at(7), nl=at(8), N=5, new=2, ot=at(9), ol=at(10), orr=at(11), os=at(12),
             ws=at(13), size=1 << 20, st=at(14))
    a.update(kw)
    return fq.fp4_kv_fork_nvfp4(c or cache(), a["r"], a["t"], a["most"], a["l"], a["B"], a["p"], a["nl"], a["N"], a["new"], a["ot"],
                                a["ol"], a["orr"], a["os"], a["ws"], a["size"], a["st"], 0, 0)


def trim(c=None, **kw):
    a = dict(r=at(4), t=at(5), most=8, l=at(6), B=3, f=at(7), e=at(8), ot=at(9), ol=at(10), orr=at(11))
    a.update(kw)
    return fq.fp4_kv_trim_nvfp4(c or cache(), a["r"], a["t"], a["most"], a["l"], a["B"], a["f"], a["e"], a["ot"], a["ol"], a["orr"], 0, 0)


def compact(c=None, **kw):
    a = dict(r=at(4), t=at(5), most=8, l=at(6), B=3, ot=at(9), orr=at(11), om=at(12), on=at(13), ws=at(14), size=1 << 20)
    a.update(kw)
    return fq.fp4_kv_compact_nvfp4(c or cache(), a["r"], a["t"], a["most"], a["l"], a["B"], a["ot"], a["orr"], a["om"], a["on"],
                                   a["ws"], a["size"], 0, 0)


CACHES = [(dict(num_pages=-1), 1), (dict(page_size=24), 2), (dict(head_dim=96), 2), (dict(num_kv_heads=0), 1), (dict(num_pages=1 << 31), 2)]


@pytest.mark.parametrize("kw,status", CACHES)
@pytest.mark.parametrize("call", [fork, trim, compact])
def test_page_calls_refuse_bad_caches(call, kw, status):
    assert call(cache(**kw)) == status


@pytest.mark.parametrize("call", [fork, compact])
def test_page_calls_refuse_bad_buffers(call):
    assert call(cache(k_sf=0)) == 1 and call(cache(v_packed=at(2) + 8)) == 3 and call(cache(v_sf=at(0) + 64)) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(most=-1), 1), (dict(new=-1), 1), (dict(size=-1), 1),
    (dict(p=0), 1), (dict(most=1 << 30), 2), (dict(B=1 << 29), 2), (dict(N=1 << 29), 2), (dict(N=1 << 20, most=1 << 12), 2),
    (dict(new=1 << 29), 2), (dict(N=1 << 20, new=1 << 12), 2),
    (dict(r=0), 1), (dict(t=0), 1), (dict(l=0), 1), (dict(ot=0), 1), (dict(ol=0), 1), (dict(orr=0), 1), (dict(os=0), 1),
    (dict(ws=0), 1), (dict(size=16), 1),
    (dict(r=at(4) + 2), 3), (dict(os=at(12) + 4), 3), (dict(ws=at(13) + 4), 3), (dict(st=at(14) + 1), 3), (dict(nl=at(8) + 2), 3),
    (dict(ot=at(5)), 1), (dict(orr=at(4)), 1), (dict(ol=at(6) + 4), 1), (dict(os=at(0) + 64), 1), (dict(ws=at(3)), 1), (dict(st=at(9) + 4), 1),
    (dict(p=at(11) + 8), 1), (dict(t=at(2) + 4), 1),
])
def test_fork_refusals(kw, status):
    assert fork(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(most=-1), 1), (dict(most=1 << 30), 2), (dict(B=1 << 29), 2), (dict(r=0), 1), (dict(t=0), 1), (dict(l=0), 1),
    (dict(ot=0), 1), (dict(ol=0), 1), (dict(orr=0), 1), (dict(f=at(7) + 2), 3), (dict(ot=at(9) + 1), 3), (dict(ot=at(5) + 4), 1),
    (dict(orr=at(4) + 8), 1), (dict(e=at(10)), 1), (dict(ol=at(9) + 4), 1),
])
def test_trim_refusals(kw, status):
    assert trim(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(most=-1), 1), (dict(size=-1), 1), (dict(most=1 << 30), 2), (dict(r=0), 1), (dict(t=0), 1), (dict(l=0), 1),
    (dict(ot=0), 1), (dict(orr=0), 1), (dict(om=0), 1), (dict(on=0), 1), (dict(ws=0), 1), (dict(size=8), 1), (dict(om=at(12) + 2), 3),
    (dict(ws=at(14) + 4), 3), (dict(ot=at(5)), 1), (dict(om=at(11) + 4), 1), (dict(on=at(4)), 1), (dict(ws=at(1) + 16), 1),
])
def test_compact_refusals(kw, status):
    assert compact(**kw) == status


def test_pages_workspace():
    f = fq.fp4_kv_pages_workspace_bytes
    assert f(-1, 0) == f(0, -1) == f(1 << 31, 0) == f(0, 1 << 30) == -1
    assert 0 < f(0, 0) <= f(10, 0) <= f(10, 7) <= f(1000, 7) and f(1000, 7) % 16 == 0


def attention(c=None, **kw):
    a = dict(q=at(4), t=at(5), most=8, l=at(6), cu=0, B=5, T=5, Hq=4, dt=0, scale=0.1, causal=1, cap=30.0, sl=at(7), w=100, pre=at(8),
             out=at(9), lse=at(10), ws=at(11), size=1 << 34, st=0)
    a.update(kw)
    return fq.fp4_attention_nvfp4_ex(a["q"], 0, c or cache(), a["t"], a["most"], a["l"], a["cu"], a["B"], a["T"], a["Hq"], a["dt"],
                                     a["scale"], a["causal"], a["cap"], a["sl"], a["w"], a["pre"], a["out"], a["lse"], a["ws"],
                                     a["size"], a["st"], 0, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(cap=-1.0), 1), (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(cap=1048577.0), 1), (dict(w=-1), 1),
    (dict(causal=0), 1), (dict(causal=0, w=0), 1), (dict(causal=0, pre=0), 1), (dict(sl=at(7) + 2), 3), (dict(pre=at(8) + 1), 3),
    (dict(out=at(7)), 1), (dict(lse=at(8) + 4), 1), (dict(ws=at(7)), 1), (dict(dt=2), 1), (dict(Hq=3), 1),
    (dict(T=0, B=0, cu=0), 0),
])
def test_masked_attention_refusals(kw, status):
    if "ws" in kw:                                                   # a call that needs a workspace
        kw = dict(kw, most=4096, w=0)
    assert attention(**kw) == status


def test_the_windowed_workspace_is_that_of_fewer_keys():
    """As the header says, and never above the bound's."""
    for B, T, Hq, Hkv, D, keys, window in [(1, 1, 8, 1, 128, 100000, 30000), (2, 600, 8, 2, 64, 20000, 5000), (3, 3, 4, 4, 128, 65536, 70000)]:
        held = min(keys, window + -(-T // B) + 63)
        need = fq.fp4_attention_workspace_bytes(B, T, Hq, Hkv, D, held)
        assert 0 <= need <= fq.fp4_attention_workspace_bound(B, T, Hq, Hkv, D, keys)
        c = cache(num_pages=1 << 16, num_kv_heads=Hkv, head_dim=D)
        args = dict(c=c, most=keys // 16, B=B, T=T, Hq=Hq, cu=at(12), w=window, cap=0.0, sl=0, pre=0)
        if need:
            assert attention(**args, ws=at(11), size=need - 1) == 1
        # a misplaced output is found behind the size's check
        assert attention(**args, ws=at(11), size=need, out=at(4) + 32) == 1


def test_status_and_types():
    assert fq.FP4_ERR_NO_PAGES == 6 and "page" in fq.fp4_status_string(6) and fq.FP4_DT_FP32 == 2


def test_tensor_calls_refuse_cpu_tensors():
    import torch
    x = torch.zeros(2, 3, 10)
    with pytest.raises(ValueError):
        fq.beam_select(x, torch.zeros(2, 3))
    with pytest.raises(ValueError):
        fq.beam_select(x[0], torch.zeros(2, 3))
    c = [torch.zeros(4, 1, 16, 32, dtype=torch.uint8), torch.zeros(4, 1, 16, 4, dtype=torch.uint8),
         torch.zeros(4, 1, 16, 32, dtype=torch.uint8), torch.zeros(4, 1, 4, 16, dtype=torch.uint8)]
    i = torch.zeros(4, dtype=torch.int32)
    for call in (fq.kv_fork_nvfp4, fq.kv_trim_nvfp4, fq.kv_compact_nvfp4):
        with pytest.raises(ValueError):
            call(c, i, i[None], i[:1])


def test_statuses_of_the_pages_are_read_with_their_own_call():
    assert fq.fp4_kv_read_status(0, 0) == fq.FP4_ERR_INVALID_ARG
    assert fq.fp4_kv_read_status(0x10002, 0) == fq.FP4_ERR_INVALID_ARG
    # every other status has the name that it has everywhere
    for status in (0, 1, 2, 3, 4, 5, 99):
        assert fq.lib().fp4_kv_status_string(status) == fq.lib().fp4_status_string(status)
