"""The NVFP4 key/value cache operators as they are measured: cases, inputs, plain forms.

Three operators work on one paged cache that holds keys and values in NVFP4 (E2M1
codes, two per byte, and one E4M3 scale per 16 channels of a head):

  append     rotates queries and keys by their positions, quantizes keys and values
             and stores them in the slots of their tokens;
  gather     reads the tokens of given slots back in 16 bits;
  attention  softmax(q k^T) v over the pages of every sequence of a batch.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own``
is true, with the library's calls.  ``exact`` computes them in 64 bits.
"""
import math
import random

import torch

own = False

# (query heads, key/value heads, channels): the hidden widths 1536, 5120 and 7168 of the
# library's own configurations in heads of 128 (12, 40 and 56), 6144 = (32 + 2 * 8) * 128
# as the width of a fused q/k/v projection, and 1536 in heads of 64 (24)
HEADS = [(12, 2, 128), (12, 12, 128), (32, 8, 128), (40, 8, 128), (56, 8, 128), (24, 8, 64), (24, 24, 64)]
PAGES = [16, 32, 48, 64, 128]
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one sequence decodes one token: launch latency only
        dict(name="append_T1", kind="append", tokens=1, heads=12, kv_heads=2, dim=128, dtype="bf16",
             page=16, rot=128, interleaved=False),
        # a decode batch of 41 sequences, pairs rotated in place, half of the channels
        dict(name="append_T41_partial", kind="append", tokens=41, heads=40, kv_heads=8, dim=128,
             dtype="fp16", page=16, rot=64, interleaved=True),
        # a prefill of 8192 tokens
        dict(name="append_T8192", kind="append", tokens=8192, heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=64, rot=128, interleaved=False),
        # an encoder's states for cross attention: keys and values only, no rotation, odd count
        dict(name="append_T30011_cross", kind="append", tokens=30011, heads=0, kv_heads=24, dim=64,
             dtype="fp16", page=48, rot=0, interleaved=False),
        # one short sequence decodes one token
        dict(name="decode_B1_L1000", kind="attention", batch=1, len_min=1000, len_max=1000, q_len=1,
             heads=12, kv_heads=2, dim=128, dtype="bf16", page=16, causal=True),
        # a decode batch of 41 sequences between 1 and 8191 tokens long
        dict(name="decode_B41_ragged", kind="attention", batch=41, len_min=1, len_max=8191, q_len=1,
             heads=32, kv_heads=8, dim=128, dtype="bf16", page=16, causal=True),
        # a large decode batch of long sequences: the cache's bytes are all that counts
        dict(name="decode_B128_L16k", kind="attention", batch=128, len_min=12001, len_max=16384, q_len=1,
             heads=56, kv_heads=8, dim=128, dtype="fp16", page=64, causal=True),
        # one very long sequence decodes one token: work split along the keys
        dict(name="decode_B1_L131071", kind="attention", batch=1, len_min=131071, len_max=131071, q_len=1,
             heads=40, kv_heads=8, dim=128, dtype="bf16", page=128, causal=True),
        # four tokens a sequence, as when drafted tokens are verified
        dict(name="verify_B16_Q4", kind="attention", batch=16, len_min=3001, len_max=5003, q_len=4,
             heads=24, kv_heads=8, dim=64, dtype="bf16", page=32, causal=True),
        # a prompt of 4096 tokens
        dict(name="prefill_B1_Q4096", kind="attention", batch=1, len_min=4096, len_max=4096, q_len=4096,
             heads=32, kv_heads=8, dim=128, dtype="bf16", page=64, causal=True),
        # the next 1021 tokens of two prompts of which up to 20000 are cached
        dict(name="chunk_B2_Q1021", kind="attention", batch=2, len_min=12007, len_max=20011, q_len=1021,
             heads=32, kv_heads=8, dim=128, dtype="fp16", page=16, causal=True),
        # cross attention: 8 decoders' 500 tokens to encoder states of another length
        dict(name="cross_B8_Q500", kind="attention", batch=8, len_min=1111, len_max=1500, q_len=500,
             heads=24, kv_heads=24, dim=64, dtype="fp16", page=48, causal=False),
    ]


def draw(rng: random.Random):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, kv_heads, dim = rng.choice(HEADS)
    common = dict(dim=dim, dtype=rng.choice(["bf16", "fp16"]), page=rng.choice(PAGES))
    if rng.random() < 0.35:
        rot = rng.choice([0, 32, dim // 2, dim, dim])
        tokens = log_int(1, 9000)
        return dict(kind="append", tokens=tokens, heads=rng.choice([0, heads, heads]), kv_heads=kv_heads, rot=rot,
                    interleaved=rng.random() < 0.4, **common)
    if rng.random() < 0.6:     # decode, or a few tokens a sequence
        batch = log_int(1, 160)
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
        len_max = max(q_len, min(log_int(1, 150000), 1100000 // (batch * q_len)))
    else:                      # prompts, or pieces of them
        batch = log_int(1, 12)
        q_len = log_int(9, max(10, 4000 // batch))
        most = int(1.2e11 / (batch * q_len * heads * dim))
        len_max = max(q_len, min(q_len + rng.choice([0, log_int(1, 20000)]), most))
    causal = rng.random() < 0.75
    len_min = len_max if rng.random() < 0.3 else rng.randint(1, len_max)
    return dict(kind="attention", batch=batch, len_min=len_min, len_max=len_max, q_len=q_len, heads=heads,
                kv_heads=kv_heads, causal=causal, **common)


def _lengths(case):
    """Lengths of the batch's sequences: evenly spread, in an order of their own."""
    b, lo, hi = case["batch"], case["len_min"], case["len_max"]
    lens = [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]
    random.Random(b).shuffle(lens)
    return lens


def work(case):
    D, hkv, hq = case["dim"], case["kv_heads"], case["heads"]
    token = 2 * hkv * (D // 2 + D // 16)              # cached bytes of one token: codes and scales of k and v
    if case["kind"] == "append":
        T = case["tokens"]
        read = 2 * T * (hq + 2 * hkv) * D + 8 * T + (8 * T + 4 * T * case["rot"] if case["rot"] else 0)
        written = 2 * T * hq * D + T * token
        back = T * token + 8 * T + 4 * T * hkv * D     # the gather: cached bytes in, 16 bits out
        flops = T * (hq + hkv) * case["rot"] * 3 + 4 * T * hkv * D * 3
        return {"bytes": read + written + back, "flops": flops}
    lens, ql = _lengths(case), case["q_len"]
    T = case["batch"] * ql
    pairs = 0
    for n in lens:
        pairs += sum(max(0, n - ql + i + 1) for i in range(ql)) if case["causal"] else n * ql
    pages = sum(-(-n // case["page"]) for n in lens)
    return {"bytes": sum(lens) * token + 4 * T * hq * D + 4 * T * hq + 4 * pages + 8 * case["batch"],
            "flops": 4 * D * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _quantize(x):
    """NVFP4 of x [..., D] (32 bits): packed codes [..., D/2] and E4M3 scale bytes [..., D/16]."""
    y = x.unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    v = torch.where(s > 0, y * (1.0 / s), torch.zeros_like(y))
    a = v.abs()
    # nearest, ties to the even code: 0 | .25 | .5 | .75 | 1 | 1.25 | 1.5 | 1.75 | 2 | 2.5 | 3 | 3.5 | 4 | 5 | 6
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(packed, sf):
    """32-bit values of packed codes [..., D/2] and scale bytes [..., D/16]."""
    table = torch.tensor(_E2M1 + [-x for x in _E2M1], device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    return (table[codes.int()].unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _empty_cache(pages, case, g):
    """A cache whose pages hold what earlier sequences left there: any bytes."""
    hkv, page, D = case["kv_heads"], case["page"], case["dim"]
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    return [u8(pages, hkv, page, D // 2), u8(pages, hkv, page, D // 16), u8(pages, hkv, page, D // 2),
            u8(pages, hkv, D // 16, page)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, D, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    randn = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    if case["kind"] == "append":
        T = case["tokens"]
        pages = T // page + 5
        # q, k and v are slices of one projection's output, as a fused product leaves them
        qkv = randn(T, (hq + 2 * hkv) * D)
        qkv[:, ::61] *= 8.0                             # channels that stick out, as projections have
        qkv = qkv.to(dt)
        q, k, v = (t.unflatten(-1, (-1, D)) if t.shape[-1] else None for t in qkv.split((hq * D, hkv * D, hkv * D), -1))
        state = dict(case=case, q=q, k=k, v=v, cache=_empty_cache(pages, case, g),
                     slots=torch.randperm(pages * page, device="cuda", generator=g)[:T],
                     out_k=torch.empty(T, hkv, D, dtype=dt, device="cuda"),
                     out_v=torch.empty(T, hkv, D, dtype=dt, device="cuda"),
                     out_q=torch.empty(T, hq, D, dtype=dt, device="cuda") if hq else None,
                     positions=None, cos_sin=None)
        if case["rot"]:
            longest = 40960
            freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
            angle = torch.arange(longest, dtype=torch.float64, device="cuda")[:, None] * freq
            state["cos_sin"] = torch.cat((angle.cos(), angle.sin()), -1).float()
            state["positions"] = torch.randint(0, longest, (T,), device="cuda", generator=g)
        return state
    lens, B, ql = _lengths(case), case["batch"], case["q_len"]
    used = [-(-n // page) for n in lens]
    most = max(used)
    pages = sum(used) + 3
    cache = _empty_cache(pages, case, g)
    order = torch.randperm(pages, device="cuda", generator=g)[: sum(used)].to(torch.int32)
    start = torch.tensor([sum(used[:i]) for i in range(B)], device="cuda")
    at = start[:, None] + torch.arange(most, device="cuda")
    tables = torch.where(torch.arange(most, device="cuda") < torch.tensor(used, device="cuda")[:, None],
                         order[at.clamp(max=len(order) - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    step = max(1, (1 << 26) // (hkv * page * D))
    for i in range(0, len(order), step):
        p = order[i:i + step].long()
        k = randn(len(p), hkv, page, D)
        k[..., 5::37] *= 4.0                            # keys have channels that stick out
        cache[0][p], cache[1][p] = _quantize(k)
        cache[2][p], sf = _quantize(randn(len(p), hkv, page, D))
        cache[3][p] = sf.transpose(-1, -2)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # slots behind a sequence's end hold anything, scale bytes that are no numbers among it
    last = torch.tensor([[int(n) // page, int(n) % page] for n in lens if n % page], device="cuda").reshape(-1, 2)
    row = torch.tensor([i for i, n in enumerate(lens) if n % page], device="cuda", dtype=torch.long)
    if len(row):
        tail = torch.arange(page, device="cuda") >= last[:, 1:]
        pg = tables[row, last[:, 0]].long()
        cache[1][pg] = torch.where(tail[:, None, :, None], torch.full((), 127, dtype=torch.uint8, device="cuda"), cache[1][pg])
        cache[3][pg] = torch.where(tail[:, None, None, :], torch.full((), 255, dtype=torch.uint8, device="cuda"), cache[3][pg])
    cu = torch.arange(0, B + 1, device="cuda", dtype=torch.int32) * ql
    q = (1.5 * randn(B * ql, hq, D)).to(dt)
    return dict(case=case, q=q, cache=cache, tables=tables.contiguous(), seq_lens=seq_lens, cu=cu,
                out=torch.empty_like(q), lse=torch.empty(B * ql, hq, device="cuda"))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _rotate(x, positions, cos_sin, rot, interleaved):
    """x [T, H, D] in 32 bits with its first `rot` channels turned by the angles of its positions."""
    cos, sin = cos_sin[positions].unsqueeze(1).chunk(2, -1)
    part = x[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else part.chunk(2, -1)
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, d), -1).flatten(-2) if interleaved else torch.cat((c, d), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    case, dt = s["case"], s["k"].dtype
    k, q = s["k"].float(), None if s["q"] is None else s["q"].float()
    if case["rot"]:
        turn = (s["positions"], s["cos_sin"], case["rot"], case["interleaved"])
        k, q = _rotate(k, *turn), None if q is None else _rotate(q, *turn)
    kc, ksf, vc, vsf = s["cache"]
    page, off = s["slots"] // case["page"], s["slots"] % case["page"]
    kc[page, :, off], ksf[page, :, off] = _quantize(k)
    vc[page, :, off], vsf[page, :, :, off] = _quantize(s["v"].float())
    # and the tokens read back from their slots
    return {"q": None if q is None else q.to(dt), "k": _values(kc[page, :, off], ksf[page, :, off]).to(dt),
            "v": _values(vc[page, :, off], vsf[page, :, :, off]).to(dt)}


def _plain_attention(s):
    case, q = s["case"], s["q"]
    hkv, D, ql, B = case["kv_heads"], case["dim"], case["q_len"], case["batch"]
    kc, ksf, vc, vsf = s["cache"]
    pages = s["tables"].clamp(min=0).long()
    L = pages.shape[1] * case["page"]
    # [B, pages, Hkv, page, D] -> [B, Hkv, L, D]; nothing behind a sequence's end is read
    j = torch.arange(L, device=q.device)
    here = (j < s["seq_lens"][:, None])[:, None, :, None]
    k = torch.where(here, _values(kc[pages], ksf[pages]).transpose(1, 2).reshape(B, hkv, L, D), 0.0)
    v = torch.where(here, _values(vc[pages], vsf[pages].transpose(-1, -2)).transpose(1, 2).reshape(B, hkv, L, D), 0.0)
    # rows: [B, Hkv, G * q_len, D]
    x = q.float().reshape(B, ql, hkv, -1, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    w = (x @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    i = torch.arange(ql, device=q.device)
    last = s["seq_lens"][:, None] - ql + i if case["causal"] else (s["seq_lens"] - 1)[:, None].expand(B, ql)
    w = w.reshape(B, hkv, -1, ql, L).masked_fill(j > last[:, None, None, :, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w = (w - top).exp()
    total = w.sum(-1, keepdim=True)
    out = w.reshape(B, hkv, -1, L) @ v
    out = out.reshape(B, hkv, -1, ql, D) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B * ql, -1, D).to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B * ql, -1)}


def run(s):
    if not own:
        return _plain_append(s) if s["case"]["kind"] == "append" else _plain_attention(s)
    import rmsnorm_fp4_quant_gb300 as fq
    case = s["case"]
    if case["kind"] == "append":
        fq.kv_append_nvfp4(s["cache"], s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"],
                           cos_sin=s["cos_sin"], interleaved=case["interleaved"], out_q=s["out_q"])
        k, v = fq.kv_gather_nvfp4(s["cache"], s["slots"], out_k=s["out_k"], out_v=s["out_v"])
        return {"q": s["out_q"], "k": k, "v": v}
    out, lse = fq.attention_nvfp4(s["q"], s["cache"], s["tables"], s["seq_lens"],
                                  cu_seqlens_q=None if case["q_len"] == 1 else s["cu"], causal=case["causal"],
                                  out=s["out"], return_lse=True, lse=s["lse"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# the same from the definition, in 64 bits
# ---------------------------------------------------------------------------
_POINTS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_numbers(device):
    """The 127 numbers of E4M3 that are not negative, by their byte; no number behind the last."""
    return torch.tensor([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=device)


def _nearest(x, points):
    """Index of the point nearest to each x >= 0 (points ascend), a tie to the even index."""
    hi = torch.searchsorted(points, x).clamp(1, len(points) - 1)
    lo = hi - 1
    below, above = x - points[lo], points[hi] - x
    return torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def _exact_block_values(x):
    """What x [..., D] (64 bits) is worth after NVFP4 quantization: value of its code times its scale.

    The rule of the library's producers is nearest-even of x * (1 / s), with the reciprocal and the
    product each rounded once to 32 bits: 16-bit inputs over a 4-bit scale fall on the middle between
    two codes often, and which side they go to is part of the rule."""
    numbers = _e4m3_numbers(x.device)
    points = torch.tensor(_POINTS, dtype=torch.float64, device=x.device)
    y = x.reshape(*x.shape[:-1], -1, 16)
    s = numbers[_nearest((y.abs().amax(-1) / 6).clamp(max=448), numbers)].unsqueeze(-1)
    ratio = (y.abs() * (1 / s).float().double()).float().double()
    mag = points[_nearest(torch.where(s > 0, ratio, 0.0), points)]
    return (torch.sign(y) * mag * s).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    D = case["dim"]
    if case["kind"] == "append":
        q, k, v = (None if t is None else t.double() for t in (s["q"], s["k"], s["v"]))
        if case["rot"]:
            h = case["rot"] // 2
            table = s["cos_sin"].double()[s["positions"]]
            z = torch.complex(table[:, :h], table[:, h:])[:, None]

            def turn(x):
                first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["interleaved"] else (slice(0, h), slice(h, 2 * h))
                y, r = x.clone(), torch.complex(x[..., first], x[..., second]) * z
                y[..., first], y[..., second] = r.real, r.imag
                return y
            q, k = None if q is None else turn(q), turn(k)
        return {"q": q, "k": _exact_block_values(k), "v": _exact_block_values(v)}
    group = case["heads"] // case["kv_heads"]
    grid = torch.tensor(_POINTS + [-p for p in _POINTS], dtype=torch.float64, device="cuda")
    numbers = torch.cat((_e4m3_numbers("cuda"), torch.zeros(129, dtype=torch.float64, device="cuda")))
    outs, lses = [], []
    for b, n in enumerate(_lengths(case)):
        q = s["q"][b * case["q_len"]:(b + 1) * case["q_len"]].double()
        ids = s["tables"][b, : -(-n // case["page"])].long()

        def tokens(codes, sf):       # [pages, Hkv, page, ...] -> [n, Hkv, D]
            c = torch.empty(*codes.shape[:-1], D, dtype=torch.long, device="cuda")
            c[..., 0::2], c[..., 1::2] = codes % 16, codes // 16
            val = grid[c] * numbers[sf.long()].repeat_interleave(16, -1)
            return val.permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], D)[:n]
        k = tokens(s["cache"][0][ids], s["cache"][1][ids])
        v = tokens(s["cache"][2][ids], s["cache"][3][ids].permute(0, 1, 3, 2))
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        for h in range(case["heads"]):
            w = q[:, h] @ k[:, h // group].T / math.sqrt(D)
            if case["causal"]:
                hidden = torch.ones_like(w, dtype=torch.bool).triu(n - case["q_len"] + 1)
                w = w.masked_fill(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(w, -1)
            p = (w - lse[:, h:h + 1].clamp(min=-1e300)).exp()
            out[:, h] = p @ v[:, h // group]
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
