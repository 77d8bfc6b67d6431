"""Decoding over the paged NVFP4 cache as it is measured: cases, inputs, plain forms.

Four operators that work on the cache of perf/operators.py (E2M1 codes, one E4M3 scale
per 16 channels of a head) between the tokens of a batch:

  beam       the best continuations of every beam search, over beams and vocabulary;
  fork       the cache's sequences continued by their children: pages shared, the last
             one copied where it is to be written, pages given up and taken;
  compact    pages of ended sequences given up, the remaining ones moved together;
  attention  softmax over the cached keys with capped logits, a bias that grows with
             distance, a window of the latest keys, a prefix that every row sees.

``run`` computes them with elementary torch operations in 32 bits (scores that are
compared in 64), or, where ``own`` is true, with the library's calls.  ``exact`` computes
them from their definitions, in 64 bits.
"""
import math
import random

import torch

own = False

# (query heads, key/value heads, channels): hidden widths of the library's configurations
# (1536, 5120, 7168; 6144 as a fused projection's) in heads of 128 and 64
HEADS = [(12, 2, 128), (12, 12, 128), (32, 8, 128), (40, 8, 128), (56, 8, 128), (24, 8, 64), (24, 24, 64)]
PAGES = [16, 32, 48, 64, 128]
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one request, four beams: latency only
        dict(name="beam_B1_K4", kind="beam", batch=1, beams=4, vocab=32768, take=4, dtype="bf16", finished=False),
        # a few requests, an odd vocabulary in 32 bits, some beams ended, twice as many candidates as beams
        dict(name="beam_B8_K5_odd", kind="beam", batch=8, beams=5, vocab=50001, take=10, dtype="fp32", finished=True),
        # a large batch over a large vocabulary: the logits' bytes are all that counts
        dict(name="beam_B64_K8", kind="beam", batch=64, beams=8, vocab=131072, take=16, dtype="fp16", finished=True),
        # one request's four beams go on: latency only
        dict(name="fork_G1_K4", kind="fork", groups=1, ins=4, outs=4, len_min=1003, len_max=1003, new=1, dead=False,
             kv_heads=2, dim=128, page=16),
        # two long prompts sampled sixteen times each: their pages are shared, the last one copied
        dict(name="fork_G2_samples", kind="fork", groups=2, ins=1, outs=16, len_min=17003, len_max=20011, new=1,
             dead=False, kv_heads=8, dim=128, page=16),
        # a large batch of beam searches goes on, some of them have ended
        dict(name="fork_G64_K8", kind="fork", groups=64, ins=8, outs=8, len_min=9, len_max=4095, new=1, dead=True,
             kv_heads=8, dim=128, page=64),
        # a few sequences, a third of them ended
        dict(name="compact_B12", kind="compact", batch=12, len_min=1, len_max=700, window=0, ended=0.34, kv_heads=2,
             dim=128, page=16),
        # many sequences, half of them ended, the pages behind the others' windows given up too
        dict(name="compact_B256", kind="compact", batch=256, len_min=100, len_max=8191, window=4096, ended=0.5,
             kv_heads=8, dim=128, page=64),
        # a decode batch: capped logits over a window of the latest keys, pages behind it given up
        dict(name="decode_B41_cap_window", kind="attention", batch=41, len_min=1, len_max=8191, q_len=1, heads=32,
             kv_heads=8, dim=128, dtype="bf16", page=16, causal=True, cap=50.0, window=1024, slopes=False, prefix=False),
        # long sequences decode one token each, with a bias that grows with distance
        dict(name="decode_B16_slopes", kind="attention", batch=16, len_min=12001, len_max=16384, q_len=1, heads=40,
             kv_heads=8, dim=128, dtype="fp16", page=64, causal=True, cap=0.0, window=0, slopes=True, prefix=False),
        # a prompt of 4096 tokens with capped logits
        dict(name="prefill_Q4096_cap", kind="attention", batch=1, len_min=4096, len_max=4096, q_len=4096, heads=32,
             kv_heads=8, dim=128, dtype="bf16", page=64, causal=True, cap=30.0, window=0, slopes=False, prefix=False),
        # the latest 500 tokens of eight sequences whose first tokens (an image's, say) see each other
        dict(name="chunk_B8_prefix_slopes", kind="attention", batch=8, len_min=1111, len_max=1500, q_len=500, heads=24,
             kv_heads=24, dim=64, dtype="fp16", page=48, causal=True, cap=0.0, window=0, slopes=True, prefix=True),
    ]


def draw(rng: random.Random):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["beam", "fork", "compact", "attention", "attention"])
    heads, kv_heads, dim = rng.choice(HEADS)
    page = rng.choice(PAGES)
    if kind == "beam":
        batch, beams = log_int(1, 96), rng.randint(1, 12)
        vocab = min(log_int(1000, 200000), 67000000 // (batch * beams))
        return dict(kind=kind, batch=batch, beams=beams, vocab=vocab, take=rng.choice([beams, 2 * beams, 2 * beams + 1]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), finished=rng.random() < 0.5)
    if kind == "fork":
        outs = rng.randint(1, 16)
        ins = rng.choice([1, outs, outs])
        groups = log_int(1, 80)
        hi = log_int(1, max(2, min(20000, 2000000 // (groups * max(ins, outs)))))
        new = rng.choice([0, 1, 1, 1, 2, 5, log_int(8, 600) if groups * outs < 64 else 3])
        return dict(kind=kind, groups=groups, ins=ins, outs=outs, len_min=hi if rng.random() < 0.3 else rng.randint(1, hi),
                    len_max=hi, new=new, dead=rng.random() < 0.4, kv_heads=kv_heads, dim=dim, page=page)
    if kind == "compact":
        batch = log_int(1, 300)
        hi = log_int(1, max(2, min(20000, 2000000 // batch)))
        return dict(kind=kind, batch=batch, len_min=rng.randint(1, hi), len_max=hi,
                    window=rng.choice([0, 0, log_int(1, 8192)]), ended=rng.choice([0.0, 0.1, 0.34, 0.5, 0.9]),
                    kv_heads=kv_heads, dim=dim, page=page)
    causal = rng.random() < 0.85
    what = dict(cap=rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]), window=0, slopes=rng.random() < 0.4, prefix=False)
    if causal:
        what["window"] = rng.choice([0, 0, log_int(1, 4096)])
        what["prefix"] = rng.random() < 0.3
    if not (what["cap"] or what["window"] or what["slopes"] or what["prefix"]):
        what["cap"] = 40.0
    if rng.random() < 0.6:     # decode, or a few tokens a sequence
        batch = log_int(1, 160)
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
        len_max = max(q_len, min(log_int(1, 150000), 250000 // (batch * q_len)))
    else:                      # prompts, or pieces of them
        batch = log_int(1, 12)
        q_len = log_int(9, max(10, 4000 // batch))
        most = int(3.3e10 / (batch * q_len * heads * dim))
        len_max = max(q_len, min(q_len + rng.choice([0, log_int(1, 20000)]), most))
    return dict(kind=kind, batch=batch, len_min=len_max if rng.random() < 0.3 else rng.randint(1, len_max),
                len_max=len_max, q_len=q_len, heads=heads, kv_heads=kv_heads, dim=dim, dtype=rng.choice(["bf16", "fp16"]),
                page=page, causal=causal, **what)


# ---------------------------------------------------------------------------
# what a case's inputs share whatever the seed
# ---------------------------------------------------------------------------
def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread, in an order of their own."""
    lens = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(n).shuffle(lens)
    return lens


def _ended_rows(case):
    return int(0.15 * case["batch"] * case["beams"]) if case["finished"] else 0


def _families(case):
    """Of every group: its sequences' length, and which of them each child continues (-1: the group has ended)."""
    rng = random.Random(case["groups"] * 31 + case["outs"])
    got = []
    for g, n in enumerate(_spread(case["groups"], case["len_min"], case["len_max"])):
        dead = case["dead"] and g % 7 == 3
        got.append((n, [-1 if dead else rng.randrange(case["ins"]) for _ in range(case["outs"])]))
    return got


def _windows(case):
    """Of every sequence: cached tokens, first and end of those that stay."""
    lens = _spread(case["batch"], case["len_min"], case["len_max"])
    order = list(range(case["batch"]))
    random.Random(case["batch"] + 1).shuffle(order)
    ended = set(order[: int(case["ended"] * case["batch"])])
    return [(n, max(0, n - case["window"]) if case["window"] else 0, 0 if i in ended else n) for i, n in enumerate(lens)]


def _prefixes(case, lens):
    ql = case["q_len"]
    return [[0, n // 2, max(0, n - ql // 2), n + 5][i % 4] for i, n in enumerate(lens)]


def work(case):
    if case["kind"] == "beam":
        rows = case["batch"] * case["beams"]
        size = 4 if case["dtype"] == "fp32" else 2
        read = (rows - _ended_rows(case)) * case["vocab"]
        return {"bytes": read * size + 4 * rows + case["finished"] * rows + (12 + case["finished"]) * case["batch"] * case["take"],
                "flops": 3 * read}
    D, hkv, page = case["dim"], case["kv_heads"], case["page"]
    token = 2 * hkv * (D // 2 + D // 16)              # cached bytes of one token: codes and scales of k and v
    if case["kind"] == "fork":
        fam, new = _families(case), case["new"]
        used = sum(-(-n // page) for n, _ in fam) * case["ins"]
        kids = case["groups"] * case["outs"]
        most = -(-(case["len_max"] + new) // page)
        # children beyond the first of a sequence copy what is in its last page, to whole 16 tokens
        copied = sum((len(c) - len(set(c))) * -(-(n % page) // 16) * 16 for n, c in fam if c[0] >= 0 and new)
        pool = _pool_pages(case)
        return {"bytes": 4 * used + 4 * len(fam) * case["ins"] + 4 * kids + 4 * kids * (most + 1) + 8 * kids * new + 8 * pool
                + 2 * copied * token, "flops": used + kids * most}
    if case["kind"] == "compact":
        wins = _windows(case)
        most = -(-case["len_max"] // page)
        live = sum(max(0, -(-to // page) - first // page) for _, first, to in wins)
        pool = _pool_pages(case)
        # a share of the live pages lies behind the first `live` ones, as the pages' order is random
        moved = live * (pool - live) // pool
        return {"bytes": 3 * 4 * case["batch"] * most + 5 * 4 * pool + 2 * moved * page * token, "flops": pool}
    lens, ql, hq, w = _spread(case["batch"], case["len_min"], case["len_max"]), case["q_len"], case["heads"], case["window"]
    pre = _prefixes(case, lens) if case["prefix"] else [0] * len(lens)
    pairs = keys = 0
    for n, pr in zip(lens, pre):
        first = n
        for i in range(ql):
            hi = max(n - ql + i + 1, min(pr, n)) if case["causal"] else n
            lo = max(0, n - ql + i + 1 - w) if w else 0
            pairs += max(0, hi - lo)
            first = min(first, lo) if hi > lo else first
        keys += n - first
    T = case["batch"] * ql
    return {"bytes": keys * token + 4 * T * hq * D + 4 * T * hq + 4 * -(-keys // page) + 8 * case["batch"],
            "flops": 4 * D * hq * pairs}


def _pool_pages(case):
    if case["kind"] == "fork":
        page, fam = case["page"], _families(case)
        pages = 0
        for n, c in fam:
            whole = int(0.6 * n) // page
            pages += whole + case["ins"] * (-(-n // page) - whole)
            pages += sum(-(-(n + case["new"]) // page) - n // page for _ in c)
        return pages + 2 * case["groups"] + 7
    return sum(-(-n // case["page"]) for n, _, _ in _windows(case)) + case["batch"] + 5


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
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(packed, sf):
    """32-bit values of packed codes [..., D/2] and scale bytes [..., D/16]."""
    table = torch.tensor(_E2M1 + [-x for x in _E2M1], device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    return (table[codes.int()].unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _any_cache(pages, case, g):
    """A cache whose pages hold any bytes."""
    hkv, page, D = case["kv_heads"], case["page"], case["dim"]
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    return [u8(pages, hkv, page, D // 2), u8(pages, hkv, page, D // 16), u8(pages, hkv, page, D // 2),
            u8(pages, hkv, D // 16, page)]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_beam(case, g):
    B, K, V, n = case["batch"], case["beams"], case["vocab"], case["take"]
    x = torch.randn(B * K, V, device="cuda", generator=g) * 2.5
    x[torch.arange(B * K, device="cuda")[:, None],           # a few tokens stick out of every row
      torch.randint(0, V, (B * K, 12), device="cuda", generator=g)] += 9.0
    x[0::3, 5::97] = -math.inf                                # tokens that may not follow
    logits = x.to(DTYPES[case["dtype"]]).view(B, K, V)
    finished = None
    if case["finished"]:
        finished = torch.zeros(B * K, dtype=torch.bool, device="cuda")
        finished[torch.randperm(B * K, device="cuda", generator=g)[: _ended_rows(case)]] = True
        finished = finished.view(B, K)
    e = lambda t: torch.empty(B, n, dtype=t, device="cuda")  # noqa: E731
    return dict(case=case, logits=logits, finished=finished, end=2,
                scores=-torch.rand(B, K, device="cuda", generator=g) * 6.0 - 12.0,
                out=[e(torch.float32), e(torch.int32), e(torch.int32)] + ([e(torch.bool)] if case["finished"] else []))


def _prepare_fork(case, g):
    page, ins, outs, new, fam = case["page"], case["ins"], case["outs"], case["new"], _families(case)
    pool = _pool_pages(case)
    most = -(-(case["len_max"] + new) // page)
    order = torch.randperm(pool, device="cuda", generator=g).tolist()
    refs, tables, lens, parents, at = [0] * pool, [], [], [], 0
    shuffle = random.Random(order[0])
    for n, kids in fam:
        whole, used = int(0.6 * n) // page, -(-n // page)
        shared = order[at:at + whole]            # the prompt's pages, held by every sequence of the group
        at += whole
        for p in shared:
            refs[p] += ins
        for p in shared[:1]:
            refs[p] += 1                         # and the first by a store of prompts, too
        for _ in range(ins):
            mine = order[at:at + used - whole]
            at += used - whole
            for p in mine:
                refs[p] += 1
            tables.append(shared + mine + [-1] * (most - used))
            lens.append(n)
        kids = list(kids)
        shuffle.shuffle(kids)
        parents += [k if k < 0 else len(tables) - ins + k for k in kids]
    for p in order[at:at + case["groups"]]:      # pages of sequences that are not in the call
        refs[p] = 1
    N = len(parents)
    return dict(case=case, cache=_any_cache(pool, case, g), refs=_i32(refs), tables=_i32(tables), lens=_i32(lens),
                parents=_i32(parents), out_tables=torch.empty(N, most, dtype=torch.int32, device="cuda"),
                out_lens=torch.empty(N, dtype=torch.int32, device="cuda"),
                out_refs=torch.empty(pool, dtype=torch.int32, device="cuda"),
                slots=torch.empty(N, new, dtype=torch.int64, device="cuda"))


def _prepare_compact(case, g):
    page, wins = case["page"], _windows(case)
    pool = _pool_pages(case)
    most = -(-case["len_max"] // page)
    order = torch.randperm(pool, device="cuda", generator=g).tolist()
    refs, tables, at = [0] * pool, [], 0
    for n, _, _ in wins:
        used = -(-n // page)
        tables.append(order[at:at + used] + [-1] * (most - used))
        for p in order[at:at + used]:
            refs[p] = 1
        at += used
    if len(tables) > 1 and tables[0][0] >= 0 and tables[1][0] >= 0:      # two that share their first page
        refs[tables[1][0]] -= 1
        tables[1][0] = tables[0][0]
        refs[tables[0][0]] += 1
    B = len(wins)
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(case=case, cache=_any_cache(pool, case, g), refs=_i32(refs), tables=_i32(tables),
                lens=_i32([w[0] for w in wins]), first=_i32([w[1] for w in wins]), end=_i32([w[2] for w in wins]),
                trimmed=[e(B, most), e(B), e(pool)], out=[e(B, most), e(pool), e(pool), e(1)])


def _prepare_attention(case, g):
    dt = DTYPES[case["dtype"]]
    hq, hkv, D, page, B, ql, w = (case[k] for k in ("heads", "kv_heads", "dim", "page", "batch", "q_len", "window"))
    randn = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    lens = _spread(B, case["len_min"], case["len_max"])
    used = [-(-n // page) for n in lens]
    # pages behind the window of a sequence's first row were given up
    gone = [max(0, n - ql + 1 - w) // page if w else 0 for n in lens]
    most, held = max(used), sum(used) - sum(gone)
    pages = held + 3
    cache = _any_cache(pages, case, g)
    order = torch.randperm(pages, device="cuda", generator=g)[:held].to(torch.int32)
    start = torch.tensor([sum(used[:i]) - sum(gone[:i + 1]) for i in range(B)], device="cuda")
    at, col = start[:, None] + torch.arange(most, device="cuda"), torch.arange(most, device="cuda")
    tables = torch.where((col < _i32(used)[:, None]) & (col >= _i32(gone)[:, None]),
                         order[at.clamp(0, max(0, len(order) - 1))], torch.full((), -1, dtype=torch.int32, device="cuda"))
    step = max(1, (1 << 26) // (hkv * page * D))
    for i in range(0, len(order), step):
        p = order[i:i + step].long()
        k = randn(len(p), hkv, page, D)
        k[..., 5::37] *= 4.0                            # keys have channels that stick out
        cache[0][p], cache[1][p] = _quantize(k)
        cache[2][p], sf = _quantize(randn(len(p), hkv, page, D))
        cache[3][p] = sf.transpose(-1, -2)
    # slots behind a sequence's end hold anything, scale bytes that are no numbers among it
    last = torch.tensor([[int(n) // page, int(n) % page] for n in lens if n % page], device="cuda").reshape(-1, 2)
    row = torch.tensor([i for i, n in enumerate(lens) if n % page], device="cuda", dtype=torch.long)
    if len(row):
        tail = torch.arange(page, device="cuda") >= last[:, 1:]
        pg = tables[row, last[:, 0]].long()
        cache[1][pg] = torch.where(tail[:, None, :, None], torch.full((), 127, dtype=torch.uint8, device="cuda"), cache[1][pg])
        cache[3][pg] = torch.where(tail[:, None, None, :], torch.full((), 255, dtype=torch.uint8, device="cuda"), cache[3][pg])
    # logits that are capped are large enough to meet the cap
    q = ((6.0 if case["cap"] else 1.5) * randn(B * ql, hq, D)).to(dt)
    slopes = prefix = None
    if case["slopes"]:
        slopes = 2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float32, device="cuda") / hq)
    if case["prefix"]:
        prefix = _i32(_prefixes(case, lens))
    return dict(case=case, q=q, cache=cache, tables=tables.contiguous(), seq_lens=_i32(lens),
                cu=torch.arange(0, B + 1, device="cuda", dtype=torch.int32) * ql, slopes=slopes, prefix=prefix,
                out=torch.empty_like(q), lse=torch.empty(B * ql, hq, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"beam": _prepare_beam, "fork": _prepare_fork, "compact": _prepare_compact, "attention": _prepare_attention}
    return make[case["kind"]](case, g)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_beam(s):
    case = s["case"]
    B, K, V, n = case["batch"], case["beams"], case["vocab"], case["take"]
    x = s["logits"]
    top = x.amax(-1, keepdim=True).float()
    lse = top.double() + (x.float() - top).exp().sum(-1, keepdim=True, dtype=torch.float64).log()
    # a row's own order is that of its logits; equal ones in the order of their tokens
    m = min(n, V)
    best, token = torch.sort(torch.where(x == x, x.float(), -math.inf), dim=-1, descending=True, stable=True)
    best, token = best[..., :m].double(), token[..., :m]
    cand = torch.where(lse.isfinite(), s["scores"].double()[..., None] + (best - lse), -math.inf)
    if s["finished"] is not None:
        done = s["finished"][..., None]
        first = torch.arange(m, device=x.device) == 0
        cand = torch.where(done, torch.where(first, s["scores"].double()[..., None], -math.inf), cand)
        token = torch.where(done, s["end"], token)
    cand = torch.where(cand == cand, cand, -math.inf).flatten(1)
    if cand.shape[1] < n:                                    # fewer candidates than places
        cand = torch.cat((cand, cand.new_full((B, n - cand.shape[1]), -math.inf)), 1)
    score, at = torch.sort(cand, dim=-1, descending=True, stable=True)
    score, at = score[:, :n], at[:, :n]
    some, at = score > -math.inf, at.clamp(max=K * m - 1)
    row = torch.arange(B, device=x.device)[:, None] * K + at // m
    out = {"scores": score.float(), "parents": torch.where(some, row, -1).int(),
           "tokens": torch.where(some, token.flatten(1).gather(1, at), -1).int()}
    if s["finished"] is not None:
        out["finished"] = some & (s["finished"].flatten()[row] | (out["tokens"] == s["end"]))
    return out


def _held(table, refs):
    return (table >= 0) & (table < len(refs))


def _count(table, mask, pool):
    """How often each page is among the table's entries of the mask."""
    at = torch.where(mask, table, pool).flatten().long()
    return torch.zeros(pool + 1, dtype=torch.int32, device=table.device).index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:pool]


def _plain_fork(s):
    case, tables, refs, cache = s["case"], s["tables"], s["refs"], s["cache"]
    page, new, pool, most = case["page"], case["new"], len(s["refs"]), tables.shape[1]
    col = torch.arange(most, device=refs.device)
    lens = s["lens"].clamp(0, most * page)
    some = (s["parents"] >= 0) & (s["parents"] < len(lens))
    par = s["parents"].clamp(0, len(lens) - 1).long()
    had = torch.where(some, lens[par], 0)
    grown = torch.where(some, (had + new).clamp(max=most * page), 0)
    used, whole, part = (had + page - 1) // page, had // page, (had % page > 0) & (grown > had)
    # references: the old sequences give theirs up, the children share what they do not write
    old = _held(tables, refs) & (col < ((lens + page - 1) // page)[:, None])
    mine = torch.where(col < used[:, None], tables[par], -1)
    kept = _held(mine, refs) & (col < torch.where(part, whole, used)[:, None])
    count = refs - _count(tables, old, pool) + _count(mine, kept, pool)
    # the last page stays with its first child if nobody else holds it; the others copy it
    last = mine.gather(1, whole.clamp(max=most - 1).long()[:, None])[:, 0]
    part = part & _held(last, refs)
    child = torch.arange(len(par), dtype=torch.int32, device=refs.device)
    at = torch.where(part, last, pool).long()
    heir = torch.full((pool + 1,), len(par), dtype=torch.int32, device=refs.device).scatter_reduce_(0, at, child, "amin")
    keeps = part & (heir[at] == child) & (torch.cat((count, count.new_zeros(1)))[at] <= 0)
    count = count + _count(last, keeps, pool)
    # pages to take, in the children's order, from the free ones, lowest first
    copies = part & ~keeps
    wants = ((col >= used[:, None]) & (col < ((grown + page - 1) // page)[:, None])) | (copies[:, None] & (col == whole[:, None]))
    free = torch.argsort((count > 0).int(), stable=True)
    rank = wants.flatten().cumsum(0).view_as(wants) - 1
    got = wants & (rank < (count <= 0).sum())
    taken = free[rank.clamp(0, pool - 1)].int()
    table = torch.where(wants, torch.where(got, taken, -1), mine)
    count = count.clamp(min=0) + _count(taken, got, pool)
    dst = table.gather(1, whole.clamp(max=most - 1).long()[:, None])[:, 0]
    copies = copies & (dst >= 0)
    a, b, n = last[copies].long(), dst[copies].long(), (had % page)[copies]
    group = (torch.arange(page, device=refs.device) // 16 * 16 < n[:, None])[:, None, :, None]
    cache[0][b], cache[1][b], cache[2][b] = [torch.where(group, c[a], c[b]) for c in cache[:3]]
    cache[3][b] = torch.where(group.transpose(-1, -2), cache[3][a], cache[3][b])
    pos = had[:, None] + torch.arange(new, device=refs.device)
    where = table.gather(1, (pos // page).clamp(max=most - 1).long())
    slots = torch.where((pos < grown[:, None]) & _held(where, refs), where.long() * page + pos % page, -1)
    return {"tables": table, "lens": grown.int(), "refs": count, "slots": slots, "cache": list(cache)}


def _plain_compact(s):
    case, refs, cache = s["case"], s["refs"], s["cache"]
    page, pool, most = case["page"], len(refs), s["tables"].shape[1]
    col = torch.arange(most, device=refs.device)
    # give up
    lens = s["lens"].clamp(0, most * page)
    end = torch.minimum(s["end"].clamp(min=0), lens)
    old = _held(s["tables"], refs) & (col < ((lens + page - 1) // page)[:, None])
    stay = old & (col >= (s["first"].clamp(min=0) // page)[:, None]) & (col < ((end + page - 1) // page)[:, None])
    tables = torch.where(stay, s["tables"], -1)
    count = refs - _count(s["tables"], old & ~stay, pool)
    # move together
    live, at = count > 0, torch.arange(pool, device=refs.device)
    n = live.sum()
    a, b = (live & (at >= n)).nonzero()[:, 0], (~live & (at < n)).nonzero()[:, 0]
    cache[0][b], cache[1][b], cache[2][b], cache[3][b] = cache[0][a], cache[1][a], cache[2][a], cache[3][a]
    to = torch.where(live, at, -1).int()
    to[a] = b.int()
    moved = torch.where(at < n, count, 0)
    moved[b] = count[a]
    return {"trimmed": tables, "lens": end, "trimmed_refs": count, "refs": moved, "map": to, "live": n.int()[None],
            "tables": torch.where(tables >= 0, to[tables.clamp(min=0).long()], -1), "cache": list(cache)}


def _plain_attention(s):
    case, q = s["case"], s["q"]
    hkv, D, ql, B = case["kv_heads"], case["dim"], case["q_len"], case["batch"]
    kc, ksf, vc, vsf = s["cache"]
    pages = s["tables"].clamp(min=0).long()
    L = pages.shape[1] * case["page"]
    i, j = torch.arange(ql, device=q.device), torch.arange(L, device=q.device)
    n = s["seq_lens"][:, None]
    pos = n - ql + i if case["causal"] else (n - 1).expand(B, ql)        # of the rows [B, q_len]
    hi = pos + 1 if s["prefix"] is None else torch.maximum(pos + 1, torch.minimum(s["prefix"][:, None], n))
    lo = (pos + 1 - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(pos)
    # [B, pages, Hkv, page, D] -> [B, Hkv, L, D]; nothing that no row sees is read
    here = ((j < n) & (j >= lo.amin(1, keepdim=True)))[:, None, :, None]
    k = torch.where(here, _values(kc[pages], ksf[pages]).transpose(1, 2).reshape(B, hkv, L, D), 0.0)
    v = torch.where(here, _values(vc[pages], vsf[pages].transpose(-1, -2)).transpose(1, 2).reshape(B, hkv, L, D), 0.0)
    # rows: [B, Hkv, G * q_len, D]
    x = q.float().reshape(B, ql, hkv, -1, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    w = (x @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    if case["cap"]:
        w = case["cap"] * torch.tanh(w / case["cap"])
    w = w.reshape(B, hkv, -1, ql, L)
    if s["slopes"] is not None:
        away = ((n - ql + i)[:, :, None] - j).abs()
        w = w - s["slopes"].view(1, hkv, -1, 1, 1) * away[:, None, None]
    seen = (j < hi[..., None]) & (j >= lo[..., None])
    w = w.masked_fill(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w = (w - top).exp()
    total = w.sum(-1, keepdim=True)
    out = (w.reshape(B, hkv, -1, L) @ v).reshape(B, hkv, -1, ql, D) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B * ql, -1, D).to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B * ql, -1)}


def run(s):
    case = s["case"]
    if not own:
        plain = {"beam": _plain_beam, "fork": _plain_fork, "compact": _plain_compact, "attention": _plain_attention}
        return plain[case["kind"]](s)
    import rmsnorm_fp4_quant_gb300 as fq
    if case["kind"] == "beam":
        got = fq.beam_select(s["logits"], s["scores"], case["take"], finished=s["finished"], end_token=s["end"], out=s["out"])
        return dict(zip(("scores", "parents", "tokens", "finished"), got))
    if case["kind"] == "fork":
        tables, lens, refs, slots = fq.kv_fork_nvfp4(
            s["cache"], s["refs"], s["tables"], s["lens"], s["parents"], new_tokens=case["new"], out_tables=s["out_tables"],
            out_seq_lens=s["out_lens"], out_refs=s["out_refs"], out_slots=s["slots"])
        return {"tables": tables, "lens": lens, "refs": refs, "slots": slots, "cache": list(s["cache"])}
    if case["kind"] == "compact":
        trimmed, lens, count = fq.kv_trim_nvfp4(
            s["cache"], s["refs"], s["tables"], s["lens"], first=s["first"], end=s["end"], out_tables=s["trimmed"][0],
            out_seq_lens=s["trimmed"][1], out_refs=s["trimmed"][2])
        tables, refs, to, live = fq.kv_compact_nvfp4(
            s["cache"], count, trimmed, lens, out_tables=s["out"][0], out_refs=s["out"][1], out_map=s["out"][2],
            out_live=s["out"][3])
        return {"trimmed": trimmed, "lens": lens, "trimmed_refs": count, "refs": refs, "map": to, "live": live,
                "tables": tables, "cache": list(s["cache"])}
    out, lse = fq.attention_nvfp4(s["q"], s["cache"], s["tables"], s["seq_lens"],
                                  cu_seqlens_q=None if case["q_len"] == 1 else s["cu"], causal=case["causal"],
                                  softcap=case["cap"] or None, window=case["window"] or None, alibi_slopes=s["slopes"],
                                  prefix_lens=s["prefix"], out=s["out"], return_lse=True, lse=s["lse"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_beam(case, s):
    B, K, V, n = case["batch"], case["beams"], case["vocab"], case["take"]
    x = s["logits"].double()
    total = torch.logsumexp(x, -1)
    score = s["scores"].double()[..., None] + (x - total[..., None])
    score = torch.where(total.isfinite()[..., None], score, -math.inf)
    if s["finished"] is not None:
        score = torch.where(s["finished"][..., None], -math.inf, score)
        score[..., s["end"]] = torch.where(s["finished"], s["scores"].double(), score[..., s["end"]])
    score = score.reshape(B, K * V)
    index = torch.arange(K * V, device=x.device)
    out = {"scores": [], "parents": [], "tokens": [], "finished": []}
    for _ in range(n):                                        # the best one left, n times
        best = score.amax(1, keepdim=True)
        first = torch.where(score == best, index, K * V).amin(1, keepdim=True)
        some = (best > -math.inf)[:, 0]
        row = torch.arange(B, device=x.device) * K + first[:, 0] // V
        token = first[:, 0] % V
        out["scores"].append(best[:, 0])
        out["parents"].append(torch.where(some, row, -1).int())
        out["tokens"].append(torch.where(some, token, -1).int())
        if s["finished"] is not None:
            out["finished"].append(some & (s["finished"].flatten()[row] | (token == s["end"])))
        score.scatter_(1, first, -math.inf)
    return {k: torch.stack(v, 1) for k, v in out.items() if v}


def _exact_fork(case, s):
    """One child after the other, with lists."""
    page, new, most = case["page"], case["new"], s["tables"].shape[1]
    refs, tables, lens, parents = (s[k].tolist() for k in ("refs", "tables", "lens", "parents"))
    pool = len(refs)
    for t, n in zip(tables, lens):
        for p in t[: -(-n // page)]:
            refs[p] -= 1
    kids, writes = [], {}
    for i, p in enumerate(parents):
        n = lens[p] if p >= 0 else 0
        m = min(n + new, most * page) if p >= 0 else 0
        mine = list(tables[p][: -(-n // page)]) if p >= 0 else []
        if n % page and m > n:
            writes.setdefault(mine[-1], []).append(i)
        kids.append([mine, n, m])
        for q in mine[:-1] if n % page and m > n else mine:
            refs[q] += 1
    keeps = {c[0] for p, c in writes.items() if refs[p] == 0}
    for i in keeps:
        refs[kids[i][0][-1]] = 1
    free = [p for p in range(pool) if refs[p] <= 0][::-1]
    cache = [c.clone() for c in s["cache"]]
    out, slots = [], []
    for i, (mine, n, m) in enumerate(kids):
        if n % page and m > n and i not in keeps:
            src, mine[-1] = mine[-1], free.pop()
            refs[mine[-1]] = 1
            g = -(-(n % page) // 16) * 16
            for k in range(3):
                cache[k][mine[-1], :, :g] = s["cache"][k][src, :, :g]
            cache[3][mine[-1], :, :, :g] = s["cache"][3][src, :, :, :g]
        while len(mine) * page < m:
            mine.append(free.pop())
            refs[mine[-1]] = 1
        out.append(mine + [-1] * (most - len(mine)))
        slots.append([mine[x // page] * page + x % page if x < m else -1 for x in range(n, n + new)])
    return {"tables": _i32(out), "lens": _i32([m for _, _, m in kids]), "refs": _i32(refs),
            "slots": torch.tensor(slots, dtype=torch.int64, device="cuda").reshape(len(kids), new), "cache": cache}


def _exact_compact(case, s):
    page, most = case["page"], s["tables"].shape[1]
    refs, tables, lens, first, end = (s[k].tolist() for k in ("refs", "tables", "lens", "first", "end"))
    pool, trimmed = len(refs), []
    for t, n, a, b in zip(tables, lens, first, end):
        keep = range(a // page, -(-min(b, n) // page))
        trimmed.append([p if i in keep else -1 for i, p in enumerate(t)])
        for i in range(-(-n // page)):
            if i not in keep:
                refs[t[i]] -= 1
    live = [p for p in range(pool) if refs[p] > 0]
    n = len(live)
    hole = [p for p in range(n) if refs[p] <= 0][::-1]
    to = {p: p if p < n else hole.pop() for p in live}
    cache = [c.clone() for c in s["cache"]]
    a, b = [p for p in live if to[p] != p], [to[p] for p in live if to[p] != p]
    for c, d in zip(cache, s["cache"]):
        c[b] = d[a]
    back = {q: p for p, q in to.items()}
    return {"trimmed": _i32(trimmed), "lens": _i32([min(b, n) for b, n in zip(end, lens)]), "trimmed_refs": _i32(refs),
            "refs": _i32([refs[back[q]] if q in back else 0 for q in range(pool)]),
            "map": _i32([to.get(p, -1) for p in range(pool)]), "live": _i32([n]),
            "tables": _i32([[to[p] if p >= 0 else -1 for p in t] for t in trimmed]), "cache": cache}


def _exact_attention(case, s):
    D, ql, page, group = case["dim"], case["q_len"], case["page"], case["heads"] // case["kv_heads"]
    grid = torch.tensor(_E2M1 + [-p for p in _E2M1], dtype=torch.float64, device="cuda")
    numbers = torch.tensor([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                            for e in range(16) for m in range(8)][:127] + [0.0] * 129, dtype=torch.float64, device="cuda")
    outs, lses = [], []
    lens = _spread(case["batch"], case["len_min"], case["len_max"])
    for b, n in enumerate(lens):
        q = s["q"][b * ql:(b + 1) * ql].double()
        ids = s["tables"][b, : -(-n // page)].long().clamp(min=0)

        def tokens(codes, sf):       # [pages, Hkv, page, ...] -> [n, Hkv, D]
            c = torch.empty(*codes.shape[:-1], D, dtype=torch.long, device="cuda")
            c[..., 0::2], c[..., 1::2] = codes % 16, codes // 16
            val = grid[c] * numbers[sf.long()].repeat_interleave(16, -1)
            return val.permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], D)[:n]
        k = tokens(s["cache"][0][ids], s["cache"][1][ids])
        v = tokens(s["cache"][2][ids], s["cache"][3][ids].permute(0, 1, 3, 2))
        here = torch.arange(n, device="cuda")
        own_place = (torch.arange(ql, device="cuda") + (n - ql))[:, None]
        hidden = here > own_place if case["causal"] else torch.zeros(ql, n, dtype=torch.bool, device="cuda")
        if case["prefix"]:
            hidden &= here >= _prefixes(case, lens)[b]
        if case["window"]:
            hidden |= here <= own_place - case["window"]
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        for h in range(case["heads"]):
            w = q[:, h] @ k[:, h // group].T / math.sqrt(D)
            if case["cap"]:
                w = case["cap"] * torch.tanh(w / case["cap"])
            if case["slopes"]:
                w = w - float(s["slopes"][h]) * (own_place - here).abs()
            w = w.masked_fill(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(w, -1)
            p = (w - lse[:, h:h + 1].clamp(min=-1e300)).exp()
            out[:, h] = p @ v[:, h // group]
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    make = {"beam": _exact_beam, "fork": _exact_fork, "compact": _exact_compact, "attention": _exact_attention}
    return make[case["kind"]](case, prepare(case, seed))
