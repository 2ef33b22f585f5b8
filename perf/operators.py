"""Workloads of the serving operators: the cache append with its rotation, the attention that reads
the cache, and the sampling of the next token.

Every workload can be computed in two ways from the same inputs: in plain torch operations (``own``
false), and by the calls that a program makes of int4_weight_only_block_amd (``own`` true).

A case is a dict of plain values; its "op" is one of

  append     kv_append_rope: RMS norms per head, rotary positions, query rows out in bf16, keys and
             values into the pages of a cache in bf16 or e4m3
  attention  paged_attention: new tokens of several sequences over their cached keys and values
  sample     sample_logits: one token per row of logits, after temperature, top-k, top-p and min-p

The head layouts are those of the decoder shapes this library serves (8 query heads over 1 or 2
key/value heads of 256, or of 512 on the layers without a window; a window of 512 tokens; a
vocabulary of 262144; logits capped at 30), next to generic ones.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
CAP = 30.0
EPS = 1e-6
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one sequence's next token on a windowed layer: the call of every layer of every decode step
        dict(name="append_decode_1", op="append", tokens=1, heads=8, kv_heads=2, dim=256, rotated=128, theta=1e4,
             cache="bf16", page=64, far=4000, norms=True, salt=1),
        # prefill chunks of many requests at once, on a layer of 512-wide heads that rotates a quarter of its pairs;
        # the cache is in 8 bits
        dict(name="append_prefill_2048_e4m3", op="append", tokens=2048, heads=8, kv_heads=2, dim=512, rotated=64,
             theta=1e6, cache="e4m3", page=64, far=120000, norms=True, salt=2),
        # one sequence's next token on a windowed layer far into a text: only the window is read
        dict(name="attn_decode_1_window", op="attention", seqs=1, chunk=1, longest=2317, shortest=2317, heads=8,
             kv_heads=2, dim=256, window=512, cache="bf16", page=64, idle=0, salt=3),
        # one sequence's next token at the end of a long text on a layer without a window
        dict(name="attn_decode_1_131072", op="attention", seqs=1, chunk=1, longest=131072, shortest=131072, heads=8,
             kv_heads=1, dim=512, window=0, cache="bf16", page=64, idle=0, salt=4),
        # a decode batch of requests of very unlike lengths, cache in 8 bits
        dict(name="attn_decode_48_e4m3", op="attention", seqs=48, chunk=1, longest=16384, shortest=300, heads=8,
             kv_heads=2, dim=256, window=0, cache="e4m3", page=32, idle=1, salt=5),
        # a speculative check of 4 draft tokens in 7 requests
        dict(name="attn_verify_4x7", op="attention", seqs=7, chunk=4, longest=5021, shortest=700, heads=8, kv_heads=2,
             dim=256, window=0, cache="bf16", page=64, idle=0, salt=6),
        # one prefill chunk of 64 tokens far into a text
        dict(name="attn_chunk_64_32768", op="attention", seqs=1, chunk=64, longest=32768, shortest=32768, heads=8,
             kv_heads=2, dim=256, window=0, cache="bf16", page=64, idle=0, salt=7),
        # prefill chunks of several requests on windowed layers
        dict(name="attn_chunk_window_6", op="attention", seqs=6, chunk=512, longest=9000, shortest=40, heads=8,
             kv_heads=2, dim=256, window=512, cache="bf16", page=64, idle=0, salt=8),
        # the largest: long prefill chunks of several requests over 128-wide heads, 4 queries to a key/value head
        dict(name="attn_chunk_2048_5", op="attention", seqs=5, chunk=2048, longest=12288, shortest=1000, heads=32,
             kv_heads=8, dim=128, window=0, cache="bf16", page=128, idle=0, salt=9),
        # the next token of one request, filtered as decoders of this kind are run: top-k 64, top-p 0.95
        dict(name="sample_1_topk", op="sample", rows=1, vocab=262144, filters="topk"),
        # a few rollouts without a filter: the whole distribution is drawn from; an odd vocabulary
        dict(name="sample_5_free", op="sample", rows=5, vocab=100003, filters="free"),
        # a full decode batch in which each request has its own settings, some of them greedy
        dict(name="sample_64_mixed", op="sample", rows=64, vocab=262144, filters="mixed"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    salt = rng.randrange(1 << 30)
    op = rng.choice(["append", "attention", "attention", "sample"])
    if op == "append":
        dim = rng.choice([64, 128, 256, 512])
        kv_heads = rng.choice([1, 2, 4, 8] if dim <= 128 else [1, 2, 4] if dim == 256 else [1, 2])
        return dict(op=op, tokens=_log_int(rng, 1, 2048), heads=kv_heads * rng.choice([1, 3, 4, 8]), kv_heads=kv_heads,
                    dim=dim, rotated=rng.choice([dim // 2, dim // 8]), theta=rng.choice([1e4, 1e6]),
                    cache=rng.choice(["bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128]),
                    far=_log_int(rng, 2, 130000), norms=rng.random() < 0.7, salt=salt)
    if op == "attention":
        dim = rng.choice([64, 128, 256, 512])
        kv_heads = rng.choice([1, 2, 4, 8] if dim <= 128 else [1, 2])
        group = rng.choice([1, 4, 5, 8])
        kind = rng.choice(["decode", "verify", "chunk"])
        seqs = _log_int(rng, 1, 48 if kind == "decode" else 16 if kind == "verify" else 6)
        chunk = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 9, 1024)
        # the cache is kept under 2**19 tokens of 512 values over all sequences
        most = min(65536, (1 << 28) // (seqs * kv_heads * dim))
        longest = max(chunk, _log_int(rng, 16, most))
        return dict(op=op, seqs=seqs, chunk=chunk, longest=longest, shortest=rng.randint(1, longest),
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, window=rng.choice([0, 0, 100, 512, 1024]),
                    cache=rng.choice(["bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128]),
                    idle=rng.choice([0, 0, 1]), salt=salt)
    return dict(op=op, rows=_log_int(rng, 1, 64), vocab=_log_int(rng, 1000, 262144),
                filters=rng.choice(["topk", "free", "mixed"]))


def _lengths(case):
    """(new tokens, cached tokens) of each sequence of an attention case; an idle one has no new token."""
    rng = random.Random(case["salt"])
    q, kv = [], []
    for b in range(case["seqs"]):
        q.append(case["chunk"] if b == 0 else rng.randint(1, case["chunk"]))
        kv.append(max(q[-1], case["longest"] if b == 0 else _log_int(rng, case["shortest"], case["longest"])))
    for _ in range(case["idle"]):
        q.append(0)
        kv.append(case["shortest"])
    return q, kv


def _first_key(position, window):
    return max(0, position - window + 1) if window else 0


def work(case):
    if case["op"] == "append":
        wide = case["dim"] * case["tokens"]
        stored = 2 if case["cache"] == "bf16" else 1
        heads, kv = case["heads"], case["kv_heads"]
        return {"bytes": wide * (4 * (heads + 2 * kv) + 2 * heads + 2 * stored * kv) + 8 * case["tokens"],
                "flops": wide * (8 * heads + 12 * kv)}
    if case["op"] == "attention":
        q, kv = _lengths(case)
        stored = 2 if case["cache"] == "bf16" else 1
        pairs = keys = 0
        for new, long in zip(q, kv):
            if not new:
                continue
            keys += long - _first_key(long - new, case["window"])
            pairs += sum(p + 1 - _first_key(p, case["window"]) for p in range(long - new, long))
        return {"bytes": 2 * stored * keys * case["kv_heads"] * case["dim"]
                + 4 * sum(q) * case["heads"] * case["dim"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    n = case["rows"] * case["vocab"]
    return {"bytes": 4 * n + 28 * case["rows"], "flops": 8 * n}


# ------------------------------------------------------------------ inputs


def _generator(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 1000003 + case.get("salt", 0) % 999983)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE)


def _scales(g, n):
    return 0.01 + 0.02 * _uniform(g, n)


def prepare(case, seed):
    return {"append": _prepare_append, "attention": _prepare_attention, "sample": _prepare_sample}[case["op"]](case, seed)


def _prepare_append(case, seed):
    g = _generator(case, seed)
    t, h, n, d, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    qkv = _normal(g, t, (h + 2 * n) * d) * 1.7  # one fused projection's rows
    pages = -(-t // page) + 3
    slots = torch.randperm(pages * page, generator=g, device=DEVICE)[:t].to(torch.int32)
    positions = torch.randint(0, case["far"], (t,), generator=g, device=DEVICE, dtype=torch.int32)
    shape = (pages, n, page, d)
    s = {"case": case, "q": qkv[:, :h * d], "k": qkv[:, h * d:(h + n) * d], "v": qkv[:, (h + n) * d:],
         "slots": slots, "positions": positions,
         "freqs": case["theta"] ** (-2.0 * torch.arange(case["rotated"], dtype=torch.float64, device=DEVICE) / d),
         "q_norm": None, "k_norm": None, "k_scale": None, "v_scale": None}
    if case["norms"]:
        s["q_norm"], s["k_norm"] = 0.5 + _uniform(g, d), 0.5 + _uniform(g, d)
    for name in ("k_cache", "v_cache"):  # what earlier tokens have left in the pages
        s[name] = _normal(g, *shape).to(torch.bfloat16 if case["cache"] == "bf16" else E4M3)
    if case["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = _scales(g, n), _scales(g, n)
    return s


def _prepare_attention(case, seed):
    g = _generator(case, seed)
    h, n, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    q_lens, kv_lens = _lengths(case)
    widths = [-(-long // page) for long in kv_lens]
    pages = sum(widths) + 2
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32).cpu()
    table = torch.full((len(widths), max(widths)), -1, dtype=torch.int32)
    at = 0
    for b, w in enumerate(widths):
        table[b, :w] = order[at:at + w]
        at += w
    s = {"case": case, "k_scale": None, "v_scale": None,
         "q": (_normal(g, sum(q_lens), h, d) * (2.5 / math.sqrt(d))).to(torch.bfloat16),
         "page_table": table.to(DEVICE),
         "q_starts": torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32).to(DEVICE),
         "kv_lens": torch.tensor(kv_lens, dtype=torch.int32).to(DEVICE),
         "max_q": max(q_lens), "max_kv": max(kv_lens), "ws": None}
    for name in ("k_cache", "v_cache"):
        x = _normal(g, pages, n, page, d)
        if case["cache"] == "e4m3":
            s[name[0] + "_scale"] = _scales(g, n)
            x = (x / s[name[0] + "_scale"].view(1, n, 1, 1)).clamp(-448, 448).to(E4M3)
        s[name] = x.to(torch.bfloat16) if case["cache"] == "bf16" else x
    if own:  # a serving loop keeps one workspace for all its layers and steps
        import int4_weight_only_block_amd as q4
        s["ws"] = torch.empty(q4.paged_attention_workspace_bytes(len(q_lens), h, n, d, s["max_q"], s["max_kv"],
                                                                 case["window"]), dtype=torch.uint8, device=DEVICE)
    return s


def _prepare_sample(case, seed):
    g = _generator(case, seed)
    r, v = case["rows"], case["vocab"]
    # a broad floor with a few dozen plausible tokens above it
    logits = 2.5 * _normal(g, r, v) - 4.0
    some = torch.randint(0, v, (r, 40), generator=g, device=DEVICE)
    logits.scatter_add_(1, some, 12.0 * _uniform(g, r, 40) ** 2 + 4.0)
    s = {"case": case, "logits": logits, "u": _uniform(g, r), "ws": None}
    pick = lambda values, kind: torch.tensor(values, dtype=kind, device=DEVICE)[  # noqa: E731
        torch.randint(0, len(values), (r,), generator=g, device=DEVICE)]
    if case["filters"] == "topk":
        s["temperature"], s["top_k"] = pick([1.0], torch.float32), pick([64], torch.int32)
        s["top_p"], s["min_p"] = pick([0.95], torch.float32), None
    elif case["filters"] == "free":
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = pick([1.0], torch.float32), None, None, None
    else:
        s["temperature"] = pick([0.0, 0.3, 0.7, 1.0, 1.0, 1.4], torch.float32)
        s["top_k"] = pick([0, 0, 1, 20, 64, 1000], torch.int32)
        s["top_p"] = pick([1.0, 0.95, 0.9, 0.5], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.02, 0.1], torch.float32)
    if own:
        import int4_weight_only_block_amd as q4
        s["ws"] = torch.empty(q4.sample_logits_workspace_bytes(r, v), dtype=torch.uint8, device=DEVICE)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        import int4_weight_only_block_amd as q4
        if op == "append":
            q = q4.kv_append_rope(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                                  s["freqs"], q_norm=s["q_norm"], k_norm=s["k_norm"], v_norm=s["case"]["norms"],
                                  eps=EPS, k_scale=s["k_scale"], v_scale=s["v_scale"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "attention":
            return q4.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_starts"],
                                      s["kv_lens"], s["max_q"], s["max_kv"], scale=1.0, window=s["case"]["window"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"], ws=s["ws"])
        idx, prob = q4.sample_logits(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                     top_p=s["top_p"], min_p=s["min_p"], cap=CAP, ws=s["ws"])
        return {"idx": idx, "prob": prob}
    return {"append": _plain_append, "attention": _plain_attention, "sample": _plain_sample}[op](s)


def _rms(x, weight):
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x if weight is None else x * weight


def _rotate(x, positions, freqs):
    """x [T, heads, D]: the pairs (j, j + D/2) of the first len(freqs) j's, turned by positions * freqs."""
    d, r = x.shape[-1], freqs.numel()
    angle = positions.double()[:, None] * freqs[None, :]
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    a, b = x[..., :r], x[..., d // 2:d // 2 + r]
    return torch.cat([a * c - b * s, x[..., r:d // 2], b * c + a * s, x[..., d // 2 + r:]], -1)


def _store(cache, slots, x, scale):
    page = cache.shape[2]
    if scale is not None:
        x = (x / scale.view(1, -1, 1)).clamp(-448, 448)
    x = x.to(cache.dtype)
    if cache.dtype == E4M3:  # moved as bytes
        cache, x = cache.view(torch.uint8), x.view(torch.uint8)
    at = slots.long()
    cache[at // page, :, at % page] = x


def _plain_append(s):
    case = s["case"]
    t, h, n, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    q, k, v = s["q"].reshape(t, h, d), s["k"].reshape(t, n, d), s["v"].reshape(t, n, d)
    if case["norms"]:
        q, k, v = _rms(q, s["q_norm"]), _rms(k, s["k_norm"]), _rms(v, None)
    q, k = _rotate(q, s["positions"], s["freqs"]), _rotate(k, s["positions"], s["freqs"])
    _store(s["k_cache"], s["slots"], k, s["k_scale"])
    _store(s["v_cache"], s["slots"], v, s["v_scale"])
    return {"q": q.to(torch.bfloat16), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _paged(cache, table, scale):
    """The sequences' rows of the cache, [B, kv_heads, tokens, D] in 32 bits."""
    b, w = table.shape
    n, page, d = cache.shape[1:]
    at = table.clamp(min=0).long()
    x = cache.view(torch.uint8)[at].view(E4M3).float() if cache.dtype == E4M3 else cache[at].float()
    if scale is not None:
        x = x * scale.view(1, 1, n, 1, 1)
    return x.permute(0, 2, 1, 3, 4).reshape(b, n, w * page, d)


def _plain_attention(s):
    case = s["case"]
    h, n, d, window = case["heads"], case["kv_heads"], case["dim"], case["window"]
    starts, kv_lens = s["q_starts"].long(), s["kv_lens"].long()
    b, total, group = kv_lens.numel(), s["q"].shape[0], h // n
    k, v = _paged(s["k_cache"], s["page_table"], s["k_scale"]), _paged(s["v_cache"], s["page_table"], s["v_scale"])
    q_lens = starts[1:] - starts[:-1]
    i = torch.arange(s["max_q"], device=DEVICE)
    live = i[None, :] < q_lens[:, None]  # [B, Q]
    token = (starts[:-1, None] + i[None, :]).clamp(max=total - 1)
    q = s["q"][token].float().view(b, -1, n, group, d).permute(0, 2, 1, 3, 4).reshape(b, n, -1, d)
    scores = torch.matmul(q, k.transpose(-1, -2)).view(b, n, s["max_q"], group, -1)
    place = (kv_lens - q_lens)[:, None] + i[None, :]  # [B, Q]
    j = torch.arange(scores.shape[-1], device=DEVICE)
    seen = (j <= place[..., None]) & live[..., None]
    if window:
        seen = seen & (j > place[..., None] - window)
    scores = scores.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total_p = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, n, -1, p.shape[-1]), v).view(b, n, s["max_q"], group, d)
    o = o / torch.where(total_p == 0, 1.0, total_p)
    return o.permute(0, 2, 1, 3, 4).reshape(b, s["max_q"], h, d)[live].to(torch.bfloat16)


def _plain_sample(s):
    """In 64 bits: a filter's border and the drawn number can lie anywhere between two running sums."""
    z, rows = s["logits"], s["logits"].shape[0]
    ones = torch.ones(rows, device=DEVICE)
    heat = (ones if s["temperature"] is None else s["temperature"]).double()[:, None]
    top_p = (ones if s["top_p"] is None else s["top_p"]).double()[:, None]
    min_p = (0 * ones if s["min_p"] is None else s["min_p"]).double()[:, None]
    top_k = (0 * ones if s["top_k"] is None else s["top_k"]).long()[:, None]
    greedy = heat <= 0
    capped = CAP * torch.tanh(z.double() / CAP) / torch.where(greedy, 1.0, heat)
    w = torch.exp(capped - capped.amax(-1, keepdim=True))
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices
    sorted_w = w.gather(-1, order)
    rank = torch.arange(z.shape[1], device=DEVICE)[None, :]
    sorted_w = torch.where((top_k > 0) & (rank >= top_k), 0.0, sorted_w)
    upto = torch.cumsum(sorted_w, -1)
    keep = (upto - sorted_w < top_p * upto[:, -1:]) | (top_p >= 1) | (rank == 0)
    keep = keep & (sorted_w >= min_p) & (~greedy | (rank == 0))
    kept = torch.zeros_like(w).scatter(-1, order, torch.where(keep, sorted_w, 0.0))
    running = torch.cumsum(kept, -1)
    whole = running[:, -1:]
    idx = torch.searchsorted(running, s["u"].double()[:, None] * whole, right=True)
    prob = kept.gather(-1, idx) / whole
    return {"idx": idx[:, 0].to(torch.int32), "prob": prob[:, 0].float()}


# ------------------------------------------------------------------ in 64 bits, from the definitions


def exact(case, seed):
    return {"append": _exact_append, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](case, seed)


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    t, d, page, r = case["tokens"], case["dim"], case["page"], case["rotated"]
    unit = torch.polar(torch.ones(t, r, dtype=torch.float64, device=DEVICE),
                       s["positions"].double().view(t, 1) * s["freqs"].view(1, r)).view(t, 1, r)
    out = {}
    for name in ("q", "k", "v"):
        x = s[name].double().reshape(t, -1, d)
        if case["norms"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
            if name != "v":
                x = x * s[name + "_norm"].double()
        if name != "v":
            x = x.clone()
            turned = torch.complex(x[..., :r].contiguous(), x[..., d // 2:d // 2 + r].contiguous()) * unit
            x[..., :r], x[..., d // 2:d // 2 + r] = turned.real, turned.imag
        if name == "q":
            out["q"] = x
            continue
        if case["cache"] == "e4m3":
            x = (x / s[name + "_scale"].double().view(1, -1, 1)).clamp(-448, 448)
        cache = s[name + "_cache"].double().transpose(1, 2).reshape(-1, x.shape[1], d)
        cache[s["slots"].long()] = x
        out[name + "_cache"] = cache.view(-1, page, x.shape[1], d).transpose(1, 2).contiguous()
    return out


def _exact_attention(case, seed):
    s = _prepare_attention(case, seed)
    n, d, page, window = case["kv_heads"], case["dim"], case["page"], case["window"]
    group = case["heads"] // n
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    at = 0
    for b, (new, long) in enumerate(zip(*_lengths(case))):
        if not new:
            continue
        low = _first_key(long - new, window)
        pages = s["page_table"][b, low // page:-(-long // page)].long()
        base = low // page * page
        place = torch.arange(long - new, long, device=DEVICE)[:, None]
        j = torch.arange(base, base + pages.numel() * page, device=DEVICE)[None, :]
        hidden = (j > place) | ((j <= place - window) if window else (j < 0))
        for h in range(n):
            k, v = (s[c + "_cache"][:, h].view(torch.uint8 if case["cache"] == "e4m3" else torch.bfloat16)[pages]
                    .view(s[c + "_cache"].dtype).reshape(-1, d).double()
                    * (1.0 if s[c + "_scale"] is None else s[c + "_scale"][h].double()) for c in "kv")
            for g in range(group):
                head = h * group + g
                x = s["q"][at:at + new, head].double() @ k.T
                out[at:at + new, head] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v
        at += new
    return out


def _exact_sample(case, seed):
    s = _prepare_sample(case, seed)
    host = {k: v.double().cpu().numpy() if torch.is_tensor(v) else v for k, v in s.items()}
    ids, probs = [], []
    for r in range(case["rows"]):
        z = host["logits"][r]
        heat, top_k, top_p, min_p = (default if host[name] is None else host[name][r] for name, default in (
            ("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)))
        order = np.argsort(-z, kind="stable")
        if heat <= 0:
            ids.append(int(order[0]))
            probs.append(1.0)
            continue
        x = CAP * np.tanh(z[order] / CAP) / heat
        if top_k > 0:
            order, x = order[:int(top_k)], x[:int(top_k)]
        w = np.exp(x - x[0])
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        stays = (before < top_p * w.sum()) if top_p < 1 else np.ones(len(w), bool)
        stays[0] = True
        stays &= w >= min_p
        order, w = order[stays], w[stays]
        by_index = np.argsort(order)
        order, w = order[by_index], w[by_index]
        running = np.cumsum(w)
        at = min(int(np.searchsorted(running, host["u"][r] * running[-1], side="right")), len(w) - 1)
        ids.append(int(order[at]))
        probs.append(w[at] / running[-1])
    return {"idx": np.array(ids, dtype=np.int32), "prob": np.array(probs)}
