"""Workloads of two more serving operators: the attention of a batch whose sequences begin with the same
text, and the check of drafted tokens against the target's probabilities.

Every workload can be computed in two ways from the same inputs: in plain torch operations (``own``
false), and by the calls that a program makes of int4_weight_only_block_amd (``own`` true).

A case is a dict of plain values; its "op" is one of

  shared     paged_attention_shared: new tokens of several sequences over their cached keys and values,
             the sequences in groups that share the pages of a common beginning
  verify     verify_drafts: which drafted tokens stay, and the token after them, from the target's and
             the drafter's logits (or drafts without any) and given random numbers, after temperature,
             top-k, top-p and min-p

The head layouts are those of the decoder shapes this library serves (8 query heads over 1 or 2
key/value heads of 256, or of 512 on the layers without a window; a vocabulary of 262144; logits
capped at 30), next to generic ones.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
CAP = 30.0
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a few answers to one short question, sampled side by side
        dict(name="shared_decode_4_1100", op="shared", groups="4", alone=0, chunk=1, shared=1100, own=60, heads=8,
             kv_heads=2, dim=256, cache="bf16", page=64, salt=1),
        # many continuations of one long document: a rollout batch
        dict(name="shared_decode_32_32768", op="shared", groups="32", alone=0, chunk=1, shared=32768, own=700, heads=8,
             kv_heads=2, dim=256, cache="bf16", page=64, salt=2),
        # the same on a layer of 512-wide heads; the text does not end where a page does
        dict(name="shared_decode_24_50001", op="shared", groups="24", alone=0, chunk=1, shared=50001, own=900, heads=8,
             kv_heads=1, dim=512, cache="bf16", page=64, salt=3),
        # a server's decode batch: three system prompts and some requests without one, cache in 8 bits
        dict(name="shared_decode_groups_e4m3", op="shared", groups="21+9+13", alone=3, chunk=1, shared=12000, own=2500,
             heads=8, kv_heads=2, dim=256, cache="e4m3", page=32, salt=4),
        # a speculative check of 4 drafted tokens in 16 requests behind one prompt
        dict(name="shared_verify_16x5", op="shared", groups="16", alone=0, chunk=5, shared=9000, own=1000, heads=32,
             kv_heads=8, dim=128, cache="bf16", page=128, salt=5),
        # the largest: prefill chunks of several requests behind one system prompt
        dict(name="shared_chunk_512_6", op="shared", groups="6", alone=0, chunk=512, shared=8192, own=2000, heads=32,
             kv_heads=8, dim=128, cache="bf16", page=128, salt=6),
        # one request with 3 drafts that a table of earlier texts gave, without probabilities; greedy decoding
        dict(name="verify_1x3_certain_greedy", op="verify", seqs=1, drafts=3, vocab=262144, filters="greedy",
             drafter=False, salt=7),
        # one request with 4 drafts of a drafter, filtered as decoders of this kind are run: top-k 64, top-p 0.95
        dict(name="verify_1x4_topk", op="verify", seqs=1, drafts=4, vocab=262144, filters="topk", drafter=True, salt=8),
        # a few rollouts without a filter: the whole distributions count; an odd vocabulary
        dict(name="verify_5x5_free", op="verify", seqs=5, drafts=5, vocab=100003, filters="free", drafter=True, salt=9),
        # a decode batch whose requests have their own settings and numbers of drafts, some of them none
        dict(name="verify_24x4_mixed", op="verify", seqs=24, drafts=4, vocab=262144, filters="mixed", drafter=True,
             salt=10),
        # a full batch of rollouts without a filter: the most that is read
        dict(name="verify_64x3_free", op="verify", seqs=64, drafts=3, vocab=262144, filters="free", drafter=True,
             salt=11),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    salt = rng.randrange(1 << 30)
    if rng.random() < 0.5:
        dim = rng.choice([64, 128, 256, 512])
        kv_heads = rng.choice([1, 2, 4, 8] if dim <= 128 else [1, 2])
        heads = kv_heads * rng.choice([1, 4, 5, 8])
        kind = rng.choice(["decode", "verify", "chunk"])
        chunk = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 9, 400)
        most = 48 if kind == "decode" else 16 if kind == "verify" else 5
        groups = [_log_int(rng, 2, most) for _ in range(rng.choice([1, 1, 1, 2, 3]))]
        seqs = sum(groups)
        # the products of queries and keys stay under 2**36, the caches of the sequences' own tokens under 2**28 elements
        longest = max(64, min(65536, (1 << 36) // (seqs * chunk * heads * dim)))
        shared = _log_int(rng, 40, longest)
        beside = max(chunk, min(_log_int(rng, 8, 4096), longest, (1 << 28) // (seqs * kv_heads * dim)))
        return dict(op="shared", groups="+".join(map(str, groups)), alone=rng.choice([0, 0, 2]), chunk=chunk, shared=shared, own=beside,
                    heads=heads, kv_heads=kv_heads, dim=dim, cache=rng.choice(["bf16", "e4m3"]),
                    page=rng.choice([16, 32, 64, 128]), salt=salt)
    vocab, drafts = _log_int(rng, 1000, 262144), rng.randint(1, 7)
    seqs = _log_int(rng, 1, max(1, min(64, (1 << 26) // (vocab * (drafts + 1)))))
    return dict(op="verify", seqs=seqs, drafts=drafts, vocab=vocab, filters=rng.choice(["greedy", "topk", "free", "mixed"]),
                drafter=rng.random() < 0.75, salt=salt)


def _groups(case):
    """The number of sequences in each group."""
    return [int(x) for x in case["groups"].split("+")]


def _lengths(case):
    """Of a shared case: (new tokens, cached tokens, shared tokens) of each sequence and its group, -1 for
    one that shares nothing. The first group has the longest beginning."""
    rng = random.Random(case["salt"])
    groups = _groups(case)
    q, kv, shared, group = [], [], [], []
    for g, members in enumerate(groups + [1] * case["alone"]):
        common = case["shared"] if g == 0 else _log_int(rng, max(1, case["shared"] // 5), case["shared"])
        for i in range(members):
            q.append(case["chunk"] if i == 0 else rng.randint(1, case["chunk"]))
            kv.append(common + q[-1] + rng.randint(0, max(0, case["own"] - q[-1])))
            shared.append(common if g < len(groups) else 0)
            group.append(g if g < len(groups) else -1)
    return q, kv, shared, group


def _rows(case):
    """Of a verify case: rows of logits of each sequence, one more than its drafts."""
    rng = random.Random(case["salt"])
    if case["filters"] != "mixed":
        return [case["drafts"] + 1] * case["seqs"]
    return [case["drafts"] + 1 if b == 0 else rng.randint(0, case["drafts"]) + 1 for b in range(case["seqs"])]


def work(case):
    if case["op"] == "shared":
        q, kv, shared, group = _lengths(case)
        stored = 2 if case["cache"] == "bf16" else 1
        keys = sum(long - common for long, common in zip(kv, shared))
        keys += sum({g: common for g, common in zip(group, shared) if g >= 0}.values())
        pairs = sum(new * long - new * (new - 1) // 2 for new, long in zip(q, kv))
        return {"bytes": 2 * stored * keys * case["kv_heads"] * case["dim"]
                + 4 * sum(q) * case["heads"] * case["dim"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    rows = _rows(case)
    n = (sum(rows) + (sum(rows) - len(rows) if case["drafter"] else 0)) * case["vocab"]
    return {"bytes": 4 * n + 16 * sum(rows) + 32 * len(rows), "flops": 8 * n}


# ------------------------------------------------------------------ inputs


def _generator(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 1000003 + case["salt"] % 999983)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32).to(DEVICE)


def prepare(case, seed):
    return {"shared": _prepare_shared, "verify": _prepare_verify}[case["op"]](case, seed)


def _prepare_shared(case, seed):
    g = _generator(case, seed)
    h, n, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    q_lens, kv_lens, shared, group = _lengths(case)
    widths = [-(-long // page) for long in kv_lens]
    table = torch.full((len(widths), max(widths)), -1, dtype=torch.int64)
    used, rewritten = 0, []
    for b, w in enumerate(widths):
        # a group's full common pages are the first member's; the page that the common text ends in is each one's own
        follows = b > 0 and group[b] >= 0 and group[b] == group[b - 1]
        common = shared[b] // page if follows else 0
        if follows:
            table[b, :common] = table[b - 1, :common]
            if shared[b] % page:
                rewritten.append((used, int(table[b - 1, common])))
        table[b, common:w] = torch.arange(used, used + w - common)
        used += w - common
    pages = used + 2
    order = torch.randperm(pages, generator=g, device=DEVICE).cpu()
    table = torch.where(table >= 0, order[table.clamp(min=0)], -1).to(torch.int32)
    q_starts = [0] + [int(x) for x in np.cumsum(q_lens)]
    starts, lens = [0], []
    for members in _groups(case):
        lens.append(shared[starts[-1]])
        starts.append(starts[-1] + members)
    s = {"case": case, "k_scale": None, "v_scale": None,
         "q": (_normal(g, sum(q_lens), h, d) * (2.5 / math.sqrt(d))).to(torch.bfloat16),
         "page_table": table.to(DEVICE), "q_starts": _ints(q_starts), "kv_lens": _ints(kv_lens),
         "group_starts": _ints(starts), "shared_lens": _ints(lens),
         "max_q": max(q_lens), "max_kv": max(kv_lens), "max_shared": max(lens), "ws": None}
    for name in ("k_cache", "v_cache"):
        x = _normal(g, pages, n, page, d)
        if case["cache"] == "e4m3":
            s[name[0] + "_scale"] = 0.01 + 0.02 * _uniform(g, n)
            x = (x / s[name[0] + "_scale"].view(1, n, 1, 1)).clamp(-448, 448)
        x = x.to(torch.bfloat16 if case["cache"] == "bf16" else E4M3)
        raw = x.view(torch.int16 if case["cache"] == "bf16" else torch.uint8)
        for to, fr in rewritten:  # the common text's last page, copied where a sequence writes on in it
            raw[int(order[to])] = raw[int(order[fr])]
        s[name] = x
    if own:  # a serving loop keeps one workspace for all its layers and steps
        import int4_weight_only_block_amd as q4
        s["ws"] = torch.empty(q4.paged_attention_shared_workspace_bytes(
            sum(q_lens), len(q_lens), len(lens), h, n, d, s["max_q"], s["max_kv"], s["max_shared"]),
            dtype=torch.uint8, device=DEVICE)
    return s


def _prepare_verify(case, seed):
    g = _generator(case, seed)
    rows, v = _rows(case), case["vocab"]
    t, b = sum(rows), len(rows)
    # a broad floor with a few dozen plausible tokens above it, and a drafter that differs from it a little
    logits = 2.5 * _normal(g, t, v) - 4.0
    some = torch.randint(0, v, (t, 40), generator=g, device=DEVICE)
    logits.scatter_add_(1, some, 12.0 * _uniform(g, t, 40) ** 2 + 4.0)
    drafter = logits + 0.6 * _normal(g, t, v)
    s = {"case": case, "starts": _ints([0] + [int(x) for x in np.cumsum(rows)]), "u": _uniform(g, t),
         "u_draw": _uniform(g, b), "temperature": None, "top_k": None, "top_p": None, "min_p": None, "ws": None}
    pick = lambda values, kind: torch.tensor(values, dtype=kind, device=DEVICE)[  # noqa: E731
        torch.randint(0, len(values), (b,), generator=g, device=DEVICE)]
    if case["filters"] == "greedy":
        s["temperature"] = pick([0.0], torch.float32)
    elif case["filters"] == "topk":
        s["temperature"], s["top_k"] = pick([1.0], torch.float32), pick([64], torch.int32)
        s["top_p"] = pick([0.95], torch.float32)
    elif case["filters"] == "free":
        s["temperature"] = pick([1.0], torch.float32)
    else:
        s["temperature"] = pick([0.0, 0.3, 0.7, 1.0, 1.0, 1.4], torch.float32)
        s["top_k"] = pick([0, 0, 1, 20, 64, 1000], torch.int32)
        s["top_p"] = pick([1.0, 0.95, 0.9, 0.5], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.02, 0.1], torch.float32)
        # a grammar forbids a third of the tokens in some rows, to the target and the drafter alike
        masked = (_uniform(g, t, 1) < 0.25) & (_uniform(g, t, v) < 0.33)
        logits.masked_fill_(masked, -math.inf)
        drafter.masked_fill_(masked, -math.inf)
    # the drafts are drawn as the drafter's distribution has them
    kept = _weights(drafter, s)
    running = torch.cumsum(kept, -1)
    at = torch.searchsorted(running, _uniform(g, t, 1).double() * running[:, -1:], right=True)
    s["drafts"] = at[:, 0].clamp(max=v - 1).to(torch.int32)
    s["logits"], s["draft_logits"] = logits, drafter if case["drafter"] else None
    if own:
        import int4_weight_only_block_amd as q4
        s["ws"] = torch.empty(q4.verify_drafts_workspace_bytes(t, b, v, case["drafter"]), dtype=torch.uint8,
                              device=DEVICE)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        import int4_weight_only_block_amd as q4
        if s["case"]["op"] == "shared":
            return q4.paged_attention_shared(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_starts"],
                                             s["kv_lens"], s["group_starts"], s["shared_lens"], s["max_q"], s["max_kv"],
                                             s["max_shared"], scale=1.0, k_scale=s["k_scale"], v_scale=s["v_scale"],
                                             ws=s["ws"])
        tokens, prob, count = q4.verify_drafts(s["logits"], s["drafts"], s["starts"], s["u"], s["u_draw"],
                                               draft_logits=s["draft_logits"], temperature=s["temperature"],
                                               top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], cap=CAP, ws=s["ws"])
        return {"tokens": tokens, "prob": prob, "count": count}
    return {"shared": _plain_shared, "verify": _plain_verify}[s["case"]["op"]](s)


def _pages(cache, at, scale):
    """Pages `at` [..., W] of the cache as [..., kv_heads, tokens, D] in 32 bits."""
    n, page, d = cache.shape[1:]
    at = at.clamp(min=0).long()
    x = cache.view(torch.uint8)[at].view(E4M3).float() if cache.dtype == E4M3 else cache[at].float()
    if scale is not None:
        x = x * scale.view(n, 1, 1)
    return x.movedim(-3, -4).reshape(*at.shape[:-1], n, at.shape[-1] * page, d)


def _plain_shared(s):
    """The common beginnings once per group, the rest once per sequence; one softmax over both."""
    case = s["case"]
    h, n, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    group, total, max_q = h // n, s["q"].shape[0], s["max_q"]
    starts, kv_lens = s["q_starts"].long(), s["kv_lens"].long()
    q_lens = starts[1:] - starts[:-1]
    b = kv_lens.numel()
    q_lens_host, kv_host, shared_host, group_host = _lengths(case)  # a server has these on the host as well
    shared = torch.tensor(shared_host, device=DEVICE)
    i = torch.arange(max_q, device=DEVICE)
    live = i[None, :] < q_lens[:, None]
    token = (starts[:-1, None] + i[None, :]).clamp(max=total - 1)
    q = s["q"][token].float().view(b, max_q, n, group, d).permute(0, 2, 1, 3, 4).reshape(b, n, max_q * group, d)
    # each sequence's own part, from the page that the shared part ends in
    wide = max(-(-long // page) - common // page for long, common in zip(kv_host, shared_host))
    at = (shared // page)[:, None] + torch.arange(wide, device=DEVICE)[None, :]
    table = s["page_table"].gather(1, at.clamp(max=s["page_table"].shape[1] - 1))
    k, v = _pages(s["k_cache"], table, s["k_scale"]), _pages(s["v_cache"], table, s["v_scale"])
    scores = torch.matmul(q, k.transpose(-1, -2)).view(b, n, max_q, group, -1)
    j = (shared // page * page)[:, None] + torch.arange(wide * page, device=DEVICE)[None, :]
    place = (kv_lens - q_lens)[:, None] + i[None, :]
    seen = (j[:, None, :] <= place[..., None]) & (j >= shared[:, None])[:, None, :]
    scores = scores.masked_fill(~seen[:, None, :, None, :], -math.inf).view(b, n, max_q * group, -1)
    top = scores.amax(-1, keepdim=True)
    common, first = [], 0
    for members in _groups(case):
        length = shared_host[first]
        at = s["page_table"][first, :-(-length // page)]
        ks, vs = (_pages(s[c + "_cache"], at, s[c + "_scale"])[:, :length] for c in "kv")
        rows = q[first:first + members].transpose(0, 1).reshape(n, -1, d)
        x = torch.matmul(rows, ks.transpose(-1, -2))
        common.append((first, members, x, vs))
        most = x.amax(-1).view(n, members, -1, 1).transpose(0, 1)
        top[first:first + members] = torch.maximum(top[first:first + members], most)
        first += members
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    whole, o = p.sum(-1, keepdim=True), torch.matmul(p, v)
    for first, members, x, vs in common:
        p = torch.exp(x - top[first:first + members].transpose(0, 1).reshape(n, -1, 1))
        whole[first:first + members] += p.sum(-1, keepdim=True).view(n, members, -1, 1).transpose(0, 1)
        o[first:first + members] += torch.matmul(p, vs).view(n, members, -1, d).transpose(0, 1)
    o = (o / torch.where(whole == 0, 1.0, whole)).view(b, n, max_q, group, d)
    return o.permute(0, 2, 1, 3, 4).reshape(b, max_q, h, d)[live].to(torch.bfloat16)


def _weights(z, s):
    """Of each row of logits, in 64 bits: the weights of the tokens that its sequence's filters leave."""
    rows, b = z.shape[0], s["starts"].numel() - 1
    lengths = (s["starts"][1:] - s["starts"][:-1]).long()
    owner = torch.repeat_interleave(torch.arange(b, device=DEVICE), lengths, output_size=rows)
    of = lambda name, off: (torch.full((b,), off, device=DEVICE) if s[name] is None else s[name])[owner][:, None]  # noqa: E731
    heat, top_k, top_p = of("temperature", 1.0).double(), of("top_k", 0).long(), of("top_p", 1.0).double()
    greedy = heat <= 0
    capped = CAP * torch.tanh(z.double() / CAP) / torch.where(greedy, 1.0, heat)
    w = torch.exp(torch.where(z == -math.inf, -math.inf, capped - capped.amax(-1, keepdim=True)))
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices
    sorted_w = w.gather(-1, order)
    rank = torch.arange(z.shape[1], device=DEVICE)[None, :]
    sorted_w = torch.where((top_k > 0) & (rank >= top_k), 0.0, sorted_w)
    upto = torch.cumsum(sorted_w, -1)
    keep = (upto - sorted_w < top_p * upto[:, -1:]) | (top_p >= 1) | (rank == 0)
    keep = keep & (sorted_w >= of("min_p", 0.0).double()) & (~greedy | (rank == 0))
    return torch.zeros_like(w).scatter(-1, order, torch.where(keep, sorted_w, 0.0))


def _plain_verify(s):
    """In 64 bits: a filter's border and the drawn number can lie anywhere between two running sums."""
    starts = s["starts"].long()
    first, last = starts[:-1], starts[1:] - 1
    rows, vocab = s["logits"].shape
    at = s["drafts"].long()[:, None]
    p = _weights(s["logits"], s)
    p = p / p.sum(-1, keepdim=True)
    p_draft = p.gather(-1, at)[:, 0]
    if s["draft_logits"] is None:
        q, q_draft = None, torch.ones_like(p_draft)
    else:
        q = _weights(s["draft_logits"], s)
        q = q / q.sum(-1, keepdim=True)
        q_draft = q.gather(-1, at)[:, 0]
    rejected = ~(s["u"].double() * q_draft < p_draft)
    rejected[last] = True  # no draft there
    row = torch.arange(rows, device=DEVICE)
    stop = torch.where(rejected, row, rows)  # the first rejected row from each row on
    stop = torch.flip(torch.cummin(torch.flip(stop, [0]), 0).values, [0])[first]
    taken = stop - first
    rest = p[stop]
    checked = (stop < last)[:, None]
    if q is None:
        away = torch.zeros_like(rest).scatter(-1, at[stop], 1.0)
    else:
        away = q[stop]
    rest = torch.where(checked, (rest - away).clamp(min=0.0), rest)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p[stop])
    running = torch.cumsum(rest, -1)
    new = torch.searchsorted(running, s["u_draw"].double()[:, None] * running[:, -1:], right=True)
    owner = torch.repeat_interleave(torch.arange(first.numel(), device=DEVICE), last + 1 - first, output_size=rows)
    tokens = torch.where(row < stop[owner], s["drafts"].long(), -1)
    prob = torch.where(row < stop[owner], p_draft, 0.0)
    tokens[stop], prob[stop] = new[:, 0], p[stop].gather(-1, new)[:, 0]
    return {"tokens": tokens.to(torch.int32), "prob": prob.float(), "count": (taken + 1).to(torch.int32)}


# ------------------------------------------------------------------ in 64 bits, from the definitions


def exact(case, seed):
    return {"shared": _exact_shared, "verify": _exact_verify}[case["op"]](case, seed)


def _exact_shared(case, seed):
    """Each sequence for itself, as if nothing were shared."""
    s = _prepare_shared(case, seed)
    n, d = case["kv_heads"], case["dim"]
    group, page = case["heads"] // n, case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    at = 0
    q_lens, kv_lens, _, _ = _lengths(case)
    for b, (new, long) in enumerate(zip(q_lens, kv_lens)):
        pages = s["page_table"][b, :-(-long // page)].long()
        hidden = torch.arange(long, device=DEVICE)[None, :] > torch.arange(long - new, long, device=DEVICE)[:, None]
        for h in range(n):
            k, v = (s[c + "_cache"][:, h].view(torch.uint8 if case["cache"] == "e4m3" else torch.bfloat16)[pages]
                    .view(s[c + "_cache"].dtype).reshape(-1, d)[:long].double()
                    * (1.0 if s[c + "_scale"] is None else s[c + "_scale"][h].double()) for c in "kv")
            for g in range(group):
                x = s["q"][at:at + new, h * group + g].double() @ k.T
                out[at:at + new, h * group + g] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v
        at += new
    return out


def _exact_verify(case, seed):
    if (sum(_rows(case)) * (2 if case["drafter"] else 1)) * case["vocab"] > 60 * 262144:
        return None  # sorted on the host: too long
    s = _prepare_verify(case, seed)
    host = {k: v.double().cpu().numpy() if torch.is_tensor(v) else v for k, v in s.items()}

    def distribution(z, b):
        heat, top_k, top_p, min_p = (off if host[name] is None else host[name][b] for name, off in (
            ("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)))
        out = np.zeros(len(z))
        order = np.argsort(-z, kind="stable")
        if heat <= 0:
            out[order[0]] = 1.0
            return out
        order = order[z[order] > -np.inf]
        if top_k > 0:
            order = order[:int(top_k)]
        x = CAP * np.tanh(z[order] / CAP) / heat
        w = np.exp(x - x[0])
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        stays = (before < top_p * w.sum()) if top_p < 1 else np.ones(len(w), bool)
        stays[0] = True
        stays &= w >= min_p
        out[order[stays]] = w[stays] / w[stays].sum()
        return out

    tokens, probs, counts, start = [], [], [], 0
    for b, rows in enumerate(_rows(case)):
        got, of = [], []
        for i in range(rows):
            p = distribution(host["logits"][start + i], b)
            rest = p
            if i + 1 < rows:
                x = int(host["drafts"][start + i])
                q = np.zeros(len(p))
                if host["draft_logits"] is None:
                    q[x] = 1.0
                else:
                    q = distribution(host["draft_logits"][start + i], b)
                if host["u"][start + i] * q[x] < p[x]:
                    got.append(x)
                    of.append(p[x])
                    continue
                rest = np.maximum(p - q, 0.0)
                if rest.sum() <= 0:
                    rest = p
            running = np.cumsum(rest)
            new = min(int(np.searchsorted(running, host["u_draw"][b] * running[-1], side="right")), len(p) - 1)
            got.append(new)
            of.append(p[new])
            break
        counts.append(len(got))
        tokens += got + [-1] * (rows - len(got))
        probs += of + [0.0] * (rows - len(of))
        start += rows
    return {"tokens": np.array(tokens, dtype=np.int32), "prob": np.array(probs), "count": np.array(counts, dtype=np.int32)}
