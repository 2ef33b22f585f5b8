"""Child process of test_gpu_debug_rollout.py (run with Q4DEC_LIB pointing at
libq4dec_debug.so): calls the rollout operators of the debug build in every
variant and over ragged sizes, then reports the launch-contract words as one
JSON line. Not collected by pytest (no test_ prefix)."""
import json

import torch

import int4_weight_only_block_amd as q4

dev = torch.device("cuda:0")
out = {"lib": q4.LIB_PATH, "start": list(q4.debug_status())}
gen = torch.Generator(device=dev)
gen.manual_seed(7)
ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
close = True
loose = 1 << 19  # under this bound every call shares

for cache in ("bf16", "e4m3"):
    kind = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    for n_q, n_kv, D, page, groups, new in [
            (8, 2, 256, 64, [4], 1), (8, 2, 256, 32, [17, 9], 1), (8, 1, 512, 16, [3], 2), (8, 1, 512, 64, [24, 2], 1),
            (32, 8, 128, 128, [16], 5), (4, 4, 128, 16, [5], 1), (8, 2, 64, 16, [40, 3, 30], 1), (4, 2, 64, 64, [3], 2)]:
        print("case", cache, n_q, n_kv, D, groups, new, flush=True)
        n = sum(groups) + 2  # two of no group
        shared, lens, starts = [], [], [0]
        for g, members in enumerate(groups):
            shared.append(700 - 93 * g)
            lens += [shared[-1] + new + 11 * i for i in range(members)]
            starts.append(starts[-1] + members)
        lens += [new, 300]
        width = loose // page + 1
        kc, vc = ((torch.randn(200, n_kv, page, D, generator=gen, device=dev) * 0.5).to(kind) for _ in "kv")
        table = torch.randint(0, 200, (n, -(-max(lens) // page)), generator=gen, device=dev).int()
        for g in range(len(groups)):
            table[starts[g]:starts[g + 1], :-(-shared[g] // page)] = table[starts[g], :-(-shared[g] // page)].clone()
        table = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1).contiguous()
        q = (torch.randn(n * new, n_q, D, generator=gen, device=dev)).bfloat16()
        at = ints(list(range(0, n * new + 1, new)))
        y = q4.paged_attention_shared(q, kc, vc, table, at, ints(lens), ints(starts), ints(shared), new, loose, loose, D ** -0.5)
        want = q4.paged_attention(q, kc, vc, table, at, ints(lens), new, max(lens), D ** -0.5)
        # each is off by 2^-8 of its value, and by 2^-8 of the largest value for its probabilities
        slack = 2.0 ** -7 * (want.abs().float() + vc.float().abs().amax())
        close = close and bool(((y.float() - want.float()).abs() <= slack).all())

for B, drafts, V in [(1, 3, 262144), (3, 5, 100003), (5, 1, 1), (2, 4, 257), (64, 2, 1000), (2, 1, 1 << 20), (3, 70, 5000)]:
    print("case verify", B, drafts, V, flush=True)
    T = B * (drafts + 1)
    z = torch.randn(T, V, generator=gen, device=dev) * 3
    zd = z + torch.randn(T, V, generator=gen, device=dev) * 0.3
    full = lambda v, t=torch.float32: torch.full((B,), v, dtype=t, device=dev)  # noqa: E731
    at = ints(list(range(0, T + 1, drafts + 1)))
    for kw in ({}, dict(top_k=full(64, torch.int32), top_p=full(0.9)), dict(top_p=full(0.95), min_p=full(0.01)),
               dict(top_k=full(5000, torch.int32)), dict(temperature=full(0.0))):
        tokens, prob, count = q4.verify_drafts(z, torch.argmax(zd, -1).int(), at, torch.rand(T, generator=gen, device=dev),
                                               torch.rand(B, generator=gen, device=dev), draft_logits=zd, **kw)
        kept = torch.arange(drafts + 1, device=dev)[None] < count[:, None]
        tokens, prob = tokens.view(B, -1), prob.view(B, -1)
        close = close and bool(((count >= 1) & (count <= drafts + 1)).all()) and bool(
            ((tokens >= 0) == kept).all() and (tokens < V).all() and (prob[kept] > 0).all() and (prob[~kept] == 0).all())

torch.cuda.synchronize()
out["after_calls"] = list(q4.debug_status())
out["close"] = close
print(json.dumps(out), flush=True)
