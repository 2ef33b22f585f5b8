"""Child process of test_gpu_debug_serve.py (run with Q4DEC_LIB pointing at
libq4dec_debug.so): calls the serving operators of the debug build in every
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

for cache in ("bf16", "e4m3"):
    kind = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    for n_q, n_kv, D, page, q_lens, kv_lens, window in [
            (8, 2, 256, 64, [1], [700], 512), (8, 1, 512, 64, [1, 1, 1], [5, 4000, 333], 0), (4, 4, 64, 16, [1], [1], 0),
            (32, 8, 128, 128, [7, 3], [900, 64], 0), (8, 2, 256, 32, [64], [3000], 0), (6, 1, 512, 16, [50, 9], [2500, 9], 0),
            (32, 8, 128, 64, [300, 0, 41], [300, 12, 6000], 0), (16, 2, 64, 16, [200], [5000], 700),
            (8, 2, 256, 64, [130, 64], [130, 90], 0), (5, 5, 64, 16, [40] * 70, list(range(40, 110)), 0)]:
        print("case", cache, n_q, n_kv, D, len(q_lens), max(kv_lens), window, flush=True)
        T, width = sum(q_lens), -(-max(kv_lens) // page)
        kc, vc = (torch.zeros(len(q_lens) * width, n_kv, page, D, device=dev).to(kind) for _ in "kv")
        table = torch.randperm(len(q_lens) * width, generator=gen, device=dev).int().view(len(q_lens), width)
        # every key is stored by the append
        q = None
        for b, long in enumerate(kv_lens):
            x = torch.randn(long, (n_q + 2 * n_kv) * D, generator=gen, device=dev) * 0.5
            pos = torch.arange(long, device=dev)
            slots = (table[b, pos // page].long() * page + pos % page).int()
            freqs = 1e4 ** (-torch.arange(D // 4, dtype=torch.float64, device=dev) / (D // 4))
            got = q4.kv_append_rope(x[:, :n_q * D], x[:, n_q * D:(n_q + n_kv) * D], x[:, (n_q + n_kv) * D:], pos.int(),
                                    slots, kc, vc, freqs, v_norm=True)
            q = got[long - q_lens[b]:] if q is None else torch.cat([q, got[long - q_lens[b]:]])
        starts = ints([0] + torch.tensor(q_lens).cumsum(0).tolist())
        y = q4.paged_attention(q.contiguous(), kc, vc, table, starts, ints(kv_lens), max(q_lens), max(kv_lens),
                               scale=D ** -0.5, window=window)
        # the last row of each sequence, plainly
        for b, long in enumerate(kv_lens):
            if not q_lens[b]:
                continue
            pos = torch.arange(max(0, long - window) if window else 0, long, device=dev)
            rows = [c.float()[table[b, pos // page].long(), :, pos % page].repeat_interleave(n_q // n_kv, 1) for c in (kc, vc)]
            at = int(starts[b + 1]) - 1
            p = torch.softmax((rows[0] * q[at].float()).sum(-1) * D ** -0.5, 0)
            want = (p[..., None] * rows[1]).sum(0)
            # 2^-8 of the value for its rounding; 2^-8 of the largest value for the probabilities'
            close = close and bool(((y[at].float() - want).abs() <= 2.0 ** -8 * (want.abs() + rows[1].abs().amax(0)) + 1e-5).all())

for B, V in [(1, 262144), (3, 100003), (5, 1), (2, 257), (64, 1000), (7, 1 << 20)]:
    print("case sample", B, V, flush=True)
    z = torch.randn(B, V, generator=gen, device=dev) * 3
    u = torch.rand(B, generator=gen, device=dev)
    full = lambda v, t=torch.float32: torch.full((B,), v, dtype=t, device=dev)  # noqa: E731
    for kw in ({}, dict(top_k=full(64, torch.int32), top_p=full(0.9)), dict(top_p=full(0.95), min_p=full(0.01)),
               dict(top_k=full(5000, torch.int32)), dict(temperature=full(0.0))):
        idx, prob = q4.sample_logits(z, u, **kw)
        close = close and bool(((idx >= 0) & (idx < V) & (prob > 0) & (prob <= 1)).all())

torch.cuda.synchronize()
out["after_calls"] = list(q4.debug_status())
out["close"] = close
print(json.dumps(out), flush=True)
