"""The serving operators (cache append, paged attention, sampling) on the GPU
against their fp64 oracle. Tolerances count the roundings of the definitions
(see serve_oracle.attention_tolerance); half a step of bf16 is 2^-8 of the
value, of e4m3 2^-4 (2^-10 below its smallest normal)."""
import math

import numpy as np
import pytest
import torch

import int4_weight_only_block_amd as q4
import oracle
import synth
from oracle import serve_oracle as so

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def f64(t):
    """The values of a tensor (bf16, e4m3, fp32) as float64 numpy."""
    if t.dtype == E4M3:
        return so.e4m3_values()[t.contiguous().view(torch.uint8).cpu().numpy()]
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ append

APPEND = [
    # T, n_q, n_kv, D, rot_dim, n_freqs, cache, page, norms, far
    (1, 8, 2, 256, 256, 128, "bf16", 64, True, 5000),
    (1, 8, 1, 512, 512, 64, "e4m3", 16, True, 131072),
    (7, 5, 1, 64, 64, 32, "bf16", 16, False, 100),
    (33, 4, 4, 128, 64, 20, "e4m3", 32, True, 1 << 30),
    (129, 3, 3, 128, 128, 64, "bf16", 4096, True, 3000),
    (50, 12, 2, 64, 2, 1, "e4m3", 128, False, 70),
    (5, 8, 2, 512, 510, 255, "bf16", 64, True, 1 << 20),
    (600, 1, 1, 256, 256, 0, "bf16", 32, True, 9),
    (300, 16, 8, 64, 64, 32, "e4m3", 64, True, 4000),
]


def append_inputs(T, n_q, n_kv, D, n_freqs, cache, page, norms, far, seed):
    g = generator(seed)
    fused = torch.randn(T, (n_q + 2 * n_kv) * D + 12, generator=g, device=DEV) * 2
    q, k, v = fused[:, :n_q * D], fused[:, n_q * D:(n_q + n_kv) * D], fused[:, (n_q + n_kv) * D:(n_q + 2 * n_kv) * D]
    pages = -(-T // page) + 2
    kinds = torch.bfloat16 if cache == "bf16" else E4M3
    caches = [torch.randn(pages, n_kv, page, D, generator=g, device=DEV).to(kinds) for _ in "kv"]
    kw = dict(eps=1e-5)
    if norms:
        kw.update(q_norm=torch.rand(D, generator=g, device=DEV) + 0.5, k_norm=torch.rand(D, generator=g, device=DEV) + 0.5,
                  v_norm=True)
    if cache == "e4m3":
        kw.update(k_scale=torch.rand(n_kv, generator=g, device=DEV) * 0.02 + 0.005,
                  v_scale=torch.rand(n_kv, generator=g, device=DEV) * 0.02 + 0.002)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].int()
    positions = torch.randint(0, far, (T,), generator=g, device=DEV).int()
    freqs = 1e4 ** (-torch.arange(n_freqs, dtype=torch.float64, device=DEV) / max(n_freqs, 1))
    return q, k, v, positions, slots, caches, freqs, kw


@pytest.mark.parametrize("T,n_q,n_kv,D,rot,n_freqs,cache,page,norms,far", APPEND)
def test_append_against_oracle(T, n_q, n_kv, D, rot, n_freqs, cache, page, norms, far):
    q, k, v, positions, slots, caches, freqs, kw = append_inputs(T, n_q, n_kv, D, n_freqs, cache, page, norms, far, T)
    was = [c.clone() for c in caches]
    err = flag()
    out = q4.kv_append_rope(q, k, v, positions, slots, *caches, freqs, rot_dim=rot, err_flag=err, **kw)
    assert err.item() == 0
    host = [f64(x).reshape(T, -1, D) for x in (q, k, v)]
    norm = dict(q_norm=f64(kw["q_norm"]), k_norm=f64(kw["k_norm"]), v_norm=True) if norms else {}
    want = so.append(*host, positions.cpu().numpy(), f64(freqs), rot // 2, eps=1e-5, **norm)
    # before its last rounding: sums of squares, norm, weight, two products and their sum, with sin and cos
    # off by a few 2^-24 each; no more than 64 roundings of the pair's size (at most sqrt(2) of a row's largest)
    inner = [64 * 2.0 ** -24 * np.abs(w).max(-1, keepdims=True) * 1.5 for w in want]
    assert (np.abs(f64(out) - want[0]) <= 2.0 ** -8 * np.abs(want[0]) * (1 + 2.0 ** -8) + inner[0]).all()
    at = slots.cpu().numpy()
    for name, cache_t, old, w, slack in zip("kv", caches, was, want[1:], inner[1:]):
        flat = f64(cache_t).transpose(0, 2, 1, 3).reshape(-1, n_kv, D)
        if cache == "bf16":
            ok = np.abs(flat[at] - w) <= 2.0 ** -8 * np.abs(w) * (1 + 2.0 ** -8) + slack
        else:
            s = f64(kw[name + "_scale"])[None, :, None]
            w = np.clip(w / s, -448, 448)
            ok = np.abs(flat[at] - w) <= np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10) * 1.001 + slack / s
        assert ok.all()
        rest = np.ones(flat.shape[0], bool)
        rest[at] = False
        kept = bits(cache_t).reshape(*cache_t.shape[:3], -1).transpose(0, 2, 1, 3).reshape(flat.shape[0], -1)
        had = bits(old).reshape(*cache_t.shape[:3], -1).transpose(0, 2, 1, 3).reshape(flat.shape[0], -1)
        assert np.array_equal(kept[rest], had[rest])


def test_append_padding_bad_slots_and_parts():
    q, k, v, positions, slots, caches, freqs, kw = append_inputs(6, 4, 2, 128, 64, "bf16", 16, True, 50, 3)
    full = [c.clone() for c in caches]
    whole = q4.kv_append_rope(q, k, v, positions, slots, *full, freqs, **kw)
    # only q; only k and v; rows as [T, heads, D]; both give what the whole call gives
    only_q = q4.kv_append_rope(q, None, None, positions, None, None, None, freqs, head_dim=128, q_norm=kw["q_norm"],
                               eps=1e-5)
    assert torch.equal(only_q, whole)
    part = [c.clone() for c in caches]
    kw_kv = {n: kw[n] for n in ("k_norm", "v_norm", "eps")}
    k3, v3 = k.contiguous().view(6, 2, 128), v.contiguous().view(6, 2, 128)
    assert q4.kv_append_rope(None, k3, v3, positions, slots, *part, freqs, **kw_kv) is None
    assert torch.equal(part[0], full[0]) and torch.equal(part[1], full[1])
    # padded tokens are not stored and set no flag; slots past the end are not stored and set it
    for bad, want in ((-1, 0), (-(1 << 31), 0), (caches[0].shape[0] * 16, 1), ((1 << 31) - 1, 1)):
        s2, err, got = slots.clone(), flag(), [c.clone() for c in caches]
        s2[4] = bad
        out = q4.kv_append_rope(q, k, v, positions, s2, *got, freqs, err_flag=err, **kw)
        assert err.item() == want and torch.equal(out, whole)
        at = int(slots[4])
        for g, f, c in zip(got, full, caches):
            f = f.clone()
            f[at // 16, :, at % 16] = c[at // 16, :, at % 16]
            assert torch.equal(g, f)


def test_empty_calls():
    """No tokens, no rows, no sequences: nothing is done, and what comes back is empty."""
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    x = torch.zeros(0, 8 * 64, device=DEV)
    caches = [torch.ones(2, 2, 16, 64, device=DEV).bfloat16() for _ in "kv"]
    freqs = torch.ones(32, dtype=torch.float64, device=DEV)
    assert q4.kv_append_rope(x, x[:, :128], x[:, 128:256], i, i, *caches, freqs).shape == (0, 8, 64)
    assert q4.kv_append_rope(None, x[:, :128], x[:, 128:256], i, i, *caches, freqs) is None
    assert q4.kv_append_rope(x, None, None, i, None, None, None, freqs, head_dim=64).shape == (0, 8, 64)
    q = torch.zeros(0, 8, 64, device=DEV).bfloat16()
    table, two = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    assert q4.paged_attention(q, *caches, table, two, two[:2], 1, 16).shape == (0, 8, 64)
    assert q4.paged_attention(q, *caches, table[:0], two[:1], two[:0], 1, 16).shape == (0, 8, 64)
    idx, prob = q4.sample_logits(torch.zeros(0, 100, device=DEV), torch.zeros(0, device=DEV))
    assert idx.shape == prob.shape == (0,)
    torch.cuda.synchronize()
    assert all((c == 1).all() for c in caches)


def test_append_e4m3_saturates_and_keeps_nan():
    D = 64
    x = torch.zeros(1, 2 * D, device=DEV)
    x[0, :6] = torch.tensor([1e30, -1e30, math.inf, -math.inf, math.nan, 2.0 ** -10 * 0.01])
    c = [torch.zeros(1, 2, 16, D, device=DEV).to(E4M3) for _ in "kv"]
    scale = torch.full((2,), 0.01, device=DEV)
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    q4.kv_append_rope(None, x, x, i, i, *c, None, rot_dim=2, k_scale=scale, v_scale=scale)
    for t in c:
        got = f64(t)[0, 0, 0, :6]
        # 2^-10 is halfway between 0 and the smallest subnormal: ties go to even
        assert list(got[:4]) == [448, -448, 448, -448] and np.isnan(got[4]) and got[5] == 0


# ------------------------------------------------------------------ attention

# q_lens, kv_lens, n_q, n_kv, D, page, cache, window
ATTENTION = [
    ([1], [1], 8, 2, 256, 64, "bf16", 0),
    ([1], [17], 8, 1, 512, 16, "bf16", 0),
    ([1], [700], 8, 2, 256, 64, "bf16", 512),
    ([1], [5000], 4, 2, 64, 32, "bf16", 0),
    ([1], [5000], 8, 2, 128, 128, "e4m3", 0),
    ([1] * 9, [1, 2, 15, 16, 17, 63, 64, 65, 1000], 8, 2, 256, 16, "bf16", 0),
    ([1] * 5, [300, 1, 900, 33, 512], 8, 1, 512, 64, "e4m3", 100),
    ([1, 0, 1, 0], [40, 80, 90, 0], 5, 1, 128, 32, "bf16", 0),
    ([1, 1], [3000, 64], 16, 1, 128, 64, "bf16", 7),
    ([1], [129], 64, 1, 64, 16, "e4m3", 0),
    ([1], [260], 3, 3, 512, 4096, "bf16", 0),
    ([4, 4, 4], [4, 100, 777], 8, 2, 256, 64, "bf16", 0),
    ([2, 8, 5], [900, 8, 64], 8, 1, 512, 32, "e4m3", 50),
    ([3], [2], 4, 4, 128, 16, "bf16", 0),        # the first row sees nothing
    ([9], [5], 2, 1, 64, 16, "bf16", 3),         # so do several, with a window
    ([7], [600], 12, 4, 64, 64, "bf16", 1),      # each sees itself alone
    ([64], [64], 8, 2, 256, 64, "bf16", 0),
    ([64], [2000], 8, 2, 256, 64, "bf16", 512),
    ([64, 1, 13, 100], [3000, 500, 13, 133], 8, 1, 512, 64, "bf16", 0),
    ([37, 0, 130], [1037, 10, 130], 8, 2, 128, 16, "e4m3", 0),
    ([65, 33], [65, 1500], 10, 2, 64, 32, "bf16", 200),
    ([257], [301], 4, 4, 128, 128, "bf16", 0),
    ([20], [90], 40, 1, 128, 16, "bf16", 0),
    ([17, 40], [50, 300], 6, 2, 512, 16, "e4m3", 64),
    ([200], [200], 3, 1, 256, 32, "e4m3", 0),
    ([150], [100], 2, 2, 64, 16, "e4m3", 40),     # rows that see nothing, over several tiles
    ([1], [0], 8, 2, 256, 16, "bf16", 0),         # nothing cached: all rows are zero
    ([5, 1], [0, 0], 4, 1, 512, 16, "e4m3", 9),
    ([70, 2, 1], [0, 5, 0], 4, 2, 128, 16, "bf16", 0),
]


def attention_inputs(q_lens, kv_lens, n_q, n_kv, D, page, cache, window, seed, peak=2.5, spare=3):
    """Caches whose rows no query sees hold NaN, tables whose entries no query sees hold garbage."""
    g = generator(seed)
    T = sum(q_lens)
    q = (torch.randn(T, n_q, D, generator=g, device=DEV) * (peak / math.sqrt(D))).bfloat16()
    widths = [-(-n // page) for n in kv_lens]
    pages = sum(widths) + spare
    order = torch.randperm(pages, generator=g, device=DEV).cpu().numpy().astype(np.int32)
    table = np.full((len(kv_lens), max(max(widths), 1) + 1), -77, dtype=np.int32)
    kind, scales, host = (torch.bfloat16, {}, {}) if cache == "bf16" else (E4M3, {}, {})
    caches = []
    for name in "kv":
        x = torch.randn(pages, n_kv, page, D, generator=g, device=DEV)
        if cache == "e4m3":
            s = torch.rand(n_kv, generator=g, device=DEV) * 0.02 + 0.01
            scales[name + "_scale"] = s
            x = (x / s.view(1, -1, 1, 1)).clamp(-448, 448)
        x = x.to(kind)
        seen = torch.zeros(pages, page, dtype=torch.bool)
        at, rows = 0, []
        val = f64(x) * (f64(scales[name + "_scale"])[None, :, None, None] if scales else 1.0)
        for b, (n, long) in enumerate(zip(q_lens, kv_lens)):
            mine = order[at:at + widths[b]]
            at += widths[b]
            lo = max(0, long - n - window + 1) if window else 0
            if n:
                for j in range(lo, long):
                    seen[mine[j // page], j % page] = True
                table[b, lo // page:widths[b]] = mine[lo // page:]
            rows.append(val[mine].transpose(0, 2, 1, 3).reshape(-1, n_kv, D)[:long])
        host[name] = rows
        raw = x.view(torch.uint8) if cache == "e4m3" else x.view(torch.int16)
        raw.permute(0, 2, 1, 3)[~seen.to(DEV)] = 0x7F if cache == "e4m3" else 0x7FC0
        caches.append(x)
    ints = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device=DEV)  # noqa: E731
    return dict(q=q, caches=caches, table=ints(table), starts=ints([0] + list(np.cumsum(q_lens))), lens=ints(kv_lens),
                max_q=max(q_lens), max_kv=max(kv_lens), scales=scales, host=host)


def attend(x, window, scale=1.0, **kw):
    return q4.paged_attention(x["q"], *x["caches"], x["table"], x["starts"], x["lens"], x["max_q"], x["max_kv"],
                              scale=scale, window=window, **x["scales"], **kw)


def check_attention(x, out, q_lens, kv_lens, window, scale=1.0):
    want, mag, span = so.attention(f64(x["q"]), x["host"]["k"], x["host"]["v"], q_lens, kv_lens, scale, window)
    got = f64(out)
    keys = min(max(kv_lens), window + 1 if window else max(kv_lens))
    tol = so.attention_tolerance(want, mag, span, keys, got.shape[-1])
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


@pytest.mark.parametrize("q_lens,kv_lens,n_q,n_kv,D,page,cache,window", ATTENTION)
def test_attention_against_oracle(q_lens, kv_lens, n_q, n_kv, D, page, cache, window):
    x = attention_inputs(q_lens, kv_lens, n_q, n_kv, D, page, cache, window, seed=sum(kv_lens) + D)
    err = flag()
    out = attend(x, window, err_flag=err)
    assert err.item() == 0
    check_attention(x, out, q_lens, kv_lens, window)
    assert torch.equal(out, attend(x, window))


@pytest.mark.parametrize("D,peak,scale", [(256, 40.0, 1.0), (64, 2.5, -0.7), (128, 300.0, 0.03), (512, 2.5, 0.0)])
@pytest.mark.parametrize("n", [1, 5, 70])
def test_attention_peaked_and_other_scales(D, peak, scale, n):
    x = attention_inputs([n], [400 + n], 4, 2, D, 16, "bf16", 0, seed=n, peak=peak)
    check_attention(x, attend(x, 0, scale=scale), [n], [400 + n], 0, scale)


@pytest.mark.parametrize("n,D", [(1, 256), (4, 128), (80, 256), (80, 512)])
def test_attention_loose_bounds_give_the_same_values(n, D):
    """max_q_len and max_kv_len size the launch; looser ones change at most how the sums are split."""
    lens = [300 + n, n]
    x = attention_inputs([n, n], lens, 8, 2, D, 16, "bf16", 0, seed=5)
    wide = torch.full((2, 1000), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, :x["table"].shape[1]] = x["table"]
    x.update(table=wide, max_q=900, max_kv=16000)
    check_attention(x, attend(x, 0), [n, n], lens, 0)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,group,D,longest", [(1, 1, 64, 0), (1, 8, 128, 0), (1, 8, 256, 0), (2, 8, 512, 0), (4, 8, 256, 0),
                                               (8, 4, 64, 8192), (1, 4, 128, 8192), (32, 1, 256, 8192), (3, 5, 512, 8192)])
def test_attention_few_rows_keep_sixteen_bits_of_a_probability(n, group, D, longest, cache):
    """Keys of two kinds by turns, of probability 1 and p (to a common factor), with values a and -a c, c about
    1 / p: the sums all but cancel, so what is left of the probabilities' rounding shows beside the output's own.
    In two bf16 parts a probability is off by 2^-16 (half a step, 2^-8, of a rest of at most 2^-8 of it); in one
    part p, which lies far from its nearest bf16 value, is off by more than 2^-10."""
    score, c = -1.375, 4.0
    p = math.exp(score)
    assert abs(float(torch.tensor(p).bfloat16()) / p - 1) > 2.0 ** -10 and abs(p * c - 1) < 0.1
    long, page, kind = 300, 16, torch.bfloat16 if cache == "bf16" else E4M3
    g = generator(D + n)
    T, pages = n, -(-long // page)
    k, v = torch.zeros(long, D, device=DEV), torch.empty(long, D, device=DEV)
    sign = torch.randint(0, 2, (D,), generator=g, device=DEV) * 2.0 - 1
    v[::2], v[1::2], k[1::2, 0] = sign, -sign * c, score
    k[:, 1:] = torch.randint(-2, 3, (long, D - 1), generator=g, device=DEV)  # (met by zeros of q)
    q = torch.zeros(T, group, D, device=DEV)
    q[..., 0] = 1.0
    room = lambda x: torch.cat([x, x.new_zeros(pages * page - long, D)]).view(pages, 1, page, D).to(kind)  # noqa: E731
    x = dict(q=q.bfloat16(), caches=[room(k), room(v)], table=torch.arange(pages, dtype=torch.int32, device=DEV)[None],
             starts=torch.tensor([0, n], dtype=torch.int32, device=DEV), max_q=n, max_kv=long, scales={},
             lens=torch.tensor([long], dtype=torch.int32, device=DEV))
    if longest:
        loosen(x, page, longest)
    kh, vh = f64(k)[:, None], f64(v)[:, None]
    want, mag, span = so.attention(f64(x["q"]), [kh], [vh], [n], [long], 1.0, 0)
    ds = (D + 4) * 2.0 ** -24 * span[..., None]
    inner = mag * (2 * (1.1 * ds + 2.0 ** -21 + (long + 8) * 2.0 ** -24) + 2.0 ** -16)
    tol = inner + 2.0 ** -8 * (np.abs(want) + inner)
    assert (np.abs(f64(attend(x, 0)) - want) <= tol).all()
    # the bound tells one part from two: the oracle with probabilities rounded once lies outside
    at = long - n + np.arange(n)
    w = np.where(np.arange(long) % 2, p, 1.0) * (np.arange(long)[None] <= at[:, None])
    once = (so.bf16_round(w) @ vh[:, 0]) / w.sum(-1, keepdims=True)
    assert (np.abs(once[:, None] - want) > tol).all()


@pytest.mark.parametrize("n", [1, 20])
def test_attention_widest_window_is_none(n):
    x = attention_inputs([n, n], [500, 300], 8, 2, 128, 16, "bf16", 0, seed=n)
    assert torch.equal(attend(x, (1 << 63) - 1), attend(x, 0)) and torch.equal(attend(x, 500), attend(x, 0))


@pytest.mark.parametrize("n", [1, 3, 40])
def test_attention_invalid_sequences_are_left_alone(n):
    lens = [100, 200, 300]
    for spoil in ("kv_negative", "kv_long", "q_long", "starts_down", "starts_far"):
        x = attention_inputs([n] * 3, lens, 4, 2, 128, 16, "bf16", 0, seed=9)
        want, mag, span = so.attention(f64(x["q"]), x["host"]["k"], x["host"]["v"], [n] * 3, lens, 1.0, 0)
        tol = so.attention_tolerance(want, mag, span, max(lens), 128)
        mark = torch.full_like(x["q"], 7.0)
        bad = {1}
        if spoil == "kv_negative":
            x["lens"][1] = -5
        elif spoil == "kv_long":
            x["lens"][1] = 301
        elif spoil == "q_long":
            if n == 1:
                continue
            x["starts"][2] += 1  # 1 has a row more than max_q_len, 2 one fewer
            bad = {1, 2}
        elif spoil == "starts_down":
            x["starts"][1] = -1  # neither 0 nor 1 is valid
            bad = {0, 1}
        else:
            x["starts"][3] = 3 * n + 1
            bad = {2}
        err = flag()
        out = attend(x, 0, out=mark, err_flag=err)
        assert err.item() == 1, spoil
        for b in range(3):
            rows = slice(b * n, (b + 1) * n)
            if b not in bad:
                # (not bit for bit: how the keys are cut into partial sums goes by the whole batch)
                assert (np.abs(f64(out[rows]) - want[rows]) <= tol[rows]).all(), (spoil, b)
            elif spoil != "q_long":
                assert (out[rows] == 7.0).all(), (spoil, b)


@pytest.mark.parametrize("n", [1, 6, 50])
def test_attention_rows_outside_every_sequence_stay(n):
    x = attention_inputs([n, n], [90, 70], 4, 1, 64, 16, "bf16", 0, seed=2)
    want = attend(x, 0)  # (the same lengths below: the same bits)
    pad = torch.randn(5, 4, 64, device=DEV).bfloat16()
    x["q"] = torch.cat([pad[:2], x["q"], pad[2:]])
    x["starts"] = x["starts"] + 2
    out = attend(x, 0, out=torch.full_like(x["q"], 3.0))
    assert torch.equal(out[2:2 + 2 * n], want)
    assert (out[:2] == 3.0).all() and (out[2 + 2 * n:] == 3.0).all()


@pytest.mark.parametrize("n", [1, 6, 50])
def test_attention_bad_pages_are_not_seen(n):
    """A page number out of range hides its positions: the same as a sequence without them."""
    page, lens = 16, [160, 48]
    x = attention_inputs([n, 1], lens, 4, 2, 128, page, "bf16", 0, seed=4)
    for bad in (-1, x["caches"][0].shape[0], 1 << 30, -(1 << 31)):
        y = dict(x, table=x["table"].clone())
        y["table"][0, 2] = bad
        err = flag()
        out = attend(y, 0, err_flag=err)
        assert err.item() == 1
        keep = [j for j in range(lens[0]) if j // page != 2]
        host = {c: [np.delete(x["host"][c][0], range(2 * page, 3 * page), 0), x["host"][c][1]] for c in "kv"}
        assert len(keep) == lens[0] - page
        check_attention(dict(x, host=host), out, [n, 1], [lens[0] - page, lens[1]], 0)


@pytest.mark.parametrize("n,D,cache", [(5, 128, "bf16"), (8, 512, "bf16"), (70, 64, "e4m3"), (70, 256, "bf16"),
                                       (40, 512, "bf16")])
@pytest.mark.parametrize("window", [0, 9])
def test_attention_nonfinite_keys_touch_only_rows_that_see_them(n, D, cache, window):
    """NaN in a new token's key or value: the rows before it, and those whose window has passed it, are
    untouched; the rows that see it are NaN (its key) or NaN where it is (its value)."""
    long, at = 150, n // 2  # the at-th new token
    x = attention_inputs([n], [long], 4, 2, D, 16, cache, window, seed=8)
    want, mag, span = so.attention(f64(x["q"]), x["host"]["k"], x["host"]["v"], [n], [long], 1.0, window)
    # the order of the sums is not defined, so a value that is not finite may change it for the other rows and
    # columns: each result is within the bound of the exact one, whatever the order
    tol = so.attention_tolerance(want, mag, span, long, D)
    pos = long - n + at
    page = int(x["table"][0, pos // 16])
    sees = np.array([at <= i and (not window or i < at + window) for i in range(n)])
    for which in (0, 1):
        y = dict(x, caches=[c.clone() for c in x["caches"]])
        raw = y["caches"][which].view(torch.uint8 if cache == "e4m3" else torch.int16)
        raw[page, 1, pos % 16, 3] = 0x7F if cache == "e4m3" else 0x7FC0
        got = f64(attend(y, window))
        hit = np.zeros(got.shape, bool)
        hit[np.ix_(sees, [2, 3], range(D) if which == 0 else [3])] = True
        assert np.isnan(got[hit]).all()
        assert (np.abs(got - want) <= tol)[~hit].all()


LONG = [  # long units, cut over workgroups and joined
    ([70], [5000], 8, 2, 256, 64, "bf16", 0),
    ([64, 200], [3000, 4500], 8, 2, 256, 32, "e4m3", 0),
    ([100, 40], [2500, 6000], 4, 1, 512, 64, "bf16", 0),
    ([130], [3000], 8, 1, 512, 16, "e4m3", 1500),
    ([300, 40, 0, 65], [5000, 9000, 70, 300], 8, 2, 128, 128, "bf16", 0),
    ([150], [7000], 4, 4, 128, 16, "e4m3", 4000),
    ([600, 33], [600, 8000], 4, 2, 64, 16, "bf16", 0),
    ([257], [6000], 3, 1, 64, 64, "e4m3", 3000),
    # units of a few to 32 blocks of keys with a compute unit each, the keys in two halves
    ([64, 40], [1000, 641], 8, 2, 64, 16, "bf16", 0),
    ([100], [1985], 4, 4, 64, 64, "e4m3", 0),
    ([64, 0, 129], [600, 30, 1024], 8, 2, 128, 32, "bf16", 0),
    ([90, 66], [1300, 66], 16, 4, 128, 64, "e4m3", 555),
    ([300], [300], 4, 2, 256, 16, "bf16", 0),
    ([64, 35], [289, 900], 8, 1, 256, 64, "e4m3", 0),
    ([200, 64], [950, 900], 3, 3, 256, 32, "bf16", 300),
    ([150], [400], 2, 1, 256, 128, "e4m3", 1),
    ([400], [310], 2, 2, 256, 16, "bf16", 0),  # the first rows see nothing
    # many short sequences of few rows: a workgroup each
    ([1] * 40, [2000 - 51 * i for i in range(40)], 16, 8, 128, 32, "bf16", 0),
    ([4, 0, 1, 3] * 10, [4 + 45 * i for i in range(40)], 64, 8, 64, 64, "e4m3", 0),
    ([2] * 33, [1 + 60 * i for i in range(33)], 16, 8, 128, 16, "e4m3", 700),
    # more sequences than a wave has lanes
    ([1] * 70, [1 + 37 * (i % 29) for i in range(70)], 8, 2, 128, 16, "bf16", 0),
    ([1, 3, 0, 2] * 40, [5 + 11 * (i % 90) for i in range(160)], 4, 1, 64, 32, "bf16", 70),
    ([40, 1, 0, 66, 17] * 28, [66 + 31 * (i % 80) for i in range(140)], 4, 2, 64, 16, "bf16", 0),
    ([33] * 90, [33 + 90 * (i % 11) for i in range(90)], 2, 1, 256, 64, "e4m3", 0),
]


@pytest.mark.parametrize("q_lens,kv_lens,n_q,n_kv,D,page,cache,window", LONG)
def test_attention_cut_over_workgroups(q_lens, kv_lens, n_q, n_kv, D, page, cache, window):
    x = attention_inputs(q_lens, kv_lens, n_q, n_kv, D, page, cache, window, seed=sum(kv_lens) + D)
    if len(q_lens) > 64:  # (bounds that leave the cut to the lengths)
        loosen(x, page, 8192)
    err = flag()
    out = attend(x, window, err_flag=err)
    assert err.item() == 0
    check_attention(x, out, q_lens, kv_lens, window)
    assert torch.equal(out, attend(x, window))


def loosen(x, page, longest):
    """The same sequences under a bound on their lengths that is far above them."""
    wide = torch.full((x["table"].shape[0], longest // page), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, :x["table"].shape[1]] = x["table"]
    x.update(table=wide, max_kv=longest)


@pytest.mark.parametrize("n,longest", [(3, 16384), (70, 16384), (70, 1008)])
@pytest.mark.parametrize("D", [128, 256])
def test_attention_faults_of_the_batch_when_cut(n, longest, D):
    """A sequence that is not valid, a page out of range and a key that is not finite, in stretches and joins and
    (few keys at most) in units whose keys two groups of waves share."""
    lens = [150 + n, 300 + n, 200 + n]
    x = attention_inputs([n] * 3, lens, 4, 2, D, 16, "bf16", 0, seed=n + D)
    loosen(x, 16, longest)
    want, mag, span = so.attention(f64(x["q"]), x["host"]["k"], x["host"]["v"], [n] * 3, lens, 1.0, 0)
    tol = so.attention_tolerance(want, mag, span, max(lens), D)

    y = dict(x, lens=x["lens"].clone())
    y["lens"][0] = longest + 1
    err = flag()
    got = f64(attend(y, 0, out=torch.full_like(x["q"], 7.0), err_flag=err))
    assert err.item() == 1 and (got[:n] == 7.0).all()
    assert (np.abs(got - want) <= tol)[n:].all()

    y = dict(x, table=x["table"].clone())
    y["table"][1, 5] = -1
    err = flag()
    out = attend(y, 0, err_flag=err)
    assert err.item() == 1
    host = {c: [x["host"][c][0], np.delete(x["host"][c][1], range(80, 96), 0), x["host"][c][2]] for c in "kv"}
    check_attention(dict(x, host=host), out, [n] * 3, [lens[0], lens[1] - 16, lens[2]], 0)

    at, pos = n // 2, lens[2] - n + n // 2
    y = dict(x, caches=[c.clone() for c in x["caches"]])
    y["caches"][1][int(x["table"][2, pos // 16]), 1, pos % 16, 5] = float("inf")
    got = f64(attend(y, 0))
    hit = np.zeros(got.shape, bool)
    hit[2 * n + at:, 2:, 5] = True
    assert np.isposinf(got[hit]).all()
    assert (np.abs(got - want) <= tol)[~hit].all()


@pytest.mark.parametrize("n,long,n_q,n_kv,D,longest", [
    (1, 150, 4, 2, 64, 0), (4, 150, 4, 2, 128, 0),                            # few rows, a unit a workgroup
    (1, 150, 4, 2, 256, 0), (4, 150, 4, 2, 512, 0),                           # in stretches
    (1, 3000, 8, 2, 64, 8192), (4, 3000, 8, 2, 128, 0), (4, 900, 8, 1, 512, 4096),  # cut and joined
    (70, 150, 4, 2, 64, 0), (70, 150, 4, 2, 256, 0), (40, 150, 4, 2, 512, 0),  # many rows, a unit a workgroup
    (70, 700, 8, 2, 128, 1008),                                               # its keys in two halves
    (70, 3000, 8, 2, 64, 8192), (70, 2000, 4, 2, 256, 16384), (40, 2500, 4, 1, 512, 8192),  # cut and joined
])
@pytest.mark.parametrize("far", ["", "key", "half"])
def test_attention_infinite_values_that_every_row_sees(n, long, n_q, n_kv, D, longest, far):
    """An infinity among the values of a key that all rows see is the result in its column, both signs of one are
    NaN; all other columns and heads are untouched. The key stands first, in the middle and last of those that all
    rows see. far: its score, or those of the first half of the keys, lie so far below the others that their
    probabilities are no fp32 numbers, nor the weight of the pieces that hold them alone."""
    x = attention_inputs([n], [long], n_q, n_kv, D, 16, "bf16", 0, seed=n + D)
    x["q"] = x["q"].abs()
    if longest:
        loosen(x, 16, longest)
    at = lambda pos: (int(x["table"][0, pos // 16]), n_kv - 1, pos % 16)  # noqa: E731
    mine = slice((n_kv - 1) * (n_q // n_kv), n_q)  # the query heads that read it
    for pos in (0, (long - n) // 2, long - n):
        other = (pos + 33) % (long - n + 1)
        y = dict(x, caches=[c.clone() for c in x["caches"]], host={c: [h.copy() for h in x["host"][c]] for c in "kv"})
        # (sum |q| is about 0.8 * 2.5 sqrt(D): 100 sqrt(D) below the others' scores)
        for j in {"": [], "key": [pos], "half": range((long - n) // 2)}[far]:
            y["caches"][0][at(j)] = -50.0
            y["host"]["k"][0][j, n_kv - 1] = -50.0
        v = y["caches"][1]
        v[at(pos)][3] = v[at(pos)][D - 2] = math.inf
        v[at(pos)][7] = v[at(other)][D - 2] = -math.inf
        y["host"]["v"][0][[pos, pos, pos, other], n_kv - 1, [3, D - 2, 7, D - 2]] = 0
        want, mag, span = so.attention(f64(y["q"]), y["host"]["k"], y["host"]["v"], [n], [long], 1.0, 0)
        tol = so.attention_tolerance(want, mag, span, long, D)
        got = f64(attend(y, 0))
        assert np.isposinf(got[:, mine, 3]).all() and np.isneginf(got[:, mine, 7]).all()
        assert np.isnan(got[:, mine, D - 2]).all()
        hit = np.zeros(got.shape, bool)
        for col in (3, 7, D - 2):
            hit[:, mine, col] = True
        assert (np.abs(got - want) <= tol)[~hit].all()


@pytest.mark.parametrize("n,long,D", [(1, 150, 64), (4, 150, 256), (4, 3000, 128), (70, 150, 64), (70, 150, 256),
                                      (40, 150, 512), (70, 700, 128), (70, 6000, 256)])
def test_attention_nan_key_and_infinite_value(n, long, D):
    """Rows that see a NaN in a key are NaN, also in the column of an infinite value; those before the key are not."""
    x = attention_inputs([n], [long], 4, 2, D, 16, "bf16", 0, seed=n + D)
    pos, at = 7, n // 2
    for c, (j, col) in enumerate(((long - n + at, 9), (pos, 3))):  # a new key, an old value
        x["caches"][c][int(x["table"][0, j // 16]), 1, j % 16, col] = math.nan if c == 0 else math.inf
    got = f64(attend(x, 0))[:, 2:]
    assert np.isnan(got[at:]).all()
    assert np.isposinf(got[:at, :, 3]).all() and np.isfinite(np.delete(got[:at], 3, 2)).all()


@pytest.mark.parametrize("n,long,n_q,n_kv,D,longest", [
    (1, 150, 4, 2, 64, 0), (4, 150, 4, 2, 128, 0), (1, 150, 4, 2, 256, 0), (4, 150, 4, 2, 512, 0),
    (1, 3000, 8, 2, 64, 8192), (4, 3000, 8, 2, 128, 0), (1, 9000, 8, 1, 512, 0),
    (70, 150, 4, 2, 64, 0), (70, 150, 4, 2, 256, 0), (40, 150, 4, 2, 512, 0), (70, 700, 8, 2, 128, 1008),
    (70, 3000, 8, 2, 64, 8192), (70, 2000, 4, 2, 256, 16384), (40, 2500, 4, 1, 512, 8192),
])
def test_attention_scores_of_minus_infinity(n, long, n_q, n_kv, D, longest):
    """A score of -infinity gives its key no weight, so a row that sees no other is 0 / 0, which is NaN; a row that
    sees nothing (its pages are out of range) is zero as ever."""
    x = attention_inputs([n], [long], n_q, n_kv, D, 16, "bf16", 0, seed=n + D)
    x["q"] = x["q"].abs().clamp(min=0.01)
    if longest:
        loosen(x, 16, longest)
    mine = slice((n_kv - 1) * (n_q // n_kv), n_q)  # the query heads of the head of keys that is changed
    pages = x["table"][0, :-(-long // 16)].long()

    def attended(keys, bad_pages=0):
        y = dict(x, caches=[x["caches"][0].clone(), x["caches"][1]], table=x["table"].clone())
        pos = torch.arange(keys, device=DEV)
        y["caches"][0][pages[pos // 16], n_kv - 1, pos % 16, 5] = -math.inf
        y["table"][0, :bad_pages] = -1
        return f64(attend(y, 0))

    rest = np.ones(n_q, bool)
    rest[mine] = False
    want, mag, span = so.attention(f64(x["q"]), x["host"]["k"], x["host"]["v"], [n], [long], 1.0, 0)
    tol = so.attention_tolerance(want, mag, span, long, D)
    got = attended(long)
    assert np.isnan(got[:, mine]).all() and (np.abs(got - want) <= tol)[:, rest].all()
    # the keys before the new ones: the rows are what they are without those keys
    few = dict(x, host={c: [h[0][long - n:]] for c, h in x["host"].items()})
    want, mag, span = so.attention(f64(x["q"]), few["host"]["k"], few["host"]["v"], [n], [n], 1.0, 0)
    tol = so.attention_tolerance(want, mag, span, long, D)
    assert (np.abs(attended(long - n) - want) <= tol)[:, mine].all()
    # pages out of range, and -infinity in the rest; all out of range
    got = attended(long, bad_pages=(long - n) // 16)
    assert np.isnan(got[:, mine]).all()
    assert not attended(long, bad_pages=pages.numel()).any()


def test_attention_other_streams_graph_and_shared_workspace():
    """Eager, on a side stream, and replayed in two graphs that share one workspace one after the other."""
    cases = [([1] * 3, [900, 40, 2000], 0), ([64], [700], 0), ([4, 4], [500, 90], 128)]
    xs = [attention_inputs(a, b, 8, 2, 256, 64, "bf16", w, seed=i) for i, (a, b, w) in enumerate(cases)]
    want = [attend(x, w) for x, (_, _, w) in zip(xs, cases)]
    need = max(q4.paged_attention_workspace_bytes(len(b), 8, 2, 256, max(a), max(b), w) for a, b, w in cases)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [attend(x, w) for x, (_, _, w) in zip(xs, cases)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(x["q"]) for x in xs]
    graphs = []
    for order in ((0, 1, 2), (2, 0, 1)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for i in order:
                attend(xs[i], cases[i][2], ws=ws, out=outs[i])
        graphs.append(g)
    for turn in range(3):
        for g in graphs:
            for o in outs:
                o.zero_()
            g.replay()
            ws_noise = attend(xs[turn], cases[turn][2], ws=ws)
            torch.cuda.synchronize()
            assert torch.equal(ws_noise, want[turn])
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # other lengths in the same graph: the lengths are read on the device
    x = xs[0]
    x["lens"].copy_(torch.tensor([100, 1, 64], dtype=torch.int32))
    graphs[0].replay()
    assert torch.equal(outs[0], attend(x, 0))
    host = {c: [h[:n] for h, n in zip(x["host"][c], (100, 1, 64))] for c in "kv"}
    check_attention(dict(x, host=host), outs[0], [1] * 3, [100, 1, 64], 0)


@pytest.mark.parametrize("q_lens,kv_lens,n_q,n_kv,D,longest", [
    ([1, 1, 0, 1], [900, 40, 30, 2500], 8, 2, 256, 4096),  # few rows, fewer units than workgroups
    ([1] * 90, [50 + 20 * i for i in range(90)], 16, 8, 64, 4096),  # and more
    ([70, 0, 200], [3000, 10, 900], 8, 2, 128, 8192),  # many rows in stretches
    ([64] * 40, [64 + 40 * i for i in range(40)], 32, 16, 64, 8192),
    ([130, 64, 0], [400, 300, 9], 8, 2, 256, 512),  # units alone on a compute unit
])
def test_attention_dirty_workspaces_two_at_once_and_new_lengths(q_lens, kv_lens, n_q, n_kv, D, longest):
    """Nothing is expected of what a workspace holds; calls with workspaces of their own may overlap; a captured
    call follows lengths, rows and pages that change on the device."""
    x = attention_inputs(q_lens, kv_lens, n_q, n_kv, D, 32, "bf16", 0, seed=len(q_lens) + D)
    loosen(x, 32, longest)
    want = attend(x, 0)
    check_attention(x, want, q_lens, kv_lens, 0)
    need = q4.paged_attention_workspace_bytes(len(q_lens), n_q, n_kv, D, max(q_lens), longest, 0)
    ws = [torch.empty(max(need, 1), dtype=torch.uint8, device=DEV) for _ in "ab"]
    outs = [torch.empty_like(x["q"]) for _ in "ab"]
    streams = [torch.cuda.Stream() for _ in "ab"]
    for fill in (0, 255, 127, 1):
        for w, o in zip(ws, outs):
            w.fill_(fill)
            o.fill_(9.0)
        torch.cuda.synchronize()
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                for _ in range(5):
                    attend(x, 0, ws=w, out=o)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(x, 0, ws=ws[0], out=outs[0])
    # the first sequence gives up its last row and some keys, all of the next one's rows go
    n, lens = list(q_lens), list(kv_lens)
    n[0] -= 1
    lens[0] = max(kv_lens[0] - 37, 0)
    n[1] = 0
    starts = np.array([0] + list(np.cumsum(n)), dtype=np.int32)
    x["starts"].copy_(torch.from_numpy(starts))
    x["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
    host = {c: [h[:m] for h, m in zip(x["host"][c], lens)] for c in "kv"}
    for _ in range(3):
        outs[0].fill_(9.0)
        graph.replay()
        total = int(starts[-1])
        assert (outs[0][total:] == 9.0).all()
        check_attention(dict(x, q=x["q"][:total], host=host), outs[0][:total], n, lens, 0)
        assert torch.equal(outs[0][:total], attend(x, 0)[:total])


def test_attention_cache_past_four_gib_elements():
    """Pages whose element offsets pass 2^32: 70000 pages of 64 rows x 2 heads x 512 values, 9.2 GB each."""
    pages, n_kv, page, D = 70000, 2, 64, 512
    caches = [torch.empty(pages, n_kv, page, D, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    small = attention_inputs([1, 2], [130, 64], 4, n_kv, D, page, "bf16", 0, seed=12, spare=0)
    used = [69999, 69998, 65536, 1][:small["caches"][0].shape[0]]
    for big, c in zip(caches, small["caches"]):
        big[used] = c
    table = torch.where((small["table"] >= 0), torch.tensor(used, dtype=torch.int32, device=DEV)[
        small["table"].clamp(min=0).long()], small["table"])
    x = dict(small, caches=caches, table=table.contiguous())
    assert torch.equal(attend(x, 0), attend(small, 0))
    # and appended there
    rows = torch.randn(2, n_kv * D, device=DEV)
    slots = torch.tensor([69999 * page + 63, 65536 * page + 5], dtype=torch.int32, device=DEV)
    pos = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    q4.kv_append_rope(None, rows, rows, pos, slots, *caches, None)
    for c in caches:
        assert torch.equal(c[69999, :, 63].reshape(-1), rows[0].bfloat16())
        assert torch.equal(c[65536, :, 5].reshape(-1), rows[1].bfloat16())


# ------------------------------------------------------------------ sampling


def sampler(z, u, **kw):
    rows = z.shape[0]
    par = {}
    for name, kind in (("temperature", torch.float32), ("top_k", torch.int32), ("top_p", torch.float32),
                       ("min_p", torch.float32)):
        if name in kw:
            v = kw[name]
            par[name] = torch.tensor(v if isinstance(v, (list, np.ndarray)) else [v] * rows, dtype=kind, device=DEV)
    u = torch.tensor(u if isinstance(u, (list, np.ndarray)) else [u] * rows, dtype=torch.float32, device=DEV)
    return q4.sample_logits(z, u, cap=kw.get("cap", 30.0), **par), u, par


def check_sample(z, u, strict=True, **kw):
    (idx, prob), u, par = sampler(z, u, **kw)
    zh, uh = f64(z), f64(u)
    host = {n: f64(p) if p.dtype != torch.int32 else p.cpu().numpy() for n, p in par.items()}
    for r in range(z.shape[0]):
        args = {n: (int if n == "top_k" else float)(v[r]) for n, v in host.items()}
        i, p, border = so.sample(zh[r], uh[r], cap=kw.get("cap", 30.0), **args)
        # the kernel's running sums are off by at most vocab 2^-43 of the heaviest weight, 2^-23
        if border < 2.0 ** -22 and not strict:
            continue
        assert int(idx[r]) == i, (r, args, uh[r], border)
        if np.isnan(p):
            assert math.isnan(float(prob[r]))
        else:  # that, and the rounding of the result
            assert abs(float(prob[r]) - p) <= p * (2.0 ** -24 + 2.0 ** -22), (r, args)
    return idx


FILTERS = [dict(), dict(temperature=0.0), dict(top_k=1), dict(top_k=64, top_p=0.95), dict(top_p=0.9),
           dict(top_p=0.3, temperature=1.7), dict(min_p=0.05), dict(top_k=500, top_p=0.99, min_p=0.001),
           dict(temperature=0.05), dict(temperature=8.0, top_p=0.5), dict(temperature=100.0, top_k=700),
           dict(top_p=0.0), dict(top_k=3, min_p=1.0), dict(temperature=0.02, top_k=50)]


@pytest.mark.parametrize("vocab", [1, 2, 63, 1000, 1025, 50257, 262144])
@pytest.mark.parametrize("kw", FILTERS)
def test_sample_against_oracle(vocab, kw):
    g = generator(vocab)
    rows = 3
    z = torch.randn(rows, vocab + 3, generator=g, device=DEV)[:, :vocab] * 4
    for u in (torch.rand(rows, generator=g, device=DEV).cpu().numpy(), [0.0, 0.5, 1 - 2.0 ** -24]):
        check_sample(z, u, strict=False, **kw)


def test_sample_rows_with_their_own_settings():
    g = generator(1)
    rows = 40
    z = torch.randn(rows, 20011, generator=g, device=DEV) * 3
    z[::3] *= 8  # some capped hard
    pick = lambda v: np.random.RandomState(2 + len(v)).choice(v, rows)  # noqa: E731
    kw = dict(temperature=pick([0.0, 0.5, 1.0, 2.0, -1.0]), top_k=pick([0, 1, 40, 20011, 30000, -4]),
              top_p=pick([1.0, 0.9, 0.5, 0.0, 2.0, -1.0, 0.99]), min_p=pick([0.0, 0.1, -1.0, 0.01, 0.0, 2.0, 0.5, 0.02]))
    u = torch.rand(rows, generator=g, device=DEV).cpu().numpy()
    check_sample(z, u, strict=False, **kw)
    check_sample(z, u, strict=False, cap=0.0, **kw)
    # not-a-number settings switch a filter off, a not-a-number temperature is greedy
    nan = [math.nan] * rows
    a = sampler(z, u, top_p=nan, min_p=nan)[0][0]
    assert torch.equal(a, sampler(z, u)[0][0])
    assert torch.equal(sampler(z, u, temperature=nan)[0][0].long(), z.argmax(-1))
    # numbers outside [0, 1) are clamped into it
    for odd, same in ((-1.0, 0.0), (math.nan, 0.0), (5.0, 1 - 2.0 ** -24), (1.0, 1 - 2.0 ** -24)):
        assert torch.equal(sampler(z, odd, top_k=5)[0][0], sampler(z, same, top_k=5)[0][0])


@pytest.mark.parametrize("vocab", [5, 4096, 70000, 262144])
def test_sample_equal_logits(vocab):
    """All weights equal: every sum is a whole number of them, and borders fall on ties by index."""
    z = torch.full((4, vocab), -2.5, device=DEV)
    z[1] = 0.0
    z[1, ::2] = -0.0
    u = [0.0, 0.25, 0.5, 0.75]
    idx = sampler(z, u)[0][0].tolist()
    assert idx == [int(x * vocab) for x in u]
    k = max(1, vocab // 3)
    (idx, prob), _, _ = sampler(z, u, top_k=k)
    assert idx.tolist() == [int(x * k) for x in u] and (prob - 1 / k).abs().max() <= 2.0 ** -23 / k
    kept = math.ceil(0.5 * vocab)
    assert sampler(z, u, top_p=0.5)[0][0].tolist() == [int(x * kept) for x in u]
    assert sampler(z, u, temperature=0.0)[0][0].tolist() == [0] * 4


def test_sample_special_values():
    inf, nan = math.inf, math.nan
    base = torch.randn(1, 3001, generator=generator(4), device=DEV)
    # a row with nothing to draw
    for v in (nan, -inf):
        z = torch.full((2, 777), v, device=DEV)
        (idx, prob), _, _ = sampler(z, 0.5)
        assert idx.tolist() == [-1, -1] and prob.isnan().all()
        assert sampler(z, 0.5, temperature=0.0)[0][0].tolist() == [-1, -1]
        z[1, 700] = -1e30
        assert sampler(z, 0.5, top_k=4, top_p=0.3)[0][0].tolist() == [-1, 700]
    # NaN and -infinity are as if they were not there
    z = base.clone()
    z[0, ::3] = nan
    z[0, 1::3] = -inf
    for kw in (dict(), dict(top_k=50), dict(top_p=0.8), dict(top_k=2000)):
        for u in (0.0, 0.3, 0.99):
            i = int(check_sample(z, u, strict=False, **kw)[0])
            assert i % 3 == 2
    # +infinity takes everything when there is no cap, equal ones share
    z = base.clone()
    z[0, 5] = z[0, 2000] = inf
    assert [int(sampler(z, u, cap=0.0)[0][0]) for u in (0.0, 0.49, 0.5, 0.9)] == [5, 5, 2000, 2000]
    assert int(sampler(z, 0.9, cap=0.0, top_k=1)[0][0]) == 5
    assert int(sampler(z, 0.9, cap=0.0, top_p=0.5)[0][0]) == 5
    # with the cap infinity is 30, as are large numbers; they stay ranked by their logits
    z[0, 9] = 1e30
    assert int(sampler(z, 0.99, top_k=2)[0][0]) == 2000 and int(sampler(z, 0.99, top_k=3)[0][0]) == 2000
    assert int(sampler(z, 0.5, top_k=3)[0][0]) == 9


def test_sample_cap_and_temperature_at_their_ends():
    """No cap in each of its spellings is the same; a cap far above the logits, a temperature that levels all."""
    g = generator(12)
    z = torch.randn(8, 5000, generator=g, device=DEV) * 3
    u = torch.rand(8, generator=g, device=DEV)
    full = lambda v: torch.full((8,), v, device=DEV)  # noqa: E731
    for top_p in (None, full(0.8)):
        idx, prob = q4.sample_logits(z, u, top_p=top_p, cap=0.0)
        for cap in (-1.0, math.inf, math.nan):
            i, p = q4.sample_logits(z, u, top_p=top_p, cap=cap)
            assert torch.equal(i, idx) and torch.equal(p, prob)
    for r in range(8):
        check_sample(z[r:r + 1], float(u[r]), strict=False, cap=1e6)
        check_sample(z[r:r + 1], float(u[r]), strict=False, cap=2.0, top_p=0.7)  # most logits beyond the cap
        check_sample(z[r:r + 1], float(u[r]), strict=False, cap=0.0, temperature=0.01, top_p=0.7)
    idx, prob = q4.sample_logits(z, u, temperature=full(math.inf))
    assert idx.tolist() == [int(x * 5000) for x in u.tolist()] and (prob - 1 / 5000).abs().max() <= 2.0 ** -23 / 5000


@pytest.mark.parametrize("masked", [-1e4, float(np.finfo(np.float32).min), -math.inf])
@pytest.mark.parametrize("vocab,allowed,top_k", [(262144, 40, 64), (262144, 300, 256), (50257, 5, 200), (10000, 9999, 200),
                                                 (20011, 1, 2)])
def test_sample_small_top_k_with_masked_tokens(masked, vocab, allowed, top_k):
    """Guided decoding: a few tokens may be drawn, all others hold a finite value far below or -infinity. With fewer
    groups of an allowed token than top_k the finite ones all go on the list and overflow it."""
    g = generator(vocab + allowed)
    rows = 3
    z = torch.full((rows, vocab), masked, device=DEV)
    for r in range(rows):
        z[r, torch.randperm(vocab, generator=g, device=DEV)[:allowed]] = torch.randn(allowed, generator=g, device=DEV) * 4
    u = torch.rand(rows, generator=g, device=DEV).cpu().numpy()
    # (at T = 20 the masked ones' weights, e^(-60 / 20), are drawn too)
    for kw in (dict(), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=20.0), dict(temperature=20.0, top_p=0.7)):
        check_sample(z, u, strict=False, top_k=top_k, **kw)


@pytest.mark.parametrize("temperature", [1.3, 1.0, 0.3, 1e-6])
def test_sample_rows_far_above_the_cap(temperature):
    """Every logit 12 to 19 times the cap, where the capped ones differ in their last bits or not at all, so that
    the whole row lies in a range that is next to nothing. At T = 1e-6 each side's tanh is off by 2^-53, the
    oracle's product with the cap by another half step: 30 * 4 * 2^-53 / 1e-6 and 2^-49 / 1e-6 are 2e-8 of a
    weight in all, under check_sample's 2^-22."""
    g = generator(31)
    for vocab in (50, 999, 40009):
        z = 360 + 210 * torch.rand(4, vocab, generator=g, device=DEV)
        u = torch.rand(4, generator=g, device=DEV).cpu().numpy()
        for kw in (dict(), dict(top_p=0.37), dict(top_p=0.9), dict(top_k=300), dict(top_k=700, top_p=0.61),
                   dict(top_k=20), dict(top_k=100, top_p=0.31), dict(min_p=0.5, top_p=0.77)):
            check_sample(z, u, strict=False, temperature=temperature, **kw)


@pytest.mark.parametrize("temperature", [1.0, 1e-6, 1e-12, 1e-30])
@pytest.mark.parametrize("sign", [1, -1])
def test_sample_rows_that_the_cap_makes_equal(temperature, sign):
    """Every logit 20 to 40 times the cap: tanh is 1 in fp64 and all weights are equal at any temperature, while
    the ranking stays that of the logits. All sums are whole numbers of weights, so the oracle's index is the one."""
    g = generator(32)
    for vocab in (40, 1000, 30011):
        z = sign * (600 + 600 * torch.rand(3, vocab, generator=g, device=DEV))
        u = torch.rand(3, generator=g, device=DEV).cpu().numpy()
        for kw in (dict(), dict(top_p=0.37), dict(top_k=300), dict(top_k=700, top_p=0.61), dict(top_k=20),
                   dict(top_k=100, top_p=0.31), dict(min_p=1.0)):
            check_sample(z, u, temperature=temperature, **kw)


def test_sample_frequencies():
    """20000 draws from 6 tokens: each count within 5 standard deviations of its expectation."""
    z = torch.log(torch.tensor([[0.05, 0.3, 0.1, 0.25, 0.2, 0.1]], device=DEV)).expand(20000, 6).contiguous()
    u = torch.rand(20000, generator=generator(6), device=DEV).cpu().numpy()
    (idx, _), _, _ = sampler(z, u, cap=0.0)
    n = torch.bincount(idx, minlength=6).double().cpu().numpy()
    p = np.array([0.05, 0.3, 0.1, 0.25, 0.2, 0.1])
    assert (np.abs(n - 20000 * p) <= 5 * np.sqrt(20000 * p * (1 - p))).all()


def test_sample_streams_graph_and_one_row():
    g = generator(11)
    z = torch.randn(6, 30000, generator=g, device=DEV) * 4
    u = torch.rand(6, generator=g, device=DEV)
    kw = dict(temperature=torch.tensor([1.0, 0.0, 0.7, 1.0, 1.0, 2.0], device=DEV),
              top_k=torch.tensor([64, 0, 0, 1, 1000, 0], dtype=torch.int32, device=DEV),
              top_p=torch.tensor([0.95, 1.0, 0.9, 1.0, 0.5, 1.0], device=DEV))
    want = q4.sample_logits(z, u, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = q4.sample_logits(z, u, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = q4.sample_logits(z[0], u[:1], **{n: v[:1] for n, v in kw.items()})
    assert torch.equal(one[0], want[0][:1]) and torch.equal(one[1], want[1][:1])
    ws = torch.empty(max(1, q4.sample_logits_workspace_bytes(6, 30000)), dtype=torch.uint8, device=DEV)
    outs = [torch.empty(6, dtype=torch.int32, device=DEV), torch.empty(6, device=DEV)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.sample_logits(z, u, ws=ws, idx_out=outs[0], prob_out=outs[1], **kw)
    for turn in range(4):
        z.copy_(z.roll(1, 0) if turn else z)
        for o in outs:
            o.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        want = q4.sample_logits(z, u, **kw)
        ws.random_(0, 255)  # nothing is expected of what it holds
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


# ------------------------------------------------------------------ together


def rows_of(codes, sb):
    """The dequantised matrix in fp64."""
    return codes.astype(np.float64) * np.repeat(sb.view(np.float16).astype(np.float64), 32, axis=1)


def test_decode_steps_end_to_end():
    """One windowed attention layer and a head, token by token: q4_gemv -> kv_append_rope -> paged_attention ->
    q4_gemv -> head logits -> sample_logits, against the same steps of the oracle on the device's own
    intermediate values; the greedy draw agrees with lmhead_softcap_argmax."""
    rng = synth.rng_for(77)
    hidden, n_q, n_kv, D, vocab, page, window = 512, 4, 2, 64, 1000, 16, 20
    wide = (n_q + 2 * n_kv) * D
    mats = {}
    for name, (n, k) in dict(qkv=(wide, hidden), o=(hidden, n_q * D), head=(vocab, hidden)).items():
        codes, sb = synth.q4_weights(rng, n, k)
        mats[name] = (q4.q4_pack(torch.from_numpy(codes).to(DEV), torch.from_numpy(sb.view(np.int16)).to(DEV)), n, k,
                      rows_of(codes, sb))
    caches = [torch.full((6, n_kv, page, D), math.nan, device=DEV).bfloat16() for _ in "kv"]
    table = torch.tensor([[4, 1, 5]], dtype=torch.int32, device=DEV)
    order = table[0].tolist()
    freqs = 1e4 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=DEV) / D)
    norm = torch.ones(D, device=DEV)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    x = torch.randn(hidden, generator=generator(5), device=DEV).bfloat16()
    host = {"k": np.zeros((0, n_kv, D)), "v": np.zeros((0, n_kv, D))}
    for step in range(40):
        qkv = q4.q4_gemv(*mats["qkv"][:3], x).view(1, wide)
        slot = order[step // page] * page + step % page
        q = q4.kv_append_rope(qkv[:, :n_q * D], qkv[:, n_q * D:(n_q + n_kv) * D], qkv[:, (n_q + n_kv) * D:],
                              ints(step), ints(slot), *caches, freqs, q_norm=norm, k_norm=norm, v_norm=True)
        want = so.append(*(f64(p).reshape(1, -1, D) for p in qkv.split([n_q * D, n_kv * D, n_kv * D], 1)), [step],
                         f64(freqs), D // 2, f64(norm), f64(norm), True)
        assert (np.abs(f64(q) - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -16).all()
        for c, t, w in zip("kv", caches, want[1:]):
            got = f64(t)[slot // page, :, slot % page]
            assert (np.abs(got - w[0]) <= 2.0 ** -8 * np.abs(w[0]) + 2.0 ** -16).all()
            host[c] = np.concatenate([host[c], got[None]])
        o = q4.paged_attention(q, *caches, table, ints(0, 1), ints(step + 1), 1, step + 1, scale=0.125, window=window)
        ref, mag, span = so.attention(f64(q), [host["k"]], [host["v"]], [1], [step + 1], 0.125, window)
        assert (np.abs(f64(o) - ref) <= so.attention_tolerance(ref, mag, span, window, D)).all()
        y = q4.q4_gemv(*mats["o"][:3], o.view(-1))
        w = mats["o"][3]
        assert (np.abs(f64(y) - w @ f64(o).ravel()) <= oracle.gemv_tolerance(np.abs(w) @ np.abs(f64(o).ravel()))).all()
        x = (y / y.square().mean().sqrt()).bfloat16()
        z = q4.q4_gemv(*mats["head"][:3], x)
        greedy = q4.sample_logits(z, torch.zeros(1, device=DEV), temperature=torch.zeros(1, device=DEV))[0]
        assert int(greedy) == int(q4.lmhead_softcap_argmax(*mats["head"][:3], x)[0])
        check_sample(z.view(1, -1), float(rng.random()), strict=False, top_k=64, top_p=0.95)


def test_prefill_chunks_equal_decode_steps():
    """A prompt in chunks of 64 and less gives the cache and, within the roundings, the outputs of token-by-token."""
    T, n_q, n_kv, D, page = 150, 8, 2, 256, 16
    g = generator(21)
    qkv = torch.randn(T, (n_q + 2 * n_kv) * D, generator=g, device=DEV)
    parts = lambda lo, hi: qkv[lo:hi].split([n_q * D, n_kv * D, n_kv * D], 1)  # noqa: E731
    table = torch.randperm(12, generator=g, device=DEV).int().view(1, 12)
    freqs = 1e6 ** (-2.0 * torch.arange(D // 8, dtype=torch.float64, device=DEV) / D)
    norm = torch.full((D,), 0.3, device=DEV)
    pos = torch.arange(T, device=DEV)
    slots = (table[0].long()[pos // page] * page + pos % page).int()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    outs, stored = [], []
    for step in (64, 1):
        caches = [torch.zeros(12, n_kv, page, D, device=DEV).bfloat16() for _ in "kv"]
        got = []
        for lo in range(0, T, step):
            hi = min(lo + step, T)
            q = q4.kv_append_rope(*parts(lo, hi), pos[lo:hi].int(), slots[lo:hi], *caches, freqs, q_norm=norm, k_norm=norm)
            got.append(q4.paged_attention(q, *caches, table, ints(0, hi - lo), ints(hi), hi - lo, hi))
        outs.append(torch.cat(got))
        stored.append(caches)
    assert torch.equal(stored[0][0], stored[1][0]) and torch.equal(stored[0][1], stored[1][1])
    # each is within 2 half steps (its probabilities', its own) of the exact value: mag <= max |v| over the keys
    v = f64(stored[0][1]).transpose(0, 2, 1, 3).reshape(-1, n_kv, D)[slots.cpu().numpy()]
    mag = np.repeat(np.maximum.accumulate(np.abs(v), 0), n_q // n_kv, axis=1)
    assert (np.abs(f64(outs[0]) - f64(outs[1])) <= 4 * 2.0 ** -8 * mag * 1.05).all()
