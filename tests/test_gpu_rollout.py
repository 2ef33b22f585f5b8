"""The operators of rollouts (attention over shared beginnings, the check of
drafted tokens) on the GPU against their fp64 oracles. Tolerances count the
roundings of the definitions (see serve_oracle.attention_tolerance); half a
step of bf16 is 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import int4_weight_only_block_amd as q4
from oracle import rollout_oracle as ro
from oracle import serve_oracle as so

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def f64(t):
    if t.dtype == E4M3:
        return so.e4m3_values()[t.contiguous().view(torch.uint8).cpu().numpy()]
    return t.detach().double().cpu().numpy()


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device=DEV)


# --------------------------------------------------- shared beginnings

LOOSE = 1 << 16  # a bound on the shared positions under which every call shares


def shared_inputs(groups, n_q, n_kv, D, page, cache, seed, peak=2.5, loose=LOOSE, alone=()):
    """groups: [(shared length, [(new tokens, tokens after the shared ones, new ones included), ...]), ...]; alone:
    [(new, cached), ...] behind them. A group's full common pages are its first sequence's, the one that the common
    text ends in is copied. Cache rows that no query sees hold NaN, table entries that none needs garbage."""
    g = generator(seed)
    q_lens, kv_lens, starts, shared = [], [], [0], []
    for common, members in groups:
        q_lens += [n for n, _ in members]
        kv_lens += [common + own for _, own in members]
        starts.append(len(q_lens))
        shared.append(common)
    q_lens += [n for n, _ in alone]
    kv_lens += [long for _, long in alone]
    T = sum(q_lens)
    q = (torch.randn(T, n_q, D, generator=g, device=DEV) * (peak / math.sqrt(D))).bfloat16()
    widths = [-(-n // page) for n in kv_lens]
    table = np.full((len(kv_lens), max(-(-max(max(kv_lens), loose + page) // page), 1)), -77, dtype=np.int64)
    used, copied = 0, []
    for i, (common, members) in enumerate(groups):
        for b in range(starts[i], starts[i + 1]):
            full = common // page if b > starts[i] else 0
            table[b, :full] = table[starts[i], :full]
            if b > starts[i] and common % page:
                copied.append((used, table[starts[i], full]))
            table[b, full:widths[b]] = np.arange(used, used + widths[b] - full)
            used += widths[b] - full
    for b in range(starts[-1], len(kv_lens)):
        table[b, :widths[b]] = np.arange(used, used + widths[b])
        used += widths[b]
    pages = used + 3
    order = torch.randperm(pages, generator=g, device=DEV).cpu().numpy()
    table = np.where(table >= 0, order[np.maximum(table, 0)], table)
    kind, scales, host, caches = (torch.bfloat16 if cache == "bf16" else E4M3), {}, {}, []
    for name in "kv":
        x = torch.randn(pages, n_kv, page, D, generator=g, device=DEV)
        if cache == "e4m3":
            scales[name + "_scale"] = torch.rand(n_kv, generator=g, device=DEV) * 0.02 + 0.01
            x = (x / scales[name + "_scale"].view(1, -1, 1, 1)).clamp(-448, 448)
        x = x.to(kind)
        raw = x.view(torch.uint8) if cache == "e4m3" else x.view(torch.int16)
        for to, fr in copied:
            raw[int(order[to])] = raw[int(order[fr])]
        val = f64(x) * (f64(scales[name + "_scale"])[None, :, None, None] if scales else 1.0)
        seen = torch.zeros(pages, page, dtype=torch.bool)
        host[name] = []
        for b, long in enumerate(kv_lens):
            mine = table[b, :widths[b]]
            for j in range(long if q_lens[b] else 0):
                seen[mine[j // page], j % page] = True
            host[name].append(val[mine].transpose(0, 2, 1, 3).reshape(-1, n_kv, D)[:long])
        raw.permute(0, 2, 1, 3)[~seen.to(DEV)] = 0x7F if cache == "e4m3" else 0x7FC0
        caches.append(x)
    return dict(q=q, caches=caches, table=ints(table), starts=ints([0] + list(np.cumsum(q_lens))), lens=ints(kv_lens),
                group_starts=ints(starts), shared=ints(shared), max_q=max(q_lens), max_kv=max(max(kv_lens), loose),
                max_shared=max(max(shared), loose), scales=scales, host=host, q_lens=q_lens, kv_lens=kv_lens)


def attend(x, scale=1.0, **kw):
    return q4.paged_attention_shared(x["q"], *x["caches"], x["table"], x["starts"], x["lens"], x["group_starts"],
                                     x["shared"], x["max_q"], x["max_kv"], x["max_shared"], scale=scale, **x["scales"], **kw)


def need_of(x):
    n_tok, n_q, D = x["q"].shape
    return q4.paged_attention_shared_workspace_bytes(n_tok, x["lens"].numel(), x["shared"].numel(), n_q,
                                                     x["caches"][0].shape[1], D, x["max_q"], x["max_kv"], x["max_shared"])


def expected(x, scale=1.0):
    want, mag, span = so.attention(f64(x["q"]), x["host"]["k"], x["host"]["v"], x["q_lens"], x["kv_lens"], scale, 0)
    return want, so.attention_tolerance(want, mag, span, max(x["kv_lens"]), want.shape[-1])


def check_shared(x, out, scale=1.0):
    want, tol = expected(x, scale)
    got = f64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


ones = lambda n, own: [(1, own + 3 * i) for i in range(n)]  # noqa: E731

# groups, n_q, n_kv, D, page, cache, alone
SHARED = [
    ([(64, ones(2, 1))], 8, 2, 256, 64, "bf16", ()),
    ([(16, ones(3, 1))], 4, 4, 64, 16, "bf16", ()),
    ([(15, ones(3, 5))], 8, 1, 128, 16, "bf16", ()),       # less than a group of 16 keys
    ([(1, ones(2, 1)), (0, ones(2, 20))], 8, 2, 256, 32, "e4m3", ()),
    ([(1000, ones(5, 1))], 8, 2, 256, 64, "bf16", ()),
    ([(1037, ones(9, 40))], 8, 1, 512, 64, "bf16", ()),    # ends inside a page and a group of 16
    ([(700, ones(40, 1))], 8, 2, 256, 64, "bf16", ()),     # many rows
    ([(333, ones(17, 90))], 8, 1, 512, 16, "e4m3", ()),
    ([(2000, ones(33, 5))], 32, 8, 128, 128, "bf16", ()),
    ([(500, ones(70, 1))], 4, 4, 64, 32, "e4m3", ()),
    ([(500, ones(9, 1)), (77, ones(30, 33)), (1200, ones(2, 8))], 8, 2, 256, 32, "e4m3", [(1, 1), (1, 900)]),
    ([(90, ones(3, 1)), (40, ones(1, 7)), (200, ones(4, 50))], 5, 1, 64, 16, "bf16", [(1, 30)]),
    ([(300, [(4, 4), (1, 80), (0, 9), (3, 300), (5, 5)])], 8, 2, 256, 64, "bf16", [(2, 40)]),
    ([(450, [(8, 60), (8, 8), (7, 600)])], 16, 1, 64, 16, "bf16", ()),
    ([(640, [(5, 100 + i) for i in range(16)])], 32, 8, 128, 128, "bf16", ()),
    ([(210, [(3, 60)] * 6), (31, [(2, 2)] * 3)], 10, 2, 128, 32, "e4m3", [(4, 4)]),
    ([(130, [(2, 33)] * 7)], 64, 1, 512, 64, "bf16", ()),  # 128 rows of a sequence
    ([(96, [(1, 10)] * 130)], 6, 2, 64, 16, "bf16", ()),   # more sequences than a wave has lanes
    ([(20 + i, ones(2, 5 + i)) for i in range(70)], 8, 2, 64, 16, "bf16", ()),  # more groups
    ([(48, ones(4, 1)), (3000, ones(50, 200))], 8, 1, 512, 32, "bf16", [(1, 2000)]),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_against_oracle(case):
    groups, n_q, n_kv, D, page, cache, alone = SHARED[case]
    x = shared_inputs(groups, n_q, n_kv, D, page, cache, seed=case, alone=alone)
    err = flag()
    out = attend(x, err_flag=err)
    assert err.item() == 0
    check_shared(x, out)
    assert torch.equal(out, attend(x))


@pytest.mark.parametrize("case", [0, 4, 5, 10, 12, 14])
def test_shared_tight_bounds(case):
    groups, n_q, n_kv, D, page, cache, alone = SHARED[case]
    x = shared_inputs(groups, n_q, n_kv, D, page, cache, seed=case, alone=alone, loose=0)
    check_shared(x, attend(x))


@pytest.mark.parametrize("D,peak,scale", [(256, 40.0, 1.0), (64, 2.5, -0.7), (128, 300.0, 0.03), (512, 2.5, 0.0)])
@pytest.mark.parametrize("members", [2, 20])
def test_shared_peaked_and_other_scales(D, peak, scale, members):
    x = shared_inputs([(330, ones(members, 70))], 8, 2, D, 16, "bf16", seed=D, peak=peak)
    check_shared(x, attend(x, scale=scale), scale)


# ------------------------------------------------------ drafted tokens

FLOATS = ("temperature", "top_p", "min_p")


def draft_inputs(rows, vocab, seed, drafter=True, near=0.5, spread=4.0, **filters):
    """rows: of each sequence. Drafts drawn from the drafter's distribution on the host."""
    g = generator(seed)
    T, B = sum(rows), len(rows)
    z = torch.randn(T, vocab + 3, generator=g, device=DEV)[:, :vocab] * spread
    zd = torch.randn(T, vocab + 5, generator=g, device=DEV)[:, :vocab]
    zd = z + zd * near if near < 10 else zd * spread
    rng = np.random.default_rng(seed)
    par = {n: np.asarray(v if isinstance(v, (list, np.ndarray)) else [v] * B) for n, v in filters.items()}
    drafts = np.full(T, -7, dtype=np.int32)
    starts = np.array([0] + list(np.cumsum(rows)), dtype=np.int32)
    zh = f64(zd)
    for b in range(B):
        for r in range(starts[b], starts[b + 1] - 1):
            q, _ = ro.distribution(zh[r], **{n: v[b] for n, v in par.items()})
            drafts[r] = rng.choice(vocab, p=q / q.sum()) if q.any() else rng.integers(vocab)
    return dict(logits=z, draft_logits=zd if drafter else None, drafts=ints(drafts), starts=ints(starts),
                u=torch.rand(T, generator=g, device=DEV), u_draw=torch.rand(B, generator=g, device=DEV), par=par)


def verify(x, **kw):
    par = {n: torch.tensor(v, dtype=torch.float32 if n in FLOATS else torch.int32, device=DEV) for n, v in x["par"].items()}
    return q4.verify_drafts(x["logits"], x["drafts"], x["starts"], x["u"], x["u_draw"], draft_logits=x["draft_logits"],
                            **par, **kw)


def check_verify(x, got, cap=30.0, draft_cap=None, allow=0.1):
    """Sequences with a decision closer than 2^-20 of what it is part of to its other outcome may have that one (the
    sums are off by at most vocab 2^-43 of the heaviest weight, 2^-23; u and the logits are exact)."""
    tokens, prob, count = (t.cpu().numpy() for t in got)
    zh, uh, wh = f64(x["logits"]), f64(x["u"]), f64(x["u_draw"])
    dh = None if x["draft_logits"] is None else f64(x["draft_logits"])
    starts, drafts, close, stays = x["starts"].cpu().numpy(), x["drafts"].cpu().numpy(), 0, []
    for b in range(len(starts) - 1):
        at = slice(starts[b], starts[b + 1])
        n = starts[b + 1] - starts[b]
        if n == 0:
            assert count[b] == 0
            continue
        want, share, border = ro.check(zh[at], None if dh is None else dh[at], drafts[at], uh[at], wh[b], cap=cap,
                                       draft_cap=cap if draft_cap is None else draft_cap,
                                       **{k: v[b] for k, v in x["par"].items()})
        if border < 2.0 ** -20:
            close += 1
            continue
        assert count[b] == len(want), (b, count[b], want, tokens[at])
        assert list(tokens[at]) == want + [-1] * (n - len(want)), (b, border)
        # 2^-22: the sums' error; 2^-24: the rounding of the result
        np.testing.assert_allclose(prob[at][:len(want)], share, rtol=2.0 ** -22 + 2.0 ** -24)
        assert (prob[at][len(want):] == 0).all()
        stays.append(len(want))
    assert close <= max(1, allow * (len(starts) - 1))
    return stays


VERIFY = [dict(), dict(temperature=0.0), dict(top_k=1), dict(top_k=64, top_p=0.95), dict(top_p=0.9),
          dict(top_p=0.3, temperature=1.7), dict(min_p=0.05), dict(top_k=500, top_p=0.99, min_p=0.001),
          dict(temperature=0.05), dict(temperature=100.0, top_k=700), dict(top_p=0.0), dict(top_k=3, min_p=1.0),
          dict(top_k=300)]


@pytest.mark.parametrize("vocab", [1, 2, 63, 1000, 1025, 50257])
@pytest.mark.parametrize("kw", VERIFY)
@pytest.mark.parametrize("drafter", [True, False])
def test_verify_against_oracle(vocab, kw, drafter):
    x = draft_inputs([4, 1, 2, 6, 0, 3], vocab, seed=vocab, drafter=drafter, **kw)
    got = verify(x)
    check_verify(x, got)
    assert all(torch.equal(a, b) for a, b in zip(got, verify(x)))


def test_verify_rows_with_their_own_settings():
    rows = [3, 1, 5, 2, 4, 4, 0, 8, 2, 1, 3, 70]
    n = len(rows)
    own = dict(temperature=[0.0, 1.0, 0.7, 2.0, 1.0, 0.0, 1.0, 0.3, 1.0, 1.0, 1.3, 1.0],
               top_k=[0, 20, 0, 5, 300, 0, 0, 1, 0, 64, 0, 40], top_p=[1.0, 0.9, 0.5, 1.0, 0.95, 0.2, 1, 1, 0.99, 1.0, 0.8, 1],
               min_p=[0.0, 0.0, 0.02, 0.0, 0.0, 0.5, 0, 0, 0.1, 0.3, 0.0, 0.0])
    assert all(len(v) == n for v in own.values())
    for drafter in (True, False):
        x = draft_inputs(rows, 7000, seed=5, drafter=drafter, **own)
        check_verify(x, verify(x))


@pytest.mark.parametrize("near", [0.0, 0.1, 30.0])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=40), dict(top_p=0.9)])
def test_verify_drafters_near_and_far(near, kw):
    """The same logits: every draft stays, whatever its u. Unlike ones: hardly any."""
    x = draft_inputs([6] * 12, 3000, seed=2, near=near, **kw)
    x["u"][::2] = 1 - 2.0 ** -24
    stays = check_verify(x, verify(x)) if near else [int(c) for c in verify(x)[2]]
    if near == 0.0:
        assert stays == [6] * 12
    elif near == 30.0:
        assert sum(stays) < 30
