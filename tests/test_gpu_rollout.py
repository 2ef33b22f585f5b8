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

LOOSE = 1 << 19  # a bound on the shared positions under which every call here shares


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


def shares(x):
    """Whether the call shares, or leaves it all to paged_attention."""
    n_tok, n_q, D = x["q"].shape
    return need_of(x) != q4.paged_attention_workspace_bytes(x["lens"].numel(), n_q, x["caches"][0].shape[1], D, x["max_q"],
                                                            x["max_kv"])


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
    assert shares(x)
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


# what sharing saves is enough for it under bounds that are the lengths themselves; shared parts by few rows and by many
# (one tile of 128 and several, whose workgroups stand side by side or not), fewer workgroups than compute units and as many
TIGHT = [
    ([(5000, ones(12, 1))], 4, 4, 64, 16, "bf16", ()),
    ([(2000, ones(40, 30))], 32, 8, 64, 64, "e4m3", [(1, 700)]),
    ([(2100, [(5, 70 + i) for i in range(8)])], 32, 8, 128, 128, "bf16", ()),
    ([(2000, [(5, 60)] * 16)], 32, 8, 128, 32, "bf16", ()),
    ([(1000, ones(20, 9)), (2900, ones(14, 1))], 16, 8, 128, 64, "e4m3", [(3, 40)]),
    ([(4013, ones(8, 100))], 8, 2, 256, 64, "bf16", ()),
    ([(2003, ones(15, 20)), (900, ones(3, 3))], 8, 2, 256, 64, "bf16", [(1, 500)]),
    ([(2000, ones(33, 1))], 16, 2, 256, 16, "e4m3", ()),
    ([(7001, ones(8, 50))], 8, 2, 512, 64, "bf16", ()),
    ([(2048, ones(49, 16))], 8, 1, 512, 64, "bf16", ()),
    ([(5000, [(2, 40)] * 20)], 16, 2, 512, 32, "e4m3", [(1, 90)]),
]


@pytest.mark.parametrize("case", range(len(TIGHT)))
def test_shared_under_tight_bounds(case):
    """A workspace of exactly the bytes asked for; what lies behind it stays."""
    groups, n_q, n_kv, D, page, cache, alone = TIGHT[case]
    x = shared_inputs(groups, n_q, n_kv, D, page, cache, seed=case, alone=alone, loose=0)
    assert shares(x) and x["max_kv"] == max(x["kv_lens"]) and x["max_shared"] == max(g[0] for g in groups)
    need = need_of(x)
    room = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device=DEV)
    err = flag()
    out = attend(x, ws=room[:need], err_flag=err)
    assert err.item() == 0 and (room[need:] == 0x5A).all()
    check_shared(x, out)


@pytest.mark.parametrize("D,peak,scale", [(256, 40.0, 1.0), (64, 2.5, -0.7), (128, 300.0, 0.03), (512, 2.5, 0.0)])
@pytest.mark.parametrize("members", [2, 20])
def test_shared_peaked_and_other_scales(D, peak, scale, members):
    x = shared_inputs([(330, ones(members, 70))], 8, 2, D, 16, "bf16", seed=D, peak=peak)
    assert shares(x)
    check_shared(x, attend(x, scale=scale), scale)


def test_shared_leaves_it_to_paged_attention_where_that_is_faster():
    """Prefill chunks, short beginnings, no groups: the same bits as paged_attention's, whatever the groups say."""
    for groups, n_q, n_kv, D, loose in [([(64, [(40, 50), (33, 90)])], 8, 2, 128, LOOSE), ([(40, ones(5, 3))], 8, 2, 64, 0),
                                        ([(300, ones(3, 9))], 8, 1, 512, 0)]:
        x = shared_inputs(groups, n_q, n_kv, D, 16, "bf16", seed=D, loose=loose)
        assert not shares(x)
        want = q4.paged_attention(x["q"], *x["caches"], x["table"], x["starts"], x["lens"], x["max_q"], x["max_kv"])
        assert torch.equal(attend(x), want)
        assert torch.equal(attend(dict(x, shared=x["shared"] * 0 - 5, group_starts=x["group_starts"] * 0 + 99)), want)
    x = shared_inputs([(40, ones(5, 3))], 8, 2, 64, 16, "bf16", seed=1)
    none = dict(x, group_starts=x["group_starts"][:1], shared=x["shared"][:0])
    assert not shares(none)
    check_shared(x, attend(none))


FORMS = [(4, 8, 2, 256), (12, 8, 2, 256), (9, 32, 8, 128), (4, 4, 2, 64), (10, 8, 1, 512), (2, 8, 1, 512)]  # members, heads


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
@pytest.mark.parametrize("how", ["long", "negative", "down", "far", "before"])
def test_shared_bad_groups_share_nothing(members, n_q, n_kv, D, how):
    """The second group's values are out of their ranges: its sequences are read alone, the others as ever."""
    groups = [(200, ones(members, 20)), (150, ones(members, 9)), (90, ones(members, 30))]
    x = shared_inputs(groups, n_q, n_kv, D, 16, "bf16", seed=members)
    assert shares(x)
    if how == "long":
        x["shared"][1] = x["max_shared"] + 1
    elif how == "negative":
        x["shared"][1] = -16
    elif how == "down":
        x["group_starts"][2] = members - 1  # the first two groups overlap in a sequence, the second is none
        x["shared"][2] = 0
    elif how == "far":
        x["group_starts"][3] = 3 * members + 1
    else:
        x["group_starts"][0] = -1
    err = flag()
    out = attend(x, err_flag=err)
    assert err.item() == 1
    check_shared(x, out)


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
@pytest.mark.parametrize("common", [16, 208, 215])
def test_shared_sequences_that_end_where_the_shared_positions_do(members, n_q, n_kv, D, common):
    """A row that sees the shared positions and no more: nothing is left for its own part where they are a multiple of
    16; beside others of its group that go on."""
    for rows in ([(1, 0)] * members, [(1, 0 if i % 2 else 30 + i) for i in range(members)]):
        x = shared_inputs([(common, rows)], n_q, n_kv, D, 16, "bf16", seed=common)
        assert shares(x) and min(x["kv_lens"]) == common
        err = flag()
        out = attend(x, err_flag=err)
        assert err.item() == 0
        check_shared(x, out)


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
def test_shared_groups_of_one_share_nothing(members, n_q, n_kv, D):
    """The sequence of such a group comes out as one of no group does, bit for bit."""
    x = shared_inputs([(150, ones(members, 20)), (170, ones(1, 7)), (40, ones(1, 300))], n_q, n_kv, D, 16, "bf16", seed=members)
    assert shares(x)
    out = attend(x)
    check_shared(x, out)
    x["shared"][1:] = 0
    assert torch.equal(out, attend(x))


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
@pytest.mark.parametrize("how", ["second", "far back", "last"])
def test_shared_groups_that_overlap_share_nothing(members, n_q, n_kv, D, how):
    """group_starts that decrease: two groups of valid values name the same sequences, with unlike shared lengths. All
    are read alone, and nothing of an earlier call in the same workspace comes out."""
    groups = [(200, ones(members, 20)), (150, ones(members, 9)), (90, ones(members, 30)), (60, ones(2, 5))]
    x = shared_inputs(groups, n_q, n_kv, D, 16, "bf16", seed=members)
    assert shares(x)
    ws = torch.empty(need_of(x), dtype=torch.uint8, device=DEV)
    attend(dict(x, q=-2 * x["q"]), ws=ws)
    where, to = {"second": (2, members - 1), "far back": (3, 0), "last": (4, 1)}[how]
    x["group_starts"][where] = to
    err = flag()
    out = attend(x, ws=ws, err_flag=err)
    assert err.item() == 1
    check_shared(x, out)


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
@pytest.mark.parametrize("how", ["back", "early", "again"])
def test_shared_sequences_that_overlap(members, n_q, n_kv, D, how):
    """q_starts that decrease: rows of one valid sequence are as ever, those that none names stay, whatever an earlier
    call has left in the workspace; of rows that two sequences name nothing is asked."""
    n = 3 if n_q // n_kv * 3 <= 128 else 2
    groups = [(130, [(n, 20 + i) for i in range(members)]), (64, [(n, 40)] * 30)]
    x = shared_inputs(groups, n_q, n_kv, D, 16, "bf16", seed=members)
    total = members + 30
    ws = torch.empty(need_of(x), dtype=torch.uint8, device=DEV)
    assert shares(x)
    want, tol = expected(x)
    for other in (-2 * x["q"], x["q"].roll(7, 0)):
        attend(dict(x, q=other), ws=ws)
    starts = x["starts"].cpu().numpy().copy()
    if how == "back":
        starts[total - 5] = 1
    elif how == "early":
        starts[1] = n * total - 1
    else:
        starts[1:total - 6] = np.resize([n, 0], total - 7)  # many sequences of the same rows: more than there are slots
    x["starts"] = ints(starts)
    named = np.zeros(n * total, int)
    right = np.zeros(n * total, bool)
    for b in range(total):
        if 0 <= starts[b] <= starts[b + 1] <= n * total and starts[b + 1] - starts[b] <= n:
            named[starts[b]:starts[b + 1]] += 1
            if starts[b] == n * b and starts[b + 1] == n * b + n:
                right[n * b:n * b + n] = True
    err = flag()
    out = attend(x, ws=ws, out=torch.full_like(x["q"], 7.0), err_flag=err)
    assert err.item() == 1
    right &= named == 1
    assert right.sum() >= 4 * n and (named == 0).any()
    assert (np.abs(f64(out) - want) <= tol)[right].all()
    assert (out[torch.from_numpy(named == 0).to(DEV)] == 7.0).all()


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
@pytest.mark.parametrize("common", [208, 215])
def test_shared_sequences_that_do_not_see_it_all_are_read_alone(members, n_q, n_kv, D, common):
    """Shared lengths beyond a sequence's rows, or beyond all of it: nothing of it is taken from the group, also not the
    whole groups of 16 that it does see."""
    x = shared_inputs([(common, ones(members, 20))], n_q, n_kv, D, 16, "bf16", seed=members + 1,
                      alone=[(1, 100), (1, 208), (2, 208), (1, 1)])
    n = members + 4
    x["group_starts"][1] = n  # the alone ones hold other tokens: they are right only if they are read alone
    x["lens"][members + 1] = 207
    for c in "kv":
        x["host"][c][members + 1] = x["host"][c][members + 1][:207]
    x["kv_lens"][members + 1] = 207
    assert shares(x)
    err = flag()
    check_shared(x, attend(x, err_flag=err))
    assert err.item() == 0


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
def test_shared_invalid_sequences_are_left_alone(members, n_q, n_kv, D):
    for spoil in ("kv_negative", "kv_long", "q_long", "starts_far"):
        x = shared_inputs([(130, [(2, 20 + i) for i in range(members)])], n_q, n_kv, D, 16, "bf16", seed=3)
        assert shares(x)
        want, tol = expected(x)
        bad = {1}
        if spoil == "kv_negative":
            x["lens"][1] = -5
        elif spoil == "kv_long":
            x["lens"][1] = x["max_kv"] + 1
        elif spoil == "q_long":
            x["starts"][2] += 1  # 1 has a row more than max_q_len, 2 one fewer
            bad = {1, 2}
        else:
            x["starts"][members] = 2 * members + 1  # the group is no longer valid either
            bad = {members - 1}
        if members == 2 and spoil == "q_long":
            continue
        err = flag()
        out = attend(x, out=torch.full_like(x["q"], 7.0), err_flag=err)
        assert err.item() == 1, spoil
        for b in range(members):
            rows = slice(2 * b, 2 * b + 2)
            if b not in bad:
                assert (np.abs(f64(out[rows]) - want[rows]) <= tol[rows]).all(), (spoil, b)
            elif spoil != "q_long":
                assert (out[rows] == 7.0).all(), (spoil, b)


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
def test_shared_rows_outside_every_sequence_stay(members, n_q, n_kv, D):
    x = shared_inputs([(100, ones(members, 9))], n_q, n_kv, D, 16, "bf16", seed=2)
    pad = torch.randn(5, n_q, D, device=DEV).bfloat16()
    y = dict(x, q=torch.cat([pad[:2], x["q"], pad[2:]]), starts=x["starts"] + 2)
    for fill in (0, 255, 1):
        ws = torch.full((need_of(y),), fill, dtype=torch.uint8, device=DEV)
        attend(x, ws=ws[:need_of(x)])  # (what another call has left)
        out = attend(y, out=torch.full_like(y["q"], 3.0), ws=ws)
        check_shared(x, out[2:-3])
        assert (out[:2] == 3.0).all() and (out[-3:] == 3.0).all()


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
def test_shared_bad_pages_are_not_seen(members, n_q, n_kv, D):
    """A page number out of range hides its positions from all of the group, or behind the shared ones from one."""
    x = shared_inputs([(160, ones(members, 40))], n_q, n_kv, D, 16, "bf16", seed=4)
    for bad in (-1, x["caches"][0].shape[0], 1 << 30, -(1 << 31)):
        for page, hit in ((3, range(members)), (11, [1])):
            y = dict(x, table=x["table"].clone())
            y["table"][0 if page == 3 else 1, page] = bad
            err = flag()
            out = attend(y, err_flag=err)
            assert err.item() == 1
            cut = lambda h, b: np.delete(h, range(16 * page, 16 * page + 16), 0) if b in hit else h  # noqa: E731
            host = {c: [cut(h, b) for b, h in enumerate(x["host"][c])] for c in "kv"}
            lens = [len(h) for h in host["k"]]
            check_shared(dict(x, host=host, kv_lens=lens), out)


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("place", ["shared", "own"])
def test_shared_nonfinite_keys_and_values(members, n_q, n_kv, D, cache, place):
    """A NaN key makes the rows that see it NaN, a NaN value their column of it, an infinite value that infinity; the
    other rows and columns are as without."""
    x = shared_inputs([(170, ones(members, 20))], n_q, n_kv, D, 16, cache, seed=8)
    want, tol = expected(x)
    group, pos = n_q // n_kv, 37 if place == "shared" else 171
    sees = np.ones(members, bool) if place == "shared" else np.arange(members) == 1
    mine = slice((n_kv - 1) * group, n_q)
    page = int(x["table"][0 if place == "shared" else 1, pos // 16])
    for which, value in ((0, math.nan), (1, math.nan), (1, math.inf), (1, -math.inf)):
        if cache == "e4m3" and not math.isnan(value):
            continue  # (it has no infinity)
        y = dict(x, caches=[c.clone() for c in x["caches"]])
        if cache == "e4m3":
            y["caches"][which].view(torch.uint8)[page, n_kv - 1, pos % 16, 5] = 0x7F
        else:
            y["caches"][which][page, n_kv - 1, pos % 16, 5] = value
        got = f64(attend(y))
        hit = np.zeros(got.shape, bool)
        hit[sees, mine] = True if which == 0 else np.arange(D) == 5
        if math.isnan(value):
            assert np.isnan(got[hit]).all()
        else:
            assert (got[hit] == value).all()
        assert (np.abs(got - want) <= tol)[~hit].all()


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
def test_shared_scores_of_minus_infinity(members, n_q, n_kv, D):
    """Of all shared keys: the rows are what their own keys make them; of all keys: 0 / 0, NaN."""
    x = shared_inputs([(176, ones(members, 20))], n_q, n_kv, D, 16, "bf16", seed=9)
    x["q"] = x["q"].abs().clamp(min=0.01)
    y = dict(x, caches=[x["caches"][0].clone(), x["caches"][1]])
    pages = x["table"][0, :11].long()
    y["caches"][0][pages, :, :, 5] = -math.inf
    host = {c: [h[176:] for h in x["host"][c]] for c in "kv"}
    check_shared(dict(x, host=host, kv_lens=[len(h) for h in host["k"]]), attend(y))
    y["caches"][0][..., 5] = -math.inf
    assert torch.isnan(attend(y)).all()
    y["table"] = y["table"] * 0 - 1  # and with no page there: nothing is seen
    assert not attend(y).any()


@pytest.mark.parametrize("members,n_q,n_kv,D", FORMS)
def test_shared_streams_graphs_and_dirty_workspaces(members, n_q, n_kv, D):
    """Two calls at once with workspaces of their own; a captured call follows lengths, rows and groups that change on
    the device; two graphs share one workspace one after the other."""
    groups = [(260, [(2, 20 + i) for i in range(members)]), (70, [(1, 30)] * members)]
    x = shared_inputs(groups, n_q, n_kv, D, 16, "bf16", seed=5, alone=[(2, 50)])
    other = shared_inputs([(123, ones(members, 70))], n_q, n_kv, D, 32, "bf16", seed=6)
    want, want_other = attend(x), attend(other)
    check_shared(x, want)
    need = max(need_of(x), need_of(other))
    ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in "ab"]
    outs = [torch.empty_like(x["q"]) for _ in "ab"]
    streams = [torch.cuda.Stream() for _ in "ab"]
    for fill in (0, 255, 127):
        for w, o in zip(ws, outs):
            w.fill_(fill)
            o.fill_(9.0)
        torch.cuda.synchronize()
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                for _ in range(5):
                    attend(x, ws=w, out=o)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    out_other = torch.empty_like(other["q"])
    graphs = []
    for order in (0, 1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for which in ((x, outs[0]), (other, out_other))[::1 if order else -1]:
                attend(which[0], ws=ws[0], out=which[1])
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            outs[0].zero_()
            out_other.zero_()
            graph.replay()
            noise = attend(x, ws=ws[0])
            torch.cuda.synchronize()
            assert torch.equal(noise, want) and torch.equal(outs[0], want) and torch.equal(out_other, want_other)
    # the first sequence gives up a row, the second all of them; the first group shares less, the second nothing
    q_lens, kv_lens = list(x["q_lens"]), list(x["kv_lens"])
    q_lens[0], kv_lens[0], q_lens[1] = 1, kv_lens[0] - 1, 0
    starts = np.array([0] + list(np.cumsum(q_lens)), dtype=np.int32)
    x["starts"].copy_(torch.from_numpy(starts))
    x["lens"].copy_(torch.tensor(kv_lens, dtype=torch.int32))
    x["shared"].copy_(torch.tensor([100, 0], dtype=torch.int32))
    x["group_starts"].copy_(torch.tensor([0, members, members], dtype=torch.int32))
    host = {c: [h[:n] for h, n in zip(x["host"][c], kv_lens)] for c in "kv"}
    total = int(starts[-1])
    for _ in range(2):
        outs[0].fill_(9.0)
        graphs[0].replay()
        torch.cuda.synchronize()
        assert (outs[0][total:] == 9.0).all()
        check_shared(dict(x, q=x["q"][:total], host=host, q_lens=q_lens, kv_lens=kv_lens), outs[0][:total])


def test_shared_cache_past_four_gib_elements():
    """Pages whose element offsets pass 2^32: 70000 pages of 64 rows x 2 heads x 512 values, 9.2 GB each."""
    pages, n_kv, page, D = 70000, 2, 64, 512
    small = shared_inputs([(130, ones(3, 5))], 8, n_kv, D, page, "bf16", seed=12)
    caches = [torch.empty(pages, n_kv, page, D, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    held = small["caches"][0].shape[0]
    used = torch.tensor([69999 - 131 * i if i % 2 else i for i in range(held)], dtype=torch.int32, device=DEV)
    for big, c in zip(caches, small["caches"]):
        big[used.long()] = c
    table = torch.where(small["table"] >= 0, used[small["table"].clamp(min=0).long()], small["table"])
    assert shares(small)
    assert torch.equal(attend(dict(small, caches=caches, table=table.contiguous())), attend(small))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("groups,n_q,n_kv,D,alone", [
    ([(5000, ones(30, 40))], 8, 2, 256, ()), ([(3000, ones(20, 1)), (1500, ones(50, 300))], 8, 1, 512, [(1, 2500)]),
    ([(2600, [(5, 60)] * 20)], 32, 8, 128, ()), ([(7000, ones(9, 1000))], 4, 1, 64, ()),
    ([(4000, ones(4, 3000))], 8, 2, 256, ()),
])
def test_shared_cut_over_workgroups(groups, n_q, n_kv, D, alone, cache):
    x = shared_inputs(groups, n_q, n_kv, D, 64, cache, seed=D, alone=alone)
    check_shared(x, attend(x))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("members,n,group,D", [(3, 1, 4, 64), (40, 1, 4, 64), (7, 5, 4, 128), (33, 1, 8, 256), (2, 4, 8, 256),
                                               (2, 1, 8, 512), (19, 2, 8, 512), (3, 2, 64, 128)])
def test_shared_keeps_sixteen_bits_of_a_probability(members, n, group, D, cache):
    """As test_attention_few_rows_keep_sixteen_bits_of_a_probability: keys of two kinds by turns, of probability 1 and p,
    with values that all but cancel, 288 of them shared. In two bf16 parts a probability is off by 2^-16, in one p is
    off by more than 2^-10. The rows of one sequence by itself have two parts, and so have all of a group together."""
    score, c = -1.375, 4.0
    p = math.exp(score)
    assert abs(float(torch.tensor(p).bfloat16()) / p - 1) > 2.0 ** -10 and abs(p * c - 1) < 0.1
    common, long, page, kind = 288, 288 + n + 7, 16, torch.bfloat16 if cache == "bf16" else E4M3
    g = generator(D + n)
    pages = -(-long // page)
    k, v = torch.zeros(long, D, device=DEV), torch.empty(long, D, device=DEV)
    sign = torch.randint(0, 2, (D,), generator=g, device=DEV) * 2.0 - 1
    v[::2], v[1::2], k[1::2, 0] = sign, -sign * c, score
    k[:, 1:] = torch.randint(-2, 3, (long, D - 1), generator=g, device=DEV)  # (met by zeros of q)
    q = torch.zeros(members * n, group, D, device=DEV)
    q[..., 0] = 1.0
    room = lambda x: torch.cat([x, x.new_zeros(pages * page - long, D)]).view(pages, 1, page, D).to(kind)  # noqa: E731
    table = torch.full((members, LOOSE // page), -1, dtype=torch.int32, device=DEV)
    table[:, :pages] = torch.arange(pages, dtype=torch.int32, device=DEV)
    x = dict(q=q.bfloat16(), caches=[room(k), room(v)], table=table, starts=ints(range(0, members * n + 1, n)),
             lens=ints([long] * members), group_starts=ints([0, members]), shared=ints([common]), max_q=n, max_kv=LOOSE,
             max_shared=LOOSE, scales={})
    assert shares(x)
    kh, vh = f64(k)[:, None], f64(v)[:, None]
    want, mag, span = so.attention(f64(x["q"]), [kh] * members, [vh] * members, [n] * members, [long] * members, 1.0, 0)
    ds = (D + 4) * 2.0 ** -24 * span[..., None]
    inner = mag * (2 * (1.1 * ds + 2.0 ** -21 + (long + 8) * 2.0 ** -24) + 2.0 ** -16)
    tol = inner + 2.0 ** -8 * (np.abs(want) + inner)
    assert (np.abs(f64(attend(x)) - want) <= tol).all()
    # the bound tells one part from two: the oracle with the shared probabilities rounded once lies outside
    at = long - n + np.tile(np.arange(n), members)
    w = np.where(np.arange(long) % 2, p, 1.0) * (np.arange(long)[None] <= at[:, None])
    r = np.where(np.arange(long) < common, so.bf16_round(w), w)
    once = (r @ vh[:, 0]) / w.sum(-1, keepdims=True)
    assert (np.abs(once[:, None] - want) > tol).all()


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


def check_verify(x, got, cap=30.0, draft_cap=None, allow=0.1, near=None):
    """Sequences with a decision closer to its other outcome than the sums' errors may have that one (u and the logits
    are exact): a sum of weights is off by at most half a step of 2^-42 of the heaviest for each token, and 2^-33 of
    itself; there are two of them, of p and of q, in what is compared, and each distribution is also divided by one."""
    near = near or 4 * (x["logits"].shape[1] * 2.0 ** -43 + 2.0 ** -33)
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
        if border < near:
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


@pytest.mark.parametrize("kw", [dict(), dict(top_p=0.9), dict(top_k=40, top_p=0.95), dict(top_k=700, min_p=0.01)])
@pytest.mark.parametrize("vocab", [262144, 262145, 1 << 20])
def test_verify_wide_vocabularies(vocab, kw):
    x = draft_inputs([3, 1, 2], vocab, seed=1, **kw)
    check_verify(x, verify(x), allow=0.34)


def test_verify_single_rows_draw_what_sampling_draws():
    """A sequence of one row has no draft: the token and its share are sample_logits', bit for bit where the filters
    are the same code, to the sums' error without filters."""
    B = 40
    for kw in (dict(top_k=50, top_p=0.9), dict(top_p=0.8), dict(min_p=0.02), dict(temperature=0.0), dict()):
        x = draft_inputs([1] * B, 30011, seed=B, **kw)
        tokens, prob, count = verify(x)
        par = {n: torch.tensor(v, dtype=torch.float32 if n in FLOATS else torch.int32, device=DEV) for n, v in x["par"].items()}
        idx, share = q4.sample_logits(x["logits"], x["u_draw"], **par)
        assert (count == 1).all() and torch.equal(tokens, idx)
        if kw:
            assert torch.equal(prob, share)
        else:
            assert ((prob - share).abs() <= share * 2.0 ** -23).all()


def test_verify_special_values():
    """NaN and -infinity are never drawn, +infinity always; rows of nothing else give -1 and NaN; of the drafter's rows
    nothing is then taken off."""
    g = generator(7)
    V = 500
    inf, nan = math.inf, math.nan
    for kw in (dict(), dict(top_k=20), dict(top_p=0.9), dict(temperature=0.0), dict(min_p=0.1)):
        for drafter in (True, False):
            x = draft_inputs([3] * 8, V, seed=3, drafter=drafter, **kw)
            z = x["logits"] = x["logits"].contiguous()
            d = x["draft_logits"] = x["draft_logits"].contiguous() if drafter else None
            z[0, ::2], z[3, 7], z[6] = -inf, inf, -inf
            z[9], z[12, 1:], z[15, 3:9] = nan, -inf, nan
            z[18:21] = torch.randint(0, 2, (3, V), generator=g, device=DEV) * 2.0  # many equal ones
            z[22], z[21, 400:] = 1e30, -1e30
            if drafter:
                d[0, ::3], d[1], d[4, 5], d[16, 2] = -inf, -inf, inf, nan
                d[19] = z[19]
            got = verify(x)
            tokens, prob, count = (t.cpu().numpy() for t in got)
            starts, close = x["starts"].cpu().numpy(), 0
            zh, uh, wh, dh = f64(z), f64(x["u"]), f64(x["u_draw"]), None if d is None else f64(d)
            for b in range(8):
                at = slice(3 * b, 3 * b + 3)
                want, share, border = ro.check(zh[at], None if dh is None else dh[at], x["drafts"].cpu().numpy()[at], uh[at],
                                               wh[b], **{k: v[b] for k, v in x["par"].items()})
                if border < 2.0 ** -30:  # (vocab 2^-41 and 2^-31, as in check_verify)
                    close += 1
                    continue
                assert list(tokens[at]) == want + [-1] * (3 - len(want)), (kw, drafter, b)
                np.testing.assert_allclose(prob[at][:len(want)], share, rtol=2.0 ** -22 + 2.0 ** -24)
                assert count[b] == len(want)
            assert close <= 2


@pytest.mark.parametrize("heat", [1.0, 0.01, 1e-6, 1e-30, 1e4])
@pytest.mark.parametrize("cap,draft_cap,spread", [(30.0, 30.0, 30.0), (0.0, 0.0, 4.0), (30.0, 0.0, 8.0), (5.0, 50.0, 4.0),
                                                  (math.inf, 30.0, 4.0)])
def test_verify_caps_and_temperatures(heat, cap, draft_cap, spread):
    """Logits far above the cap, no cap, unlike caps, and temperatures at which the octaves' constant is large."""
    x = draft_inputs([4] * 6, 2000, seed=11, spread=spread, temperature=heat)
    used = [0.0 if not math.isfinite(c) else c for c in (cap, draft_cap)]
    got = verify(x, cap=cap, draft_cap=draft_cap)
    check_verify(x, got, cap=used[0], draft_cap=used[1], allow=0.5)


@pytest.mark.parametrize("heat", [0.02, 0.05, 0.3])
def test_verify_weights_of_cold_rows(heat):
    """Rows without filters whose largest logit is far from 0 against the temperature, with u the fp32 number nearest
    to the draft's probability p: which side of p it lies on is told as soon as it is off by 2^-32.4 of p. (The sum of
    weights may be off by 2^-33, a weight by ln 2 * 30 log2(e) / heat * 2^-45.9, tanh's error, at most 2^-35.4, and
    each of the 8 weights by half a step of 2^-42.)"""
    N, V = 16000, 8
    z = (13.3 + torch.randn(2 * N, V, generator=generator(15), device=DEV) * heat).clamp(max=13.49)
    t = np.tanh(f64(z[::2]).astype(np.longdouble) / 30) * 30 / np.float32(heat)
    w = np.exp(t - t.max(-1, keepdims=True))
    p = (w / w.sum(-1, keepdims=True))[:, 3]
    u = p.astype(np.float32)
    far = np.abs(u - p) / p
    told = (p < 0.9) & (far > 2.0 ** -32.4)
    assert (told & (far < 2.0 ** -30.5)).sum() > 100
    x = torch.zeros(2 * N, device=DEV)
    x[::2] = torch.from_numpy(u).to(DEV)
    count = q4.verify_drafts(z, torch.full((2 * N,), 3, dtype=torch.int32, device=DEV), ints(range(0, 2 * N + 1, 2)), x,
                             torch.zeros(N, device=DEV), temperature=torch.full((N,), heat, device=DEV))[2].cpu().numpy()
    assert ((count == 2) == (u < p))[told].all(), ((count == 2) != (u < p))[told].sum()


@pytest.mark.parametrize("masked", [-1e4, -math.inf])
@pytest.mark.parametrize("kw", [dict(top_k=64), dict(top_p=0.95), dict()])
def test_verify_masked_tokens(masked, kw):
    """A grammar that leaves 30 tokens of 40000: under a small top_k finite masks overflow the list of candidates."""
    x = draft_inputs([3, 2], 40000, seed=4, **kw)
    z, d = x["logits"].contiguous(), x["draft_logits"].contiguous()
    keep = torch.randperm(40000, generator=generator(1), device=DEV)[:30]
    for t in (z, d):
        hold = t[:, keep].clone()
        t.fill_(masked)
        t[:, keep] = hold
    x.update(logits=z, draft_logits=d)
    x["drafts"] = keep[:5].int().contiguous()
    check_verify(x, verify(x), allow=0.5)


def test_verify_bad_drafts_and_numbers():
    """A draft out of range does not stay and sets the flag; numbers outside [0, 1) are clamped into it, NaN is 0."""
    for drafter in (True, False):
        for bad in (-1, 900, -(1 << 31), (1 << 31) - 1):
            x = draft_inputs([4, 3], 900, seed=6, drafter=drafter, near=0.0)
            x["u"].zero_()
            assert [int(c) for c in verify(x)[2]] == [4, 3]
            x["drafts"][1] = bad
            err = flag()
            got = verify(x, err_flag=err)
            assert err.item() == 1
            check_verify(x, got)
            assert [int(c) for c in got[2]] == [2, 3]
            x["drafts"][1] = 0
            x["drafts"][3] = bad  # of a sequence's last row: not looked at
            err = flag()
            verify(x, err_flag=err)
            assert err.item() == 0
        x = draft_inputs([5] * 6, 900, seed=6, drafter=drafter)
        odd = torch.tensor([-1.0, 1.0, 2.0, math.nan, math.inf, -math.inf], device=DEV)
        x["u"][:30:5], x["u_draw"] = odd, odd.roll(2).contiguous()
        check_verify(x, verify(x), allow=0.4)


def test_verify_bad_sequences_are_left_alone():
    rows = [3, 4, 2, 5]
    for spoil in ("down", "negative", "far"):
        x = draft_inputs(rows, 3000, seed=8)
        want = verify(x)
        bad = {"down": {1}, "negative": {0}, "far": {3}}[spoil]
        if spoil == "down":
            # the second ends before it begins; the third names its rows and two of the first's, and what rows that two
            # sequences name hold is not defined (include/q4dec_rollout.h): the fourth is as ever
            x["starts"][2] = 1
            bad = {0, 1, 2}
        elif spoil == "negative":
            x["starts"][0] = -1
        else:
            x["starts"][4] = 15
        err = flag()
        outs = [torch.full_like(t, 77) for t in want]
        verify(x, tokens_out=outs[0], prob_out=outs[1], count_out=outs[2], err_flag=err)
        assert err.item() == 1
        for b, (s, n) in enumerate(zip([0, 3, 7, 9], rows)):
            if b not in bad:
                assert torch.equal(outs[0][s:s + n], want[0][s:s + n]) and outs[2][b] == want[2][b]
                assert torch.equal(outs[1][s:s + n], want[1][s:s + n])
            elif spoil != "down":
                assert (outs[0][s:s + n] == 77).all() and (outs[1][s:s + n] == 77).all() and outs[2][b] == 77


@pytest.mark.parametrize("kw", [dict(), dict(top_k=20)])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("n,where", [(4, 2), (4, 1), (64, 32), (65, 63), (128, 64), (128, 65), (300, 5), (300, 299)])
def test_verify_one_bad_start_spoils_its_own_sequences_only(n, where, drafter, kw):
    """The start `where` is out of range: the sequence before it and its own are left as they are, every other is as
    without it, bit for bit."""
    rows = [1 + i % 3 for i in range(n)]
    x = draft_inputs(rows, 200, seed=n, drafter=drafter, **kw)
    want = verify(x)
    total, at = sum(rows), np.array([0] + list(np.cumsum(rows)))
    for value in (-1, -(1 << 31), total + 1, (1 << 31) - 1):
        y = dict(x, starts=x["starts"].clone())
        y["starts"][where] = value
        err = flag()
        outs = [torch.full_like(t, 77) for t in want]
        verify(y, tokens_out=outs[0], prob_out=outs[1], count_out=outs[2], err_flag=err)
        assert err.item() == 1
        expect = [t.clone() for t in want]
        for b in (where - 1, where):
            expect[0][at[b]:at[b + 1]], expect[1][at[b]:at[b + 1]], expect[2][b] = 77, 77.0, 77
        for got, w in zip(outs, expect):
            assert torch.equal(got, w), (value, (got != w).nonzero().flatten().tolist()[:8])


def test_verify_rows_of_no_sequence_stay_and_strides():
    x = draft_inputs([2, 3], 777, seed=9, top_p=0.9)
    want = verify(x)
    y = dict(x)
    for name in ("logits", "draft_logits"):
        room = torch.full((9, 1000), math.nan, device=DEV)
        room[2:7, :777] = x[name]
        y[name] = room[:, :777]
    y.update(starts=x["starts"] + 2, drafts=torch.nn.functional.pad(x["drafts"], (2, 2), value=-9),
             u=torch.nn.functional.pad(x["u"], (2, 2)))
    outs = [torch.full((9,), 77, dtype=torch.int32, device=DEV), torch.full((9,), 77.0, device=DEV)]
    err = flag()
    count = verify(y, tokens_out=outs[0], prob_out=outs[1], err_flag=err)[2]
    assert err.item() == 0 and torch.equal(count, want[2])
    for o, w in zip(outs, want):
        assert torch.equal(o[2:7], w) and (o[:2] == 77).all() and (o[7:] == 77).all()


def test_verify_nearly_certain_drafts_taken_back():
    """A draft of probability about 1 - 1e-6 that is taken back all the same: what is left is the others' millionth. Its
    sums are off by half a step of 2^-42 for each token, and 2^-33 of themselves (of 1e-5 here at most). Of 300 tokens
    that tells most draws apart, of 40009 none: there the draw has to be one of the others."""
    for V in (300, 40009):
        for heat in (1.0, 0.05):
            x = draft_inputs([3] * 12, V, seed=V, drafter=False, temperature=heat)
            z = x["logits"] = torch.randn(36, V, generator=generator(2), device=DEV)
            top = torch.randint(0, V, (36,), generator=generator(3), device=DEV)
            z[torch.arange(36, device=DEV), top] = heat * (math.log(1e6) + torch.logsumexp(z / heat, -1))
            x["drafts"], x["u"] = top.int(), torch.full((36,), 1 - 2.0 ** -24, device=DEV)
            x["u"][::3] = 0.5
            got = verify(x, cap=0.0)
            stays = check_verify(x, got, cap=0.0, near=4 * (V * 2.0 ** -43 + 1e-5 * 2.0 ** -33), allow=0.5 if V == 300 else 1.0)
            assert V > 300 or len(stays) >= 6
            new = got[0][torch.arange(0, 36, 3, device=DEV) + got[2] - 1]
            assert (got[2] == 2).sum() > 6 and ((new >= 0) & (new < V)).all()
            assert (new != top[torch.arange(0, 36, 3, device=DEV) + got[2] - 1])[got[2] < 3].all()


def test_verify_tails_that_round_to_nothing():
    """All tokens but one lighter than 2^-43 of it: they are never drawn, however many they are, also where the one is
    a draft that is taken back."""
    V = 1 << 20
    z = torch.zeros(4, V, device=DEV)
    z[:, 77] = 43.2 * math.log(2.0)
    drafts = torch.full((4,), 77, dtype=torch.int32, device=DEV)
    u = torch.tensor([1 - 2.0 ** -24] * 4, device=DEV)
    for start in ([0, 1, 2, 3, 4], [0, 2, 4]):
        n = len(start) - 1
        tokens, prob, count = q4.verify_drafts(z, drafts, ints(start), u, u[:n].contiguous(), cap=0.0)
        first = [int(tokens[s]) for s in start[:-1]]
        assert first == [77] * n and (prob[start[:-1]] > 0.999).all()


def test_verify_leaves_the_target_distribution():
    """Drafts drawn from q, 32000 sequences of one draft in 4 calls: the first token is distributed as p (chi-square
    with 11 degrees of freedom, 60 is past 1e-8 of it), whatever q."""
    g = generator(10)
    V, N = 12, 8000
    for near in (0.5, 2.0):
        p_logits = torch.randn(V, generator=g, device=DEV) * 1.5
        q_logits = p_logits + near * torch.randn(V, generator=g, device=DEV)
        seen = np.zeros(V)
        q = torch.softmax(30 * torch.tanh(q_logits.double() / 30), 0)
        for _ in range(4):
            drafts = torch.zeros(2 * N, dtype=torch.int32, device=DEV)
            drafts[::2] = torch.multinomial(q, N, replacement=True, generator=g).int()
            got = q4.verify_drafts(p_logits.expand(2 * N, V).contiguous(), drafts,
                                   torch.arange(0, 2 * N + 1, 2, dtype=torch.int32, device=DEV),
                                   torch.rand(2 * N, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV),
                                   draft_logits=q_logits.expand(2 * N, V).contiguous())
            seen += np.bincount(got[0][::2].cpu().numpy(), minlength=V)
        p = ro.distribution(f64(p_logits))[0]
        assert (((seen - 4 * N * p) ** 2) / (4 * N * p)).sum() < 60


@pytest.mark.parametrize("kw", [dict(), dict(top_k=30, top_p=0.95), dict(top_p=0.9), dict(min_p=0.05)])
@pytest.mark.parametrize("drafter", [True, False])
def test_verify_streams_graphs_and_dirty_workspaces(kw, drafter):
    """Two calls at once with workspaces of their own; a captured call follows logits, numbers and rows that change on
    the device; two graphs share one workspace one after the other."""
    x = draft_inputs([4, 3, 1, 6], 40009, seed=12, drafter=drafter, **kw)
    other = draft_inputs([2, 5, 5], 5000, seed=13, drafter=drafter, **kw)
    want, want_other = verify(x), verify(other)
    need = max(q4.verify_drafts_workspace_bytes(x_["logits"].shape[0], x_["starts"].numel() - 1, x_["logits"].shape[1], drafter)
               for x_ in (x, other))
    ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in "ab"]
    fresh = lambda w: [torch.empty_like(t) for t in w]  # noqa: E731
    named = lambda o: dict(tokens_out=o[0], prob_out=o[1], count_out=o[2])  # noqa: E731
    outs = [fresh(want), fresh(want)]
    streams = [torch.cuda.Stream() for _ in "ab"]
    for fill in (0, 255, 127):
        for w, o in zip(ws, outs):
            w.fill_(fill)
            for t in o:
                t.fill_(9)
        torch.cuda.synchronize()
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                for _ in range(4):
                    verify(x, ws=w, **named(o))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    out, out_other = fresh(want), fresh(want_other)
    par = {n: torch.tensor(v, dtype=torch.float32 if n in FLOATS else torch.int32, device=DEV) for n, v in x["par"].items()}
    par_other = {n: v[:3].contiguous() for n, v in par.items()}
    call = lambda x_, p, o: q4.verify_drafts(x_["logits"], x_["drafts"], x_["starts"], x_["u"], x_["u_draw"],  # noqa: E731
                                             draft_logits=x_["draft_logits"], ws=ws[0], **p, **named(o))
    graphs = []
    for order in (1, -1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for args in ((x, par, out), (other, par_other, out_other))[::order]:
                call(*args)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            for t in out + out_other:
                t.zero_()
            graph.replay()
            noise = verify(x, ws=ws[0])
            torch.cuda.synchronize()
            for got, w in ((noise, want), (out, want), (out_other, want_other)):
                assert all(torch.equal(a, b) for a, b in zip(got, w))
    new = draft_inputs([4, 3, 1, 6], 40009, seed=14, drafter=drafter, **kw)
    for name in ("logits", "draft_logits", "drafts", "u", "u_draw"):
        if x[name] is not None:
            x[name].copy_(new[name])
    x["starts"].copy_(ints([0, 2, 7, 7, 13]))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert out[2][2] == 0
    got = verify(x)
    assert all(torch.equal(a[:13], b[:13]) for a, b in zip(out[:2], got[:2])) and torch.equal(out[2], got[2])
    check_verify(x, got)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=30, top_p=0.95)])
def test_verify_many_sequences_in_a_captured_call(kw):
    """More sequences than a wave has lanes, whose rows change on the device: the replay follows, and the rows behind
    the last of them stay."""
    rows = [1 + i % 4 for i in range(150)]
    x = draft_inputs(rows, 700, seed=16, **kw)
    total = sum(rows)
    starts = [x["starts"].clone(), ints([0] + list(np.cumsum([2 - i % 2 for i in range(150)])))]
    ws = torch.empty(q4.verify_drafts_workspace_bytes(total, 150, 700, True), dtype=torch.uint8, device=DEV)
    outs = [torch.empty(total, dtype=torch.int32, device=DEV), torch.empty(total, device=DEV),
            torch.empty(150, dtype=torch.int32, device=DEV)]
    par = {n: torch.tensor(v, dtype=torch.float32 if n in FLOATS else torch.int32, device=DEV) for n, v in x["par"].items()}
    call = lambda: q4.verify_drafts(x["logits"], x["drafts"], x["starts"], x["u"], x["u_draw"],  # noqa: E731
                                    draft_logits=x["draft_logits"], ws=ws, tokens_out=outs[0], prob_out=outs[1],
                                    count_out=outs[2], **par)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for turn in (1, 0, 1):
        x["starts"].copy_(starts[turn])
        want = verify(x)
        for o in outs:
            o.fill_(77)
        ws.fill_(turn)
        graph.replay()
        torch.cuda.synchronize()
        used = int(starts[turn][-1])
        assert all(torch.equal(o[:used], w[:used]) for o, w in zip(outs[:2], want)) and torch.equal(outs[2], want[2])
        assert (outs[0][used:] == 77).all() and (outs[1][used:] == 77).all()
        check_verify(x, want)


# ------------------------------------------------------ as they are used together


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_speculative_rollouts_end_to_end(cache):
    """Rollouts of one prompt: its keys are appended once, its full pages shared and the last one copied; each step
    appends a token and its drafts, attends, forms the logits of every row by the q4_0 head, and keeps what
    verify_drafts keeps. Every step against the parts' oracles; the kept tokens' keys stay for the next."""
    g = generator(21)
    n_q, n_kv, D, page, prompt, members, drafts, vocab = 8, 2, 128, 16, 1501, 24, 3, 4096
    k_dim = n_q * D
    embed = torch.randn(vocab, (n_q + 2 * n_kv) * D, generator=g, device=DEV) * 0.6
    rng = np.random.default_rng(3)
    codes = torch.from_numpy(rng.integers(-8, 8, (vocab, k_dim)).astype(np.int8)).to(DEV)
    scales = torch.from_numpy((rng.random((vocab, k_dim // 32)) * 0.02).astype(np.float16).view(np.int16)).to(DEV)
    head = q4.q4_pack(codes, scales)
    freqs = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device=DEV) / (D // 2))
    kind = torch.bfloat16 if cache == "bf16" else E4M3
    kw = {} if cache == "bf16" else {n + "_scale": torch.full((n_kv,), 0.02, device=DEV) for n in "kv"}
    full, each = prompt // page, 4
    pages = full + members * each
    caches = [torch.zeros(pages, n_kv, page, D, device=DEV).to(kind) for _ in "kv"]
    table = torch.full((members, full + each), -1, dtype=torch.int32, device=DEV)
    table[:, :full] = torch.arange(full, dtype=torch.int32, device=DEV)
    table[:, full:] = torch.arange(full, pages, dtype=torch.int32, device=DEV).view(members, each)

    def append(tokens, seq, positions):
        x = embed[tokens.long()]
        slots = (table[seq, positions // page].long() * page + positions % page).int()
        q, k, v = x.split([n_q * D, n_kv * D, n_kv * D], 1)
        return q4.kv_append_rope(q, k, v, positions.int(), slots, *caches, freqs, q_norm=torch.ones(D, device=DEV),
                                 k_norm=torch.ones(D, device=DEV), v_norm=True, **kw)

    at = torch.arange(prompt, device=DEV)
    first = torch.zeros(prompt, dtype=torch.long, device=DEV)
    append(torch.randint(0, vocab, (prompt,), generator=g, device=DEV), first, at)
    for c in caches:  # the page that the prompt ends in, to each one's own
        raw = c.view(torch.uint8) if cache == "e4m3" else c.view(torch.int16)
        raw[table[1:, full].long()] = raw[table[0, full].long()].expand(members - 1, -1, -1, -1)
    lens = torch.full((members,), prompt, dtype=torch.int64, device=DEV)
    last = torch.randint(0, vocab, (members,), generator=g, device=DEV)
    group = ints([0, members])
    T = members * (drafts + 1)
    starts = torch.arange(0, T + 1, drafts + 1, dtype=torch.int32, device=DEV)
    seq = torch.arange(members, device=DEV).repeat_interleave(drafts + 1)
    step_at = torch.arange(drafts + 1, device=DEV).repeat(members)
    for step in range(3):
        fed = torch.randint(0, vocab, (members, drafts + 1), generator=g, device=DEV)
        fed[:, 0] = last
        q = append(fed.view(-1), seq, lens[seq] + step_at)
        kv_lens = (lens + drafts + 1).int()
        bound, most = int(kv_lens.max()), LOOSE
        wide = torch.nn.functional.pad(table, (0, most // page + 1 - table.shape[1]), value=-1)
        args = (q, *caches, wide.contiguous(), starts, kv_lens)
        out = q4.paged_attention_shared(*args, group, ints([prompt]), drafts + 1, most, most, scale=D ** -0.5, **kw)
        alone = q4.paged_attention(*args, drafts + 1, bound, scale=D ** -0.5, **kw)
        f = {c: f64(x) * (0.02 if cache == "e4m3" else 1.0) for c, x in zip("kv", caches)}
        host = {c: [] for c in "kv"}
        for b in range(members):
            mine = table[b].cpu().numpy()[:-(-int(kv_lens[b]) // page)]
            for c in "kv":
                host[c].append(f[c][mine].transpose(0, 2, 1, 3).reshape(-1, n_kv, D)[:int(kv_lens[b])])
        want, mag, span = so.attention(f64(q), host["k"], host["v"], [drafts + 1] * members, kv_lens.tolist(), D ** -0.5, 0)
        tol = so.attention_tolerance(want, mag, span, bound, D)
        assert (np.abs(f64(out) - want) <= tol).all() and (np.abs(f64(alone) - want) <= tol).all()
        logits = torch.cat([q4.q4_gemv_multi(head, vocab, k_dim, x.contiguous()) for x in out.view(T, k_dim).split(8)])
        drafter = logits + 0.3 * torch.randn(T, vocab, generator=g, device=DEV)
        asked = dict(logits=logits, draft_logits=drafter, drafts=torch.zeros(T, dtype=torch.int32, device=DEV), starts=starts,
                     u=torch.rand(T, generator=g, device=DEV), u_draw=torch.rand(members, generator=g, device=DEV),
                     par=dict(top_k=np.full(members, 64), top_p=np.full(members, 0.95), temperature=np.full(members, 0.8)))
        # (the drafts that a drafter would have drawn one by one)
        draw = q4.sample_logits(drafter, torch.rand(T, generator=g, device=DEV),
                                temperature=torch.full((T,), 0.8, device=DEV), top_k=torch.full((T,), 64, dtype=torch.int32,
                                device=DEV), top_p=torch.full((T,), 0.95, device=DEV))[0]
        asked["drafts"].copy_(draw)
        tokens, prob, count = verify(asked)
        check_verify(asked, (tokens, prob, count))
        assert int(count.max()) > 1 and int(count.min()) < drafts + 1
        last = tokens.view(members, -1).gather(1, (count.long() - 1)[:, None])[:, 0].long()
        lens = lens + 1  # the token fed; the drafts' keys are written over by the next step
