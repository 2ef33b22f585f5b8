"""CPU checks of the rollout operators' C ABI and binding: the library exports
what include/q4dec_rollout.h declares, and refuses bad arguments on the host
before touching the GPU; and pins of their fp64 oracle."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int4_weight_only_block_amd as q4
from int4_weight_only_block_amd import build as q4build
from oracle import rollout_oracle as ro
from oracle import serve_oracle as so

HERE = os.path.dirname(os.path.abspath(__file__))
built = pytest.mark.skipif(not os.path.exists(q4.LIB_PATH), reason="libq4dec.so not built")

EXPECTED = {"paged_attention_shared", "paged_attention_shared_workspace_bytes", "verify_drafts",
            "verify_drafts_workspace_bytes"}
FAKE = 0x10000  # aligned, not NULL, never dereferenced
BIG = 1 << 40


@built
def test_rollout_header_and_exports():
    assert set(q4.header_functions(q4.ROLLOUT_HEADER_PATH)) == EXPECTED
    h = ctypes.CDLL(q4.LIB_PATH)
    for name in EXPECTED:
        assert hasattr(h, name), name


SHARED = dict(q=FAKE, n_tok=12, n_q=8, n_kv=2, head_dim=256, k_cache=FAKE, v_cache=FAKE, kv_type=0, n_pages=4000,
              page_size=64, k_scale=None, v_scale=None, page_table=FAKE, table_stride=1024, q_starts=FAKE, kv_lens=FAKE,
              n_seq=12, group_starts=FAKE, shared_lens=FAKE, n_groups=1, max_q_len=1, max_kv_len=65536,
              max_shared_len=60000, scale=1.0, ws=FAKE, ws_bytes=BIG, out=FAKE, err_flag=None, stream=None)
VERIFY = dict(logits=FAKE, n_rows=7, vocab=1000, row_stride=1000, cap=30.0, draft_logits=FAKE, draft_stride=1000,
              draft_cap=30.0, drafts=FAKE, starts=FAKE, n_seq=2, temperature=None, top_k=None, top_p=None, min_p=None, u=FAKE,
              u_draw=FAKE, ws=FAKE, ws_bytes=BIG, tokens_out=FAKE, prob_out=None, count_out=FAKE, err_flag=None, stream=None)

REFUSED = [
    ("paged_attention_shared", SHARED, [
        (dict(head_dim=80), q4.ERR_UNSUPPORTED, "head_dim"), (dict(n_kv=0), q4.ERR_SHAPE, "n_kv"),
        (dict(n_q=9), q4.ERR_SHAPE, "n_q"), (dict(n_q=130, n_kv=2), q4.ERR_UNSUPPORTED, "per key/value head"),
        (dict(n_tok=-1), q4.ERR_SHAPE, "n_tok"), (dict(n_tok=1 << 29), q4.ERR_SHAPE, "n_tok"),
        (dict(n_seq=-1), q4.ERR_SHAPE, "n_seq"), (dict(n_seq=65536), q4.ERR_SHAPE, "n_seq"),
        (dict(n_groups=-1), q4.ERR_SHAPE, "n_groups"), (dict(n_groups=65536), q4.ERR_SHAPE, "n_groups"),
        (dict(max_q_len=0), q4.ERR_SHAPE, "max_q_len"), (dict(scale=float("inf")), q4.ERR_SHAPE, "scale"),
        (dict(max_shared_len=-1), q4.ERR_SHAPE, "max_shared_len"),
        (dict(max_shared_len=65537), q4.ERR_SHAPE, "max_shared_len"),
        (dict(q=None), q4.ERR_NULL, "q is"), (dict(out=None), q4.ERR_NULL, "out"),
        (dict(page_table=None), q4.ERR_NULL, "page_table"), (dict(q_starts=None), q4.ERR_NULL, "q_starts"),
        (dict(kv_lens=None), q4.ERR_NULL, "kv_lens"), (dict(k_cache=None), q4.ERR_NULL, "k_cache"),
        (dict(group_starts=None), q4.ERR_NULL, "group_starts"), (dict(shared_lens=None), q4.ERR_NULL, "shared_lens"),
        (dict(kv_type=7), q4.ERR_SHAPE, "kv_type"), (dict(page_size=100), q4.ERR_SHAPE, "page_size"),
        (dict(table_stride=0), q4.ERR_SHAPE, "table_stride"), (dict(max_kv_len=65537), q4.ERR_SHAPE, "max_kv_len"),
        (dict(max_kv_len=-1), q4.ERR_SHAPE, "max_kv_len"), (dict(q=FAKE + 8), q4.ERR_ALIGN, "q"),
        (dict(group_starts=FAKE + 2), q4.ERR_ALIGN, "group_starts"),
        (dict(shared_lens=FAKE + 1), q4.ERR_ALIGN, "shared_lens"), (dict(k_scale=FAKE), q4.ERR_SHAPE, "k_scale"),
        (dict(ws=FAKE + 16), q4.ERR_ALIGN, "ws"),
        (dict(n_seq=65535, n_groups=100, n_tok=1 << 20, max_kv_len=1 << 30, max_shared_len=1 << 30, table_stride=1 << 30,
              n_pages=1 << 20, ws_bytes=1 << 60), q4.ERR_UNSUPPORTED, "2^31 pieces"),
    ]),
    ("verify_drafts", VERIFY, [
        (dict(n_rows=-1), q4.ERR_SHAPE, "n_rows"), (dict(n_rows=32768), q4.ERR_SHAPE, "n_rows"),
        (dict(n_seq=-1), q4.ERR_SHAPE, "n_seq"), (dict(n_seq=32768), q4.ERR_SHAPE, "n_seq"),
        (dict(vocab=0), q4.ERR_SHAPE, "vocab"), (dict(vocab=(1 << 20) + 1, row_stride=1 << 21), q4.ERR_SHAPE, "vocab"),
        (dict(row_stride=999), q4.ERR_SHAPE, "row_stride"), (dict(draft_stride=999), q4.ERR_SHAPE, "draft_stride"),
        (dict(logits=None), q4.ERR_NULL, "logits"), (dict(drafts=None), q4.ERR_NULL, "drafts"),
        (dict(starts=None), q4.ERR_NULL, "starts"), (dict(u=None), q4.ERR_NULL, "u is"),
        (dict(u_draw=None), q4.ERR_NULL, "u_draw"), (dict(tokens_out=None), q4.ERR_NULL, "tokens_out"),
        (dict(count_out=None), q4.ERR_NULL, "count_out"), (dict(top_k=FAKE + 1), q4.ERR_ALIGN, "aligned"),
        (dict(draft_logits=FAKE + 2), q4.ERR_ALIGN, "aligned"), (dict(prob_out=FAKE + 2), q4.ERR_ALIGN, "aligned"),
        (dict(err_flag=FAKE + 2), q4.ERR_ALIGN, "aligned"), (dict(ws=FAKE + 16), q4.ERR_ALIGN, "ws"),
    ]),
]


@built
@pytest.mark.parametrize("name,good,change,code,word", [(n, g, c, rc, w) for n, g, cases in REFUSED for c, rc, w in cases])
def test_refusals(name, good, change, code, word):
    rc = getattr(q4.lib(), name)(*{**good, **change}.values())
    msg = q4.q4dec_last_error()
    assert rc == code and word in msg and name in msg, (rc, msg)


@built
@pytest.mark.parametrize("change", [
    # 4096 sequences of 128 rows of 8 heads: 2^18 units of 16 rows by 16385 blocks, but 2^15 of 128 rows
    dict(n_tok=4096 * 8, n_q=128, n_kv=8, head_dim=128, n_seq=4096, max_q_len=8, max_kv_len=1 << 20, max_shared_len=1 << 18,
         table_stride=1 << 20),
    # 2048 groups of two: 6144 tiles of shared rows, by 375001 blocks, but 4096 of the sequences'
    dict(n_tok=4096, n_q=16, n_kv=1, head_dim=64, n_seq=4096, n_groups=2048, max_kv_len=24000000, max_shared_len=24000000,
         table_stride=1 << 20)])
def test_bounds_that_only_sharing_has_too_many_pieces_for(change):
    """paged_attention takes such a call, so the call that shares where it can leaves it all to it."""
    L = q4.lib()
    args = {**SHARED, **change, "ws_bytes": 0}
    sizes = [args[n] for n in ("n_seq", "n_q", "n_kv", "head_dim", "max_q_len", "max_kv_len")]
    need = q4.paged_attention_workspace_bytes(*sizes)
    assert need == q4.paged_attention_shared_workspace_bytes(
        args["n_tok"], args["n_seq"], args["n_groups"], *sizes[1:], args["max_shared_len"]) and need > 0
    assert L.paged_attention_shared(*args.values()) == q4.ERR_WORKSPACE, q4.q4dec_last_error()


@built
def test_empty_calls_do_nothing_and_need_no_pointers():
    L = q4.lib()
    none = dict.fromkeys(("q", "out", "ws"))
    assert L.paged_attention_shared(*{**SHARED, "n_tok": 0, **none}.values()) == q4.OK
    none.update(dict.fromkeys(("page_table", "kv_lens", "shared_lens")))
    assert L.paged_attention_shared(*{**SHARED, "n_seq": 0, "n_groups": 0, **none}.values()) == q4.OK
    none = dict.fromkeys(("logits", "draft_logits", "drafts", "u", "ws", "tokens_out"))
    assert L.verify_drafts(*{**VERIFY, "n_rows": 0, **none}.values()) == q4.OK
    assert L.verify_drafts(*{**VERIFY, "n_seq": 0, "u_draw": None, "count_out": None}.values()) == q4.OK


@built
def test_workspace_bounds():
    L = q4.lib()
    for n_tok, n_seq, n_groups, n_q, n_kv, d, mq, mk, ms in [
            (12, 12, 1, 8, 2, 256, 1, 65536, 60000), (40, 8, 2, 32, 8, 128, 5, 9000, 9000), (24, 24, 1, 8, 1, 512, 1, 60000, 50000),
            (6 * 512, 6, 1, 32, 8, 128, 512, 12000, 9000), (3, 3, 0, 8, 2, 256, 1, 70000, 0)]:
        need = q4.paged_attention_shared_workspace_bytes(n_tok, n_seq, n_groups, n_q, n_kv, d, mq, mk, ms)
        assert need > 0
        args = {**SHARED, "n_tok": n_tok, "n_seq": n_seq, "n_groups": n_groups, "n_q": n_q, "n_kv": n_kv, "head_dim": d,
                "max_q_len": mq, "max_kv_len": mk, "max_shared_len": ms, "table_stride": 4096, "ws_bytes": need - 1}
        assert L.paged_attention_shared(*args.values()) == q4.ERR_WORKSPACE
        assert "workspace" in q4.q4dec_last_error()
        args["ws"] = None
        assert L.paged_attention_shared(*args.values()) == q4.ERR_NULL
    for drafter in (0, 1):
        need = q4.verify_drafts_workspace_bytes(7, 2, 1000, drafter)
        args = {**VERIFY, "draft_logits": FAKE if drafter else None, "ws_bytes": need - 1}
        assert L.verify_drafts(*args.values()) == q4.ERR_WORKSPACE
        args["ws"] = None
        assert L.verify_drafts(*args.values()) == q4.ERR_NULL
    assert q4.paged_attention_shared_workspace_bytes(12, 12, 1, 8, 2, 80, 1, 100, 50) == 0
    assert q4.verify_drafts_workspace_bytes(32768, 2, 1000, True) == 0


def test_binding_rejects_what_does_not_fit():
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q4.paged_attention_shared(torch.zeros(2, 8, 64).bfloat16(), c, c, i.view(2, 1), torch.zeros(3, dtype=torch.int32), i, i,
                                  i[:1], 1, 16, 16)
    with pytest.raises(ValueError):
        q4.verify_drafts(torch.zeros(2, 8), i, i, torch.zeros(2), torch.zeros(1))
    with pytest.raises(TypeError):
        q4.verify_drafts(None, i, i, torch.zeros(2), torch.zeros(1))


@pytest.mark.skipif(not os.path.exists(q4build.ASAN_LIB_PATH), reason="libq4dec_asan.so not built")
@pytest.mark.skipif("Q4DEC_LIB" in os.environ, reason="already a child with another library")
def test_refusals_under_asan():
    env = dict(os.environ, LD_PRELOAD=q4build.asan_runtime(), Q4DEC_LIB=q4build.ASAN_LIB_PATH,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                          os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=900,
                         cwd=os.path.dirname(HERE))
    out = res.stdout[-3000:] + res.stderr[-3000:]
    assert res.returncode == 0 and "AddressSanitizer" not in res.stderr and " passed" in res.stdout, out


# ------------------------------------------------------------ oracle pins


def test_oracle_distribution_is_what_the_sampling_oracle_draws_from():
    rng = np.random.default_rng(3)
    z = rng.normal(size=60) * 4
    z[[3, 9]], z[7] = z[5], -np.inf
    for kw in (dict(), dict(top_k=7), dict(top_p=0.7), dict(top_k=20, top_p=0.9, min_p=0.05), dict(temperature=0.0),
               dict(temperature=2.5, min_p=0.2), dict(cap=0.0, top_k=2)):
        p, _ = ro.distribution(z, **kw)
        assert p.sum() == pytest.approx(1.0)
        edges = np.cumsum(p)
        for i in np.nonzero(p)[0]:
            got = so.sample(z, edges[i] - p[i] / 2, **kw)
            assert got[0] == i and got[1] == pytest.approx(p[i])
    assert not ro.distribution([np.nan, -np.inf])[0].any()


def test_oracle_check_hand_values():
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    rows, of = np.log([p, p]), np.log([q, q])

    def at(x, u, w, drafter=of):
        return ro.check(rows, drafter, [x, -1], [u, 0.0], w, cap=0.0, draft_cap=0.0)[:2]

    # token 2 stays with probability 0.2 / 0.6; tokens of which the target has more always do
    assert at(2, 0.33, 0.0)[0] == [2, 0] and at(2, 0.34, 0.0)[0] == [0]
    assert at(0, 0.99, 0.6)[0] == [0, 1] and at(1, 0.99, 0.9)[0] == [1, 2]
    # taken back: from (0.3, 0.1, 0) / 0.4
    assert [at(2, 0.9, w)[0] for w in (0.0, 0.74, 0.76, 0.99)] == [[0], [0], [1], [1]]
    assert at(2, 0.9, 0.76)[1] == [pytest.approx(0.3)]
    # without probabilities: stays with p; else from the others
    assert at(1, 0.29, 0.0, None)[0] == [1, 0] and at(1, 0.31, 0.0, None)[0] == [0]
    assert [at(1, 0.31, w, None)[0] for w in (0.71, 0.72)] == [[0], [2]]
    # out of range: does not stay, nothing is taken off
    assert at(3, 0.0, 0.4, None)[0] == [0] and at(-1, 0.0, 0.9, None)[0] == [2]


def test_oracle_check_leaves_the_target_distribution():
    """Over all drafts and many numbers the first token is distributed as p."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    rows, of = np.log([p, p]), np.log([q, q])
    seen = np.zeros(3)
    grid = (np.arange(40) + 0.5) / 40
    for x in range(3):
        for u in grid:
            for w in grid:
                seen[ro.check(rows, of, [x, -1], [u, 0.0], w, cap=0.0, draft_cap=0.0)[0][0]] += q[x] / 1600
    assert np.allclose(seen, p, atol=0.02)
