"""CPU checks of the serving operators' C ABI and binding: the library exports
what include/q4dec_serve.h declares, and refuses bad arguments on the host
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
from oracle import serve_oracle as so

HERE = os.path.dirname(os.path.abspath(__file__))
built = pytest.mark.skipif(not os.path.exists(q4.LIB_PATH), reason="libq4dec.so not built")

EXPECTED = {"kv_append_rope", "paged_attention", "paged_attention_workspace_bytes", "sample_logits",
            "sample_logits_workspace_bytes"}
FAKE = 0x10000  # aligned, not NULL, never dereferenced
BIG = 1 << 40


@built
def test_serve_header_and_exports():
    assert set(q4.header_functions(q4.SERVE_HEADER_PATH)) == EXPECTED
    h = ctypes.CDLL(q4.LIB_PATH)
    for name in EXPECTED:
        assert hasattr(h, name), name


APPEND = dict(q=FAKE, q_stride=2048, k=FAKE, k_stride=512, v=FAKE, v_stride=512, n_tok=3, n_q=8, n_kv=2, head_dim=256,
              q_norm=None, k_norm=None, v_norm=0, eps=1e-6, freqs=FAKE, n_freqs=128, rot_dim=256, positions=FAKE,
              slots=FAKE, kv_type=0, k_scale=None, v_scale=None, k_cache=FAKE, v_cache=FAKE, n_pages=4, page_size=64,
              q_out=FAKE, err_flag=None, stream=None)
ATTN = dict(q=FAKE, n_tok=3, n_q=8, n_kv=2, head_dim=256, k_cache=FAKE, v_cache=FAKE, kv_type=0, n_pages=4,
            page_size=64, k_scale=None, v_scale=None, page_table=FAKE, table_stride=4, q_starts=FAKE, kv_lens=FAKE,
            n_seq=2, max_q_len=2, max_kv_len=200, scale=1.0, window=0, ws=FAKE, ws_bytes=BIG, out=FAKE,
            err_flag=None, stream=None)
SAMPLE = dict(logits=FAKE, n_rows=2, vocab=1000, row_stride=1000, cap=30.0, temperature=None, top_k=None, top_p=None,
              min_p=None, u=FAKE, ws=FAKE, ws_bytes=BIG, idx_out=FAKE, prob_out=None, stream=None)

REFUSED = [
    ("kv_append_rope", APPEND, [
        (dict(head_dim=96), q4.ERR_UNSUPPORTED, "head_dim"), (dict(n_tok=-1), q4.ERR_SHAPE, "n_tok"),
        (dict(n_q=-1), q4.ERR_SHAPE, "n_q"), (dict(n_q=0, n_kv=0), q4.ERR_SHAPE, "n_kv"),
        (dict(rot_dim=0), q4.ERR_SHAPE, "rot_dim"), (dict(rot_dim=7), q4.ERR_SHAPE, "rot_dim"),
        (dict(rot_dim=258), q4.ERR_SHAPE, "rot_dim"), (dict(n_freqs=129), q4.ERR_SHAPE, "n_freqs"),
        (dict(n_freqs=-1), q4.ERR_SHAPE, "n_freqs"), (dict(rot_dim=64), q4.ERR_SHAPE, "n_freqs"),
        (dict(eps=-1.0), q4.ERR_SHAPE, "eps"), (dict(eps=float("nan")), q4.ERR_SHAPE, "eps"),
        (dict(freqs=None), q4.ERR_NULL, "freqs"), (dict(positions=None), q4.ERR_NULL, "positions"),
        (dict(freqs=FAKE + 4), q4.ERR_ALIGN, "freqs"), (dict(slots=FAKE + 2), q4.ERR_ALIGN, "slots"),
        (dict(q_norm=FAKE + 4), q4.ERR_ALIGN, "q_norm"), (dict(k_norm=FAKE + 4), q4.ERR_ALIGN, "k_norm"),
        (dict(q=None), q4.ERR_NULL, "q is"), (dict(q_out=None), q4.ERR_NULL, "q_out"),
        (dict(q_stride=2047), q4.ERR_SHAPE, "q_stride"), (dict(q_stride=2050), q4.ERR_SHAPE, "q_stride"),
        (dict(q=FAKE + 4), q4.ERR_ALIGN, "q"), (dict(q_out=FAKE + 8), q4.ERR_ALIGN, "q_out"),
        (dict(k=None), q4.ERR_NULL, "k is"), (dict(v=None), q4.ERR_NULL, "v is"),
        (dict(slots=None), q4.ERR_NULL, "slots"), (dict(k_stride=508), q4.ERR_SHAPE, "k_stride"),
        (dict(v_stride=514), q4.ERR_SHAPE, "v_stride"), (dict(k=FAKE + 8), q4.ERR_ALIGN, "k"),
        (dict(k_cache=None), q4.ERR_NULL, "k_cache"), (dict(v_cache=None), q4.ERR_NULL, "v_cache"),
        (dict(kv_type=2), q4.ERR_SHAPE, "kv_type"), (dict(page_size=48), q4.ERR_SHAPE, "page_size"),
        (dict(page_size=8), q4.ERR_SHAPE, "page_size"), (dict(page_size=8192), q4.ERR_SHAPE, "page_size"),
        (dict(n_pages=0), q4.ERR_SHAPE, "n_pages"), (dict(n_pages=1 << 25), q4.ERR_SHAPE, "n_pages"),
        (dict(k_scale=FAKE), q4.ERR_SHAPE, "k_scale"), (dict(v_cache=FAKE + 8), q4.ERR_ALIGN, "v_cache"),
        (dict(kv_type=1, v_scale=FAKE + 2), q4.ERR_ALIGN, "v_scale"),
    ]),
    ("paged_attention", ATTN, [
        (dict(head_dim=80), q4.ERR_UNSUPPORTED, "head_dim"), (dict(n_kv=0), q4.ERR_SHAPE, "n_kv"),
        (dict(n_q=9), q4.ERR_SHAPE, "n_q"), (dict(n_q=130, n_kv=2), q4.ERR_UNSUPPORTED, "per key/value head"),
        (dict(n_tok=-1), q4.ERR_SHAPE, "n_tok"), (dict(n_tok=1 << 29), q4.ERR_SHAPE, "n_tok"),
        (dict(n_seq=-1), q4.ERR_SHAPE, "n_seq"), (dict(n_seq=65536), q4.ERR_SHAPE, "n_seq"),
        (dict(max_q_len=0), q4.ERR_SHAPE, "max_q_len"), (dict(window=-1), q4.ERR_SHAPE, "window"),
        (dict(scale=float("inf")), q4.ERR_SHAPE, "scale"), (dict(scale=float("nan")), q4.ERR_SHAPE, "scale"),
        (dict(q=None), q4.ERR_NULL, "q is"), (dict(out=None), q4.ERR_NULL, "out"),
        (dict(page_table=None), q4.ERR_NULL, "page_table"), (dict(q_starts=None), q4.ERR_NULL, "q_starts"),
        (dict(kv_lens=None), q4.ERR_NULL, "kv_lens"), (dict(k_cache=None), q4.ERR_NULL, "k_cache"),
        (dict(kv_type=-1), q4.ERR_SHAPE, "kv_type"), (dict(page_size=100), q4.ERR_SHAPE, "page_size"),
        (dict(table_stride=0), q4.ERR_SHAPE, "table_stride"),
        (dict(max_kv_len=(1 << 30) + 1, table_stride=1 << 30), q4.ERR_SHAPE, "max_kv_len"),
        (dict(n_seq=65535, n_tok=1 << 22, max_q_len=1 << 22, max_kv_len=1 << 30, table_stride=1 << 30, ws_bytes=1 << 60),
         q4.ERR_UNSUPPORTED, "2^31 pieces"), (dict(max_kv_len=257), q4.ERR_SHAPE, "max_kv_len"),
        (dict(max_kv_len=-1), q4.ERR_SHAPE, "max_kv_len"), (dict(q=FAKE + 8), q4.ERR_ALIGN, "q"),
        (dict(kv_lens=FAKE + 2), q4.ERR_ALIGN, "kv_lens"), (dict(k_scale=FAKE), q4.ERR_SHAPE, "k_scale"),
        (dict(ws=FAKE + 16), q4.ERR_ALIGN, "ws"),
    ]),
    ("sample_logits", SAMPLE, [
        (dict(n_rows=-1), q4.ERR_SHAPE, "n_rows"), (dict(n_rows=65536), q4.ERR_SHAPE, "n_rows"),
        (dict(vocab=0), q4.ERR_SHAPE, "vocab"), (dict(vocab=(1 << 20) + 1, row_stride=1 << 21), q4.ERR_SHAPE, "vocab"),
        (dict(row_stride=999), q4.ERR_SHAPE, "row_stride"), (dict(logits=None), q4.ERR_NULL, "logits"),
        (dict(u=None), q4.ERR_NULL, "u is"), (dict(idx_out=None), q4.ERR_NULL, "idx_out"),
        (dict(top_k=FAKE + 1), q4.ERR_ALIGN, "aligned"), (dict(prob_out=FAKE + 2), q4.ERR_ALIGN, "aligned"),
        (dict(ws=FAKE + 16), q4.ERR_ALIGN, "ws"),
    ]),
]


@built
@pytest.mark.parametrize("name,good,change,code,word", [(n, g, c, rc, w) for n, g, cases in REFUSED for c, rc, w in cases])
def test_refusals(name, good, change, code, word):
    rc = getattr(q4.lib(), name)(*{**good, **change}.values())
    msg = q4.q4dec_last_error()
    assert rc == code and word in msg and name in msg, (rc, msg)


@built
def test_empty_calls_do_nothing():
    L = q4.lib()
    assert L.kv_append_rope(*{**APPEND, "n_tok": 0}.values()) == q4.OK
    assert L.paged_attention(*{**ATTN, "n_tok": 0}.values()) == q4.OK
    assert L.paged_attention(*{**ATTN, "n_seq": 0}.values()) == q4.OK
    assert L.sample_logits(*{**SAMPLE, "n_rows": 0}.values()) == q4.OK


@built
def test_empty_calls_need_no_pointers():
    """An empty torch tensor's pointer is NULL."""
    L = q4.lib()
    none = dict.fromkeys(("q", "k", "v", "positions", "slots", "q_out"))
    assert L.kv_append_rope(*{**APPEND, "n_tok": 0, **none}.values()) == q4.OK, q4.q4dec_last_error()
    assert L.kv_append_rope(*{**APPEND, "n_tok": 0, "n_q": 0, **none}.values()) == q4.OK
    assert L.kv_append_rope(*{**APPEND, "n_tok": 0, "n_kv": 0, **none}.values()) == q4.OK
    none = dict.fromkeys(("q", "out", "ws"))
    assert L.paged_attention(*{**ATTN, "n_tok": 0, **none}.values()) == q4.OK
    assert L.paged_attention(*{**ATTN, "n_seq": 0, "page_table": None, "kv_lens": None, **none}.values()) == q4.OK
    none = dict.fromkeys(("logits", "u", "idx_out", "ws"))
    assert L.sample_logits(*{**SAMPLE, "n_rows": 0, **none}.values()) == q4.OK


@built
def test_workspace_bounds():
    L = q4.lib()
    for n_seq, n_q, n_kv, d, mq, mk, w in [(1, 8, 2, 256, 1, 131072, 0), (48, 8, 1, 512, 1, 16384, 0),
                                           (5, 32, 8, 128, 2048, 12288, 0), (6, 8, 2, 256, 512, 9000, 512)]:
        need = q4.paged_attention_workspace_bytes(n_seq, n_q, n_kv, d, mq, mk, w)
        if need:
            args = {**ATTN, "n_seq": n_seq, "n_q": n_q, "n_kv": n_kv, "head_dim": d, "max_q_len": mq,
                    "max_kv_len": mk, "window": w, "table_stride": 4096, "n_tok": n_seq * mq, "ws_bytes": need - 1}
            assert L.paged_attention(*args.values()) == q4.ERR_WORKSPACE
            assert "workspace" in q4.q4dec_last_error()
            args["ws"] = None
            assert L.paged_attention(*args.values()) == q4.ERR_NULL
    need = q4.sample_logits_workspace_bytes(5, 1000)
    if need:
        assert L.sample_logits(*{**SAMPLE, "n_rows": 5, "ws_bytes": need - 1}.values()) == q4.ERR_WORKSPACE
        assert L.sample_logits(*{**SAMPLE, "n_rows": 5, "ws": None}.values()) == q4.ERR_NULL


@built
@pytest.mark.parametrize("window", [4096, 1 << 31, 1 << 62, (1 << 63) - 560, (1 << 63) - 1])
def test_windows_as_wide_as_the_cache_are_none(window):
    L = q4.lib()
    for n_q, n_kv, d, mq in [(8, 2, 128, 512), (8, 1, 512, 1), (32, 8, 64, 4), (8, 2, 256, 64)]:
        bounds = (4, n_q, n_kv, d, mq, 4096)
        need = q4.paged_attention_workspace_bytes(*bounds, 0)
        assert need > 0 and q4.paged_attention_workspace_bytes(*bounds, window) == need
        args = {**ATTN, "n_seq": 4, "n_q": n_q, "n_kv": n_kv, "head_dim": d, "max_q_len": mq, "max_kv_len": 4096,
                "table_stride": 64, "n_tok": 4 * mq, "window": window, "ws_bytes": need - 1}
        assert L.paged_attention(*args.values()) == q4.ERR_WORKSPACE, q4.q4dec_last_error()


def test_binding_rejects_host_tensors():
    x = torch.zeros(2, 512)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q4.kv_append_rope(x, x[:, :128], x[:, :128], i, i, c, c, None)
    with pytest.raises(ValueError):
        q4.paged_attention(x.view(2, 8, 64).bfloat16(), c, c, i.view(2, 1), torch.zeros(3, dtype=torch.int32), i, 1, 16)
    with pytest.raises(ValueError):
        q4.sample_logits(x, torch.zeros(2))


def test_append_refuses_halves_of_a_call():
    """Values, slots or caches without keys would not be stored, and a head width can only be the cache's."""
    x, i = torch.zeros(2, 128), torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    for kw in (dict(v=x), dict(slots=i), dict(k_cache=c), dict(v_cache=c)):
        args = {**dict(q=x, k=None, v=None, positions=i, slots=None, k_cache=None, v_cache=None, freqs=None), **kw}
        with pytest.raises(ValueError, match="need k"):
            q4.kv_append_rope(**args, head_dim=64)
    with pytest.raises(ValueError, match="head_dim"):
        q4.kv_append_rope(x, x, x, i, i, c, c, None, head_dim=128)


def test_import_without_a_gpu_backend():
    """On a torch built without one the package imports, and a call fails when it is made."""
    code = ("import torch\nif hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import int4_weight_only_block_amd as q4\n"
            "try: q4.sample_logits(torch.zeros(2, 8), torch.zeros(2))\nexcept ValueError as e: print('refused', e)")
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    res = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(HERE))
    assert res.returncode == 0 and "refused" in res.stdout, res.stderr[-2000:]


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


def test_oracle_bf16_and_e4m3_agree_with_torch():
    x = torch.randn(4096, dtype=torch.float64) * torch.logspace(-6, 3, 4096, dtype=torch.float64)
    assert np.array_equal(so.bf16_round(x.float().numpy()), x.float().bfloat16().double().numpy())
    bits = torch.arange(256, dtype=torch.uint8)
    want = bits.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(so.e4m3_values(), want, equal_nan=True)


def test_oracle_rope_hand_values():
    # a quarter turn of the first pair, none of the second
    x = so.rope_row([[1.0, 2.0, 3.0, 4.0]], 1, [np.pi / 2], 2)
    assert np.allclose(x, [[-3.0, 2.0, 1.0, 4.0]], atol=1e-15)
    # a whole number of turns far out is no turn
    x = so.rope_row([[1.0, 2.0]], 100000, [2 * np.pi], 1)
    assert np.allclose(x, [[1.0, 2.0]], atol=1e-9)
    assert np.allclose(so.rms_row([[3.0, 4.0]], [2.0, 1.0], 0.0), [[3 * 2 / np.sqrt(12.5), 4 / np.sqrt(12.5)]])


def test_oracle_attention_hand_values():
    # two keys, equal scores: the mean; a window of one: the last value; nothing to see: zero
    q = np.zeros((1, 1, 2))
    k, v = np.ones((2, 1, 2)), np.array([[[1.0, 2.0]], [[3.0, 6.0]]])
    assert np.allclose(so.attention(q, [k], [v], [1], [2], 1.0, 0)[0], [[[2.0, 4.0]]])
    assert np.allclose(so.attention(q, [k], [v], [1], [2], 1.0, 1)[0], [[[3.0, 6.0]]])
    assert not so.attention(np.zeros((2, 1, 2)), [k[:1]], [v[:1]], [2], [1], 1.0, 0)[0][0].any()
    # scores ln 3 and 0: weights 3 : 1
    q, k = np.array([[[1.0, 0.0]]]), np.array([[[np.log(3.0), 0.0]], [[0.0, 0.0]]])
    assert np.allclose(so.attention(q, [k], [v], [1], [2], 1.0, 0)[0], [[[1.5, 3.0]]])


def test_oracle_sample_hand_values():
    z = np.log([1.0, 4.0, 2.0, 1.0])  # weights 1/8, 4/8, 2/8, 1/8 in index order
    at = lambda u, **kw: so.sample(z, u, cap=0.0, **kw)[:2]  # noqa: E731
    assert [at(u)[0] for u in (0.0, 0.12, 0.13, 0.6, 0.63, 0.8, 0.9)] == [0, 0, 1, 1, 2, 2, 3]
    assert at(0.6)[1] == pytest.approx(0.5)
    assert [at(u, top_k=2)[0] for u in (0.0, 0.66, 0.67)] == [1, 1, 2]
    assert at(0.9, top_k=3)[0] == 2 and at(0.0, top_k=3)[0] == 0  # of the equals 0 and 3 the lower index stays
    assert at(0.99, top_p=0.5)[0] == 1 and at(0.99, top_p=0.51)[0] == 2
    assert at(0.99, min_p=0.3)[0] == 2 and at(0.99, min_p=0.6)[0] == 1
    assert at(0.0, temperature=0.0) == (1, 1.0)
    assert so.sample([np.nan, -np.inf], 0.5)[0] == -1
    assert so.sample([np.nan, 1.0, -np.inf], 0.5)[:2] == (1, 1.0)
