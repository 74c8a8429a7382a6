"""The paged-attention operators up to the launch: the library's refusals (with no rows, so
that nothing could be launched), and the tensor functions on CPU tensors with the library
calls recorded."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_scaled_fp4_sigmoid_gb300 as fm  # noqa: E402
from block_scaled_fp4_sigmoid_gb300 import build  # noqa: E402

BUF = (ctypes.c_uint8 * 65536)()
AT = (ctypes.addressof(BUF) + 255) // 256 * 256
INVALID, SHAPE, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def pa():
    build.build_library()
    from block_scaled_fp4_sigmoid_gb300 import paged_attention
    return paged_attention


def cache(**kw):
    d = dict(k=AT, v=AT, k_scale=None, v_scale=None, k_page=4096, k_head=2048, k_token=128, v_page=4096, v_head=2048,
             v_token=128, pages=4, page_size=16, kv_heads=2, head_dim=128, fp8=0)
    d.update(kw)
    return fm.KvCache(**d)


def batch(**kw):
    d = dict(starts=None, lens=AT, table=AT, table_ld=8, rows=0, seqs=0, table_cols=8)
    d.update(kw)
    return fm.KvBatch(**d)


def attn(**kw):
    d = dict(q=AT, q_ld=1024, out=AT, codes=None, code_scales=None, q_heads=8, window=0, sinks=0, scale=0.1)
    d.update(kw)
    return fm.Attn(**d)


BAD_CACHE = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=AT + 8), INVALID), (dict(fp8=2), INVALID),
             (dict(fp8=1), INVALID), (dict(k_scale=AT, v_scale=AT), INVALID), (dict(fp8=1, k_scale=AT, v_scale=AT + 2), INVALID),
             (dict(head_dim=96), SHAPE), (dict(head_dim=256), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
             (dict(page_size=256), SHAPE), (dict(pages=0), SHAPE), (dict(pages=(1 << 27) + 1), SHAPE), (dict(kv_heads=0), SHAPE),
             (dict(kv_heads=1025), SHAPE), (dict(k_token=132), INVALID), (dict(v_head=0), INVALID), (dict(k_page=-4096), INVALID),
             (dict(v_page=1 << 38), INVALID)]
BAD_BATCH = [(dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(rows=-1), SHAPE), (dict(rows=(1 << 20) + 1), SHAPE),
             (dict(seqs=-1), SHAPE), (dict(seqs=(1 << 16) + 1), SHAPE), (dict(table_cols=-1), SHAPE),
             (dict(table_cols=(1 << 20) + 1, table_ld=1 << 27), SHAPE), (dict(table_ld=7), INVALID), (dict(lens=AT + 2), INVALID),
             (dict(table=AT + 1), INVALID), (dict(starts=AT + 2), INVALID)]
BAD_ATTN = [(dict(q=None), INVALID), (dict(out=None), INVALID), (dict(codes=AT), INVALID), (dict(out=None, codes=AT), INVALID),
            (dict(out=None, code_scales=AT), INVALID), (dict(q_heads=0), SHAPE), (dict(q_heads=7), SHAPE),
            (dict(q_heads=130, q_ld=1 << 15), SHAPE), (dict(q_ld=1016), INVALID), (dict(q_ld=1028), INVALID), (dict(q=AT + 8), INVALID),
            (dict(out=AT + 8), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=-0.5), INVALID),
            (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID)]


def decode(c=None, b=None, a=None, ws=AT, ws_bytes=1 << 40):
    L = fm.lib()
    ref = lambda x, make: ctypes.byref(make(**(x or {})))  # noqa: E731
    return L.fp4moe_attn_decode(ref(c, cache), ref(b, batch), ref(a, attn), ws, ws_bytes, None)


def prompt(c=None, b=None, a=None, ws=AT, ws_bytes=1 << 40):
    L = fm.lib()
    ref = lambda x, make: ctypes.byref(make(**(x or {})))  # noqa: E731
    return L.fp4moe_attn_prompt(ref(c, cache), ref({"starts": AT, **(b or {})}, batch), ref(a, attn), ws, ws_bytes, None)


def append(c=None, b=None, **kw):
    d = dict(q=AT, q_ld=1024, q_heads=8, k=AT, k_ld=256, v=AT, v_ld=256, rope=AT, rope_dim=128, pairs=0, q_out=AT, q_out_ld=1024)
    d.update(kw)
    return fm.lib().fp4moe_kv_append(ctypes.byref(cache(**(c or {}))), ctypes.byref(batch(**(b or {}))),
                                     ctypes.byref(fm.Append(**d)), None)


@pytest.mark.parametrize("call", [decode, prompt, append])
def test_no_rows_are_no_work(pa, call):
    assert call() == 0
    assert call(c=dict(pages=1, k_page=0, v_page=0)) == 0  # a dimension of one has no stride
    assert call(c=dict(fp8=1, k_scale=AT, v_scale=AT)) == 0
    if call is not append:
        assert call(a=dict(out=None, codes=AT, code_scales=AT)) == 0
        assert call(a=dict(q_heads=128, q_ld=1 << 14)) == 0  # 64 query heads a key-value head


@pytest.mark.parametrize("call", [decode, prompt, append])
@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_caches_that_are_refused(pa, call, bad, status):
    assert call(c=bad) == status


@pytest.mark.parametrize("call", [decode, prompt, append])
@pytest.mark.parametrize("bad,status", BAD_BATCH)
def test_batches_that_are_refused(pa, call, bad, status):
    assert call(b=bad) == status


@pytest.mark.parametrize("call", [decode, prompt])
@pytest.mark.parametrize("bad,status", BAD_ATTN)
def test_queries_and_outputs_that_are_refused(pa, call, bad, status):
    assert call(a=bad) == status


def test_codes_of_heads_that_share_a_block(pa):
    """Heads of 64: a key-value head's queries make whole blocks of 128 columns, or no codes."""
    small = dict(head_dim=64, k_token=64, v_token=64, k_head=1024, v_head=1024)
    codes = dict(out=None, codes=AT, code_scales=AT)
    for call in (decode, prompt):
        assert call(c=small, a=dict(q_heads=8, q_ld=512, **codes)) == 0
        assert call(c=small, a=dict(q_heads=6, q_ld=512, **codes)) == SHAPE
        assert call(c=small, a=dict(q_heads=6, q_ld=512)) == 0


def test_workspaces(pa):
    long = dict(table_cols=1 << 16, table_ld=1 << 16)
    for call, size in ((decode, fm.lib().fp4moe_attn_decode_workspace_size), (prompt, fm.lib().fp4moe_attn_prompt_workspace_size)):
        n = size(ctypes.byref(cache()), 8)
        assert n > 0 and size(ctypes.byref(cache()), 7) == 0 and size(ctypes.byref(cache(head_dim=32)), 8) == 0
        assert call(ws_bytes=n) == 0 and call(ws_bytes=n - 1) == WORKSPACE and call(ws=AT + 8) == INVALID
        assert call(ws=None, ws_bytes=0) == 0  # a short table: nothing is left there
        assert call(ws=None, ws_bytes=16) == WORKSPACE
        assert call(b=long, ws=None, ws_bytes=0) == WORKSPACE
        assert call(b=long, ws_bytes=n) == 0
    assert decode(b=dict(starts=AT)) == INVALID
    assert fm.lib().fp4moe_attn_prompt(ctypes.byref(cache()), ctypes.byref(batch()), ctypes.byref(attn()), AT, 1 << 40, None) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(q_heads=0), SHAPE), (dict(q=None, q_out=None), SHAPE), (dict(rope_dim=0), SHAPE), (dict(rope_dim=24), SHAPE),
    (dict(rope_dim=144), SHAPE), (dict(rope=None), SHAPE), (dict(pairs=2), INVALID), (dict(k_ld=248), INVALID),
    (dict(v_ld=260), INVALID), (dict(q_ld=1016), INVALID), (dict(q_out_ld=1000), INVALID), (dict(k=AT + 8), INVALID),
    (dict(rope=AT + 4), INVALID), (dict(q_out=AT + 2), INVALID)])
def test_appends_that_are_refused(pa, bad, status):
    assert append(**bad) == status


def test_appends_without_rotation_or_queries(pa):
    assert append(rope=None, rope_dim=0) == 0
    assert append(q=None, q_out=None, q_heads=0, q_ld=0, q_out_ld=0) == 0


# ------------------------------------------------------------------ tensor functions
@pytest.fixture
def calls(pa, monkeypatch):
    """What would have been launched: name, arguments and the current device (0; the CPU tensors' index, -1,
    stands for another GPU)."""
    current, seen = [0], []

    class device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.before, current[0] = current[0], self.d

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(pa, "_device", lambda t: t.get_device())
    monkeypatch.setattr(pa, "_stream", lambda d: 1000 + d)
    monkeypatch.setattr(pa, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("_append", "_decode", "_prompt"):
        monkeypatch.setattr(pa, name, lambda *a, _n=name: (seen.append((_n, a, current[0])), True)[1])
    return seen


def tensors(B=3, T=None, hq=8, hkv=2, D=64, page=16, pages=9, cols=4, fp8=False):
    T = B if T is None else T
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    c = lambda: torch.zeros((pages, hkv, page, D), dtype=torch.uint8 if fp8 else torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return {"q": z(T, hq, D), "k": z(T, hkv, D), "v": z(T, hkv, D), "k_cache": c(), "v_cache": c(), "lens": i(B), "table": i(B, cols),
            "starts": i(B + 1), "rope": torch.zeros(cols * page, D)}


def run(pa, what, t, **kw):
    t = {**t, **{k: kw.pop(k) for k in list(kw) if k in t and (what, k) != ("append", "starts")}}
    if what == "append":
        return pa.append_kv(t["q"], t["k"], t["v"], t["rope"], t["k_cache"], t["v_cache"], t["lens"], t["table"], **kw)
    if what == "decode":
        return pa.decode_attention(t["q"], t["k_cache"], t["v_cache"], t["lens"], t["table"], **kw)
    return pa.prompt_attention(t["q"], t["k_cache"], t["v_cache"], t["starts"], t["lens"], t["table"], **kw)


def test_the_bytes_are_the_structs(pa, calls):
    assert len(pa._pack_cache(*[0] * 15)) == ctypes.sizeof(fm.KvCache)
    assert len(pa._pack_batch(*[0] * 7)) == ctypes.sizeof(fm.KvBatch)
    assert len(pa._pack_attn(*[0] * 9)) == ctypes.sizeof(fm.Attn)
    assert len(pa._pack_append(*[0] * 12)) == ctypes.sizeof(fm.Append)
    t = tensors()
    stored = torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16)  # token-major storage
    out = run(pa, "decode", t, v_cache=stored.permute(0, 2, 1, 3), window=7, sinks=2, scale=0.25)
    (_, a, device), = calls
    assert device == -1 and a[-1] == 999
    c, b, x = (s.from_buffer_copy(v) for s, v in zip((fm.KvCache, fm.KvBatch, fm.Attn), a))
    assert (c.k, c.v, c.k_scale, c.pages, c.page_size, c.kv_heads, c.head_dim, c.fp8) == (
        t["k_cache"].data_ptr(), stored.data_ptr(), None, 9, 16, 2, 64, 0)
    assert (c.k_page, c.k_head, c.k_token) == (2048, 1024, 64) and (c.v_page, c.v_head, c.v_token) == (2048, 64, 128)
    assert (b.starts, b.lens, b.table, b.table_ld, b.rows, b.seqs, b.table_cols) == (
        None, t["lens"].data_ptr(), t["table"].data_ptr(), 4, 3, 3, 4)
    assert (x.q, x.q_ld, x.out, x.codes, x.q_heads, x.window, x.sinks, x.scale) == (
        t["q"].data_ptr(), 512, out.data_ptr(), None, 8, 7, 2, 0.25)


def test_strides_of_dimensions_of_one(pa, calls):
    t = tensors(pages=1, hkv=1)
    odd = torch.zeros((16, 67), dtype=torch.bfloat16)[:, :64].as_strided((1, 1, 16, 64), (5, 3, 64, 1))
    run(pa, "decode", t, k_cache=odd, v_cache=odd)
    c = fm.KvCache.from_buffer_copy(calls[0][1][0])
    assert (c.k_page, c.k_head, c.k_token) == (0, 0, 64)


def test_queries_in_a_products_rows(pa, calls):
    t = tensors(T=5, B=2)
    qkv = torch.zeros((5, 12 * 64), dtype=torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, 64)) for x in qkv.split((512, 128, 128), 1))
    got = run(pa, "append", t, q=q, k=k, v=v, starts=t["starts"], q_out=q)
    a = fm.Append.from_buffer_copy(calls[0][1][2])
    assert got is q and (a.q, a.k, a.v, a.rope, a.q_out) == tuple(x.data_ptr() for x in (q, k, v, t["rope"], q))
    assert (a.q_ld, a.k_ld, a.v_ld, a.q_out_ld, a.q_heads, a.rope_dim, a.pairs) == (768, 768, 768, 768, 8, 64, 0)
    run(pa, "prompt", t, q=q)
    assert fm.Attn.from_buffer_copy(calls[1][1][2]).q_ld == 768


def test_no_rows_launch_nothing(pa, calls):
    for what in ("append", "decode", "prompt"):
        run(pa, what, tensors(B=0))
    run(pa, "prompt", tensors(B=0, T=4))
    assert not calls


BAD = {
    "another type of q": dict(q=torch.zeros(3, 8, 64)),
    "q of other heads": dict(q=torch.zeros((3, 8, 128), dtype=torch.bfloat16)),
    "heads apart": dict(q=torch.zeros((3, 16, 64), dtype=torch.bfloat16)[:, ::2]),
    "a cache of three dimensions": dict(k_cache=torch.zeros((9, 16, 64), dtype=torch.bfloat16)),
    "caches of two shapes": dict(v_cache=torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16)),
    "caches of two types": dict(v_cache=torch.zeros((9, 2, 16, 64), dtype=torch.uint8)),
    "a cache in fp32": dict(k_cache=torch.zeros(9, 2, 16, 64), v_cache=torch.zeros(9, 2, 16, 64)),
    "values apart": dict(k_cache=torch.zeros((9, 2, 16, 128), dtype=torch.bfloat16)[..., ::2]),
    "codes without scales": dict(k_cache=torch.zeros((9, 2, 16, 64), dtype=torch.uint8), v_cache=torch.zeros((9, 2, 16, 64), dtype=torch.uint8)),
    "lengths in int64": dict(lens=torch.zeros(3, dtype=torch.int64)),
    "lengths of other sequences": dict(lens=torch.zeros(4, dtype=torch.int32)),
    "a table in int64": dict(table=torch.zeros((3, 4), dtype=torch.int64)),
    "a table by columns": dict(table=torch.zeros((4, 3), dtype=torch.int32).T),
    "scales of a bf16 cache": dict(k_scale=torch.zeros(2), v_scale=torch.zeros(2)),
}


@pytest.mark.parametrize("what", ["append", "decode", "prompt"])
@pytest.mark.parametrize("kind", BAD)
def test_tensors_that_are_refused(pa, calls, what, kind):
    with pytest.raises(ValueError):
        run(pa, what, tensors(), **BAD[kind])
    assert not calls


@pytest.mark.parametrize("what", ["decode", "prompt"])
@pytest.mark.parametrize("bad", [dict(window=-1), dict(sinks=-1), dict(window=1 << 31), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(out=torch.zeros(3, 8, 64)), dict(out=torch.zeros((3, 512), dtype=torch.bfloat16)),
                                 dict(fp8=True, out=torch.zeros((3, 8, 64), dtype=torch.bfloat16)),
                                 dict(codes=torch.zeros((3, 512), dtype=torch.uint8)), dict(scales=torch.zeros(3, 4)),
                                 dict(fp8=True, scales=torch.zeros(3, 3)), dict(ws=torch.zeros(64)),
                                 dict(ws=torch.zeros((64, 2), dtype=torch.uint8)[:, 0])])
def test_options_that_are_refused(pa, calls, what, bad):
    with pytest.raises(ValueError):
        run(pa, what, tensors(), **bad)
    assert not calls


def test_more_that_is_refused(pa, calls):
    t = tensors()
    for bad in (dict(rope=t["rope"][:-1]), dict(rope=t["rope"].double()), dict(rope=t["rope"][:, ::2]), dict(q=None, q_out=t["q"]),
                dict(k=t["k"][:2]), dict(v=t["v"][:, :1]), dict(q_out=torch.zeros(3, 8, 64)), dict(starts=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            run(pa, "append", t, **bad)
    with pytest.raises(ValueError, match="starts"):
        run(pa, "prompt", t, starts=None)
    with pytest.raises(ValueError, match="starts"):
        run(pa, "decode", tensors(B=3, T=4))
    assert not calls


def test_a_workspace_is_made_where_one_is_needed(pa, calls, monkeypatch):
    tried = []

    def needs(cache_, batch_, attn_, ws, ws_bytes, stream):
        tried.append((ws, ws_bytes))
        return ws is not None

    monkeypatch.setattr(pa, "_decode", needs)
    t = tensors()
    run(pa, "decode", t)
    n = pa.decode_workspace_size(t["k_cache"], 8)
    assert tried[0] == (None, 0) and tried[1][0] and tried[1][1] == n
    ws = torch.zeros(n + 5, dtype=torch.uint8)
    run(pa, "decode", t, ws=ws)
    assert tried[2] == (ws.data_ptr(), n + 5)

    def fails(*a):
        raise fm.Fp4MoeError(SHAPE, "here")

    monkeypatch.setattr(pa, "_prompt", fails)
    with pytest.raises(fm.Fp4MoeError, match="UNSUPPORTED"):
        run(pa, "prompt", t)


def test_a_sublayer_refuses_weights_of_other_heads(pa):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    args = lambda hq, hkv, D: (None, u8((hq + 2 * hkv) * D, 256), None, u8(256, hq * D), None, hq, hkv, D, None)  # noqa: E731
    pa.Fp8BlockAttention(*args(8, 2, 64))
    for bad in ((6, 2, 64), (5, 2, 128)):
        with pytest.raises(ValueError, match="blocks"):
            pa.Fp8BlockAttention(*args(*bad))
    a = list(args(8, 2, 64))
    a[1] = u8(11 * 64, 256)
    with pytest.raises(ValueError, match="wqkv"):
        pa.Fp8BlockAttention(*a)


def test_workspace_holds_what_a_call_of_any_size_leaves(pa):
    """One size for every batch of a cache: the sums of each CTA's runs (or parts)."""
    for D in (64, 128):
        c = cache(head_dim=D)
        assert fm.attn_decode_workspace_size(c, 8) >= 2 * 152 * 2 * 16 * (4 * D + 8)
        assert fm.attn_prompt_workspace_size(c, 8) >= 152 * 256 * (4 * D + 8)
    assert np.int64(fm.attn_decode_workspace_size(cache(), 128)) > 0


@pytest.mark.parametrize("call", [decode, prompt])
def test_scales_whose_softmax_in_base_2_has_none(pa, call):
    """scale * log2(e) is fp32: infinite from 2.36e38 on, where a score of 0 would be NaN."""
    assert call(a=dict(scale=2.3e38)) == 0
    assert call(a=dict(scale=2.4e38)) == INVALID
