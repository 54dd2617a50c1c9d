"""Host-side checks of the rotary and paged-cache calls: the frequency table
against float64 and rational arithmetic, the oracle's rotation against
complex multiplication, the pool's layout, and every refusal that needs no
pool.  No call here touches a GPU."""
import ctypes
import math
from ctypes import byref, c_float, c_uint64

import numpy as np
import pytest

from oracle import positions as opos


@pytest.fixture(scope="module")
def kvq():
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if not os.path.exists(os.path.join(root, "bit_kv_cache_quant_gb300", "libkvq.so")):
        import __graft_entry__

        __graft_entry__.build()
    import bit_kv_cache_quant_gb300 as m

    return m


SCALINGS = [
    ("none", {}),
    ("linear", dict(factor=4.0)),
    ("ntk", dict(factor=4.0)),
    ("yarn", dict(factor=16.0, original_max_position=4096, beta_fast=32.0, beta_slow=1.0)),
    ("llama3", dict(factor=8.0, original_max_position=8192, low_freq_factor=1.0, high_freq_factor=4.0)),
    ("factors", dict(factors="own")),
]


def _config(kvq, rot, base, scaling, attn_factor=0.0, **p):
    f = p.pop("factors", None)
    arr = None if f is None else (ctypes.c_double * (rot // 2))(*f)
    return kvq.kvq_rope_config(rot, kvq.ROPE_SCALINGS[scaling], base, p.get("factor", 1.0),
                               p.get("original_max_position", 0.0), p.get("beta_fast", 32.0), p.get("beta_slow", 1.0),
                               p.get("low_freq_factor", 1.0), p.get("high_freq_factor", 4.0), arr, attn_factor)


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("scaling,params", SCALINGS)
def test_table_matches_the_oracle(kvq, rot, base, scaling, params):
    p = dict(params)
    if p.get("factors") == "own":
        p["factors"] = [1.0 + 0.25 * i for i in range(rot // 2)]
    if scaling == "ntk" and rot < 4:
        with pytest.raises(kvq.KvqError):
            kvq.kvq_rope_table(_config(kvq, rot, base, scaling, **p))
        return
    got, mag = kvq.kvq_rope_table(_config(kvq, rot, base, scaling, **p))
    want, wmag = opos.frequencies(rot, base, scaling, **p)
    assert mag == np.float32(wmag)
    for g, f in zip(got, want):
        # the radians of both sides come from a handful of 64-bit operations (pow, log, divisions), each
        # within an ulp or two: 16 * 2^-53 relative; the entry itself adds half a unit of 2^-64 turn
        w = opos.table_entry(float(f))
        assert abs(g - w) <= 16 * 2.0 ** -53 * w + 1, (g, w)


def test_table_entry_is_turns_modulo_one():
    # a frequency of 2 pi (1 + 1/4) radians per position is a quarter turn
    assert abs(opos.table_entry(2 * math.pi * 1.25) - 2 ** 62) <= 2 ** 12
    assert opos.table_entry(0.0) == 0


def test_wrapped_product_is_the_angle_at_any_distance(kvq):
    # p * entry modulo 2^64, in half-turns, against rational arithmetic on the same frequency
    freqs, _ = kvq.kvq_rope_table(_config(kvq, 128, 10000.0, "none"))
    want, _ = opos.frequencies(128, 10000.0)
    for p in (0, 1, -1, 4095, 1000003, 2 ** 31 - 1, -2 ** 31):
        for f, w in zip(freqs, want):
            z = (p * f) % 2 ** 64
            half = (z - 2 ** 64 if z >= 2 ** 63 else z) / 2.0 ** 63
            ref = p * w / (2 * math.pi) % 1.0 * 2.0
            d = abs((half - ref + 1.0) % 2.0 - 1.0)
            # p times the entry's error (16 * 2^-53 of w / 2 pi, see above), plus float64's own in ref
            assert d <= 4 * abs(p) * w * 16 * 2.0 ** -53 + 2.0 ** -40, (p, w, d)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_complex_multiplication(interleaved):
    g = np.random.default_rng(0)
    x = g.standard_normal((5, 3, 16))
    f, mag = opos.frequencies(12, 100.0)
    pos = np.array([0, 1, -7, 1000, 123456])
    y = opos.rotate(x, pos, f, 1.5, interleaved)
    ia = np.arange(0, 12, 2) if interleaved else np.arange(6)
    ib = ia + 1 if interleaved else ia + 6
    z = (x[..., ia] + 1j * x[..., ib]) * 1.5 * np.exp(1j * pos[:, None, None] * f)
    np.testing.assert_allclose(y[..., ia] + 1j * y[..., ib], z, atol=1e-12)
    np.testing.assert_array_equal(y[..., 12:], x[..., 12:])
    # scores depend on the distance alone
    q, k = x[0:1], x[1:2]
    s = [float((opos.rotate(q, [a], f, 1.0, interleaved) * opos.rotate(k, [b], f, 1.0, interleaved)).sum())
         for a, b in ((10, 3), (1010, 1003))]
    assert abs(s[0] - s[1]) < 1e-10


def test_oracle_norm():
    x = np.array([[3.0, 4.0]])
    np.testing.assert_allclose(opos.head_norm(x, [1.0, 2.0], 0.0), [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]])
    np.testing.assert_array_equal(opos.head_norm(np.zeros((1, 4)), np.ones(4), 1e-6), np.zeros((1, 4)))


@pytest.mark.parametrize("kw", [
    dict(rot=3), dict(rot=0), dict(rot=258), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("inf")),
    dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_max_position=4096, beta_fast=1.0),
    dict(scaling="llama3", factor=2.0, original_max_position=4096, low_freq_factor=4.0, high_freq_factor=1.0),
    dict(scaling="factors"), dict(scaling="factors", factors=[1.0, 0.0]), dict(attn_factor=-1.0),
    dict(attn_factor=float("nan")),
])
def test_table_refusals(kvq, kw):
    kw = dict(kw)
    rot, base, scaling = kw.pop("rot", 4), kw.pop("base", 10000.0), kw.pop("scaling", "none")
    cfg = _config(kvq, rot, base, scaling, **kw)
    freqs, mag = (c_uint64 * 256)(), c_float()
    assert kvq.lib.kvq_rope_table(byref(cfg), freqs, byref(mag)) == 1
    assert kvq.lib.kvq_last_error()
    assert kvq.lib.kvq_rope_table(None, freqs, byref(mag)) == 1
    cfg.scaling = 17
    assert kvq.lib.kvq_rope_table(byref(cfg), freqs, byref(mag)) == 1


def _rows(kvq, heads=4, in_=0x1000, out=0x2000, weight=None):
    return kvq.kvq_rows(in_, out, 512, 128, 512, 128, heads, weight)


def test_rope_qk_refusals(kvq):
    rope = kvq.kvq_rope(0x3000, 64, 0, 1.0)
    f = kvq.lib.kvq_rope_qk
    q, k = _rows(kvq), _rows(kvq)

    def call(q=q, k=k, n=4, d=128, dt=1, pos=0x4000, rope=rope, eps=1e-6):
        return f(None if q is None else byref(q), None if k is None else byref(k), n, d, dt, pos,
                 None if rope is None else byref(rope), eps, None)

    assert call(n=0) == 0 and kvq.lib.kvq_last_launch_count() == 0
    assert call(n=0, q=_rows(kvq, in_=None, out=None), pos=None) == 0   # as empty tensors come
    assert call(n=-1) == 1
    assert call(d=96) == 2
    assert call(dt=3) == 1
    assert call(q=None, k=None) == 1
    assert call(q=_rows(kvq, heads=0), k=None) == 1
    assert call(q=_rows(kvq, heads=-1)) == 1
    assert call(q=_rows(kvq, in_=None)) == 1
    assert call(k=_rows(kvq, out=None)) == 1
    assert call(q=_rows(kvq, in_=0x1001)) == 1
    assert call(q=_rows(kvq, weight=0x1001)) == 1
    assert call(pos=None) == 1
    assert call(pos=0x4002) == 1
    assert call(eps=-1.0) == 1
    assert call(eps=float("nan")) == 1
    for bad in (kvq.kvq_rope(None, 64, 0, 1.0), kvq.kvq_rope(0x3004, 64, 0, 1.0), kvq.kvq_rope(0x3000, 63, 0, 1.0),
                kvq.kvq_rope(0x3000, 130, 0, 1.0), kvq.kvq_rope(0x3000, 0, 0, 1.0), kvq.kvq_rope(0x3000, 64, 2, 1.0),
                kvq.kvq_rope(0x3000, 64, 0, float("inf"))):
        assert call(rope=bad) == 1


def _paged(kvq, **kw):
    d = dict(n_kv_heads=8, head_dim=128, page_size=64, n_pages=10, kf="affine_token", kb=4, kg=64, vf="affine_token",
             vb=4, vg=32)
    d.update(kw)
    return kvq.kvq_paged_config(d["n_kv_heads"], d["head_dim"], d["page_size"], d["n_pages"],
                                kvq.FORMATS[d["kf"]], d["kb"], d["kg"], kvq.FORMATS[d["vf"]], d["vb"], d["vg"])


def test_paged_layout(kvq):
    lay = kvq.kvq_paged_layout_query(_paged(kvq))
    rows = 8 * 64 * 10
    assert (lay.k_row_bytes, lay.v_row_bytes, lay.k_n_groups, lay.v_n_groups) == (64, 64, 2, 4)
    offs = [lay.state, lay.k_codes, lay.k_meta, lay.v_codes, lay.v_meta]
    assert offs == [0, 256, 256 + rows * 64, 256 + rows * 72, 256 + rows * 136]
    assert lay.total_bytes == 256 + rows * (64 + 8 + 64 + 16)
    lay = kvq.kvq_paged_layout_query(_paged(kvq, kf="fp16", kb=16, kg=0, vf="fp16", vb=16, vg=0, page_size=16,
                                            n_kv_heads=1, n_pages=1))
    assert (lay.k_codes, lay.v_codes, lay.k_meta, lay.v_meta, lay.total_bytes) == (256, 256 + 4096, 0, 0, 256 + 8192)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), 2), (dict(head_dim=32), 2), (dict(page_size=48), 2), (dict(page_size=256), 2),
    (dict(n_pages=0), 1), (dict(n_kv_heads=0), 1), (dict(n_kv_heads=65536), 2), (dict(kb=2), 1), (dict(kg=16), 1), (dict(vg=48), 1),
    (dict(head_dim=64, kg=128), 1), (dict(kf="fp16", kb=4), 1), (dict(kf="q4_0", kb=4, kg=32), 2),
    (dict(kf="kivi_chan"), 2), (dict(kb=8), 2), (dict(kf="fp16", kb=16), 2),
    (dict(n_pages=2 ** 31 - 1, n_kv_heads=2 ** 31 - 1), 2), (dict(n_pages=2 ** 22), 2),
])
def test_paged_config_refusals(kvq, kw, code):
    lay = kvq.kvq_paged_layout()
    cfg = _paged(kvq, **kw)
    assert kvq.lib.kvq_paged_layout_query(byref(cfg), byref(lay)) == code
    assert kvq.lib.kvq_last_error()
    h = ctypes.c_void_p()
    assert kvq.lib.kvq_paged_init(byref(cfg), 0x10000, 1 << 40, None, byref(h)) == code and not h.value


def test_paged_init_refusals(kvq):
    cfg, h = _paged(kvq), ctypes.c_void_p()
    need = kvq.kvq_paged_layout_query(cfg).total_bytes
    f = kvq.lib.kvq_paged_init
    assert f(byref(cfg), None, need, None, byref(h)) == 1
    assert f(byref(cfg), 0x1010, need, None, byref(h)) == 1
    assert f(byref(cfg), 0x1000, need - 1, None, byref(h)) == 3
    assert f(byref(cfg), 0x1000, need, None, None) == 1
    assert f(None, 0x1000, need, None, byref(h)) == 1


def _batch(kvq, **kw):
    d = dict(n=4, cols=8, table=0x1000, lens=0x2000, npre=2, pre=0x3000, plen=0x4000)
    d.update(kw)
    return kvq.kvq_paged_batch(d["n"], d["cols"], d["table"], d["lens"], d["npre"], d["pre"], d["plen"])


BAD_BATCHES = [dict(n=0), dict(n=4097), dict(cols=-1), dict(table=None), dict(lens=None), dict(table=0x1002),
               dict(lens=0x2001)]


@pytest.mark.parametrize("kw", BAD_BATCHES + [dict(npre=-1), dict(pre=None), dict(plen=None), dict(pre=0x3001)])
def test_decode_refuses_bad_batches(kvq, kw):
    b = _batch(kvq, **kw)
    assert kvq.lib.kvq_paged_decode_attn(None, byref(b), 0x5000, 0x6000, 32, 1, 0.0, 0x7000, 1 << 30, None) == 1
    assert b"pool" not in kvq.lib.kvq_last_error()


def test_decode_refusals(kvq):
    f, b = kvq.lib.kvq_paged_decode_attn, _batch(kvq)

    def call(q=0x5000, out=0x6000, dt=1, scale=0.0, ws=0x7000, batch=b):
        return f(None, None if batch is None else byref(batch), q, out, 32, dt, scale, ws, 1 << 30, None)

    assert call() == 1 and b"null pool" in kvq.lib.kvq_last_error()
    for kw, code in ((dict(q=None), 1), (dict(out=None), 1), (dict(dt=0), 2), (dict(dt=5), 1), (dict(q=0x5008), 1),
                     (dict(out=0x6002), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
                     (dict(ws=None), 1), (dict(ws=0x7004), 1), (dict(batch=None), 1)):
        assert call(**kw) == code, kw
        assert b"null pool" not in kvq.lib.kvq_last_error(), kw
    assert kvq.lib.kvq_paged_workspace_bytes(None, 4, 32, 0) == 0


def test_append_refusals(kvq):
    f, b = kvq.lib.kvq_paged_append, _batch(kvq)
    rope = kvq.kvq_rope(0x3000, 64, 0, 1.0)
    ok = dict(batch=b, n=4, cu=None, q=_rows(kvq), k=_rows(kvq), v=_rows(kvq), dt=1, rope=rope, pos=None, eps=1e-6)

    def call(**kw):
        a = dict(ok, **kw)
        r = lambda x: None if x is None else byref(x)
        return f(None, r(a["batch"]), a["n"], a["cu"], r(a["q"]), r(a["k"]), r(a["v"]), a["dt"], r(a["rope"]),
                 a["pos"], a["eps"], None)

    assert call() == 1 and b"null pool" in kvq.lib.kvq_last_error()
    assert call(k=_rows(kvq, out=None), v=_rows(kvq, out=None), q=None, rope=None) == 1
    assert b"null pool" in kvq.lib.kvq_last_error()
    bad = [dict(batch=None), dict(n=-1), dict(n=5), dict(cu=0x1001), dict(q=_rows(kvq, out=None)), dict(k=None),
           dict(v=None), dict(k=_rows(kvq, heads=0)), dict(v=_rows(kvq, weight=0x9000)), dict(dt=7),
           dict(rope=kvq.kvq_rope(0x3000, 5, 0, 1.0)), dict(pos=0x1002), dict(eps=-1.0),
           dict(k=_rows(kvq, in_=0x1001))] + [dict(batch=_batch(kvq, **kw)) for kw in BAD_BATCHES]
    for kw in bad:
        assert call(**kw) == 1, kw
        assert b"null pool" not in kvq.lib.kvq_last_error(), kw


def test_binding_checks_shapes(kvq):
    # shapes and dtypes are refused before any call; raw pointers carry neither
    import torch

    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kvq.rope_qk(q, q, torch.zeros(4, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="T, heads, D"):
        kvq.rope_qk(None, None, None, None)
    r = lambda **kw: kvq._rows("q", **{**dict(x=q, out=None, weight=None, tokens=4, head_dim=128, dtype=q.dtype), **kw})
    rows = kvq.kvq_rows.from_buffer_copy(r())
    assert rows.heads == 8 and rows.in_tok_stride == 1024 and rows.in_ == q.data_ptr()
    assert len(kvq._BATCH.pack(1, 2, 3, 4, 5, 6, 7)) == ctypes.sizeof(kvq.kvq_paged_batch)
    b = kvq.kvq_paged_batch.from_buffer_copy(kvq._BATCH.pack(1, 2, 3, 4, 5, 6, 7))
    assert [getattr(b, f) for f, _ in b._fields_] == [1, 2, 3, 4, 5, 6, 7]
    for kw, msg in ((dict(tokens=5), "must be"), (dict(x=q.float()), "must be"), (dict(x=q[..., ::2], head_dim=64),
                    "contiguous"), (dict(out=q[:, :4]), "q_out"), (dict(out=q.float()), "q_out"),
                    (dict(out=q[:1].expand(4, 8, 128)), "expanded"), (dict(weight=q[0, 0, :64]), "q_norm"),
                    (dict(weight=torch.zeros(128)), "q_norm")):
        with pytest.raises(ValueError, match=msg):
            r(**kw)
    with pytest.raises(ValueError, match="int32"):
        kvq._int32("positions", torch.zeros(4, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="int32"):
        kvq._int32("positions", torch.zeros(5, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="scaling"):
        kvq.Rope(128, scaling="dynamic", device="cpu")
    with pytest.raises(ValueError, match="factors"):
        kvq.Rope(128, scaling="factors", factors=[1.0], device="cpu")
