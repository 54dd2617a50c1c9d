"""GPU parity of the page pool: what append stores, bit for bit against the
quantiser's definition where its input is exact, and decode attention over
prefix and own pages against float64."""
import numpy as np
import pytest
import torch

from kvq_helpers import _bits, host
from oracle import positions as opos
from oracle import quantize as oq
from paged_helpers import check_attention, gather, make_pool, reference, tables, values

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def kvq():
    import bit_kv_cache_quant_gb300 as m

    return m


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def rand(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def coded(x, bits, group):
    """Stored codes, metadata [.., groups, 2] (fp16) and values of rows x [T, H, D] by the oracle's rules."""
    u, s, z = oq.affine_token_quantize(x.transpose(1, 0, 2)[None], bits, group)[:3]
    u, s, z = (a[0].transpose(1, 0, 2) for a in (u, s, z))
    s16, z16 = oq.to_fp16(s), oq.to_fp16(z)
    hat = u.astype(np.float64) * np.repeat(s16.astype(np.float64), group, -1) + np.repeat(z16.astype(np.float64), group, -1)
    codes = oq.stored_int8(u).view(np.uint8) if bits == 8 else oq.pack_nibbles(u)
    return codes, np.stack((s16, z16), -1), hat


# ------------------------------------------------------------------- append --

@pytest.mark.parametrize("fmt,kg,vg", [("fp16", 0, 0), ("aff8", 128, 32), ("aff4", 64, 64), ("aff4", 32, 128),
                                       ("aff8", 64, 64)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("dtype", list(DT))
def test_append_unrotated_is_bit_exact(kvq, fmt, kg, vg, D, page, dtype):
    g = torch.Generator().manual_seed(D + page)
    H, new, held = 3, [5, 0, 1, 40], [0, 7, page - 1, page + 3]
    lens = [a + b for a, b in zip(new, held)]
    table, _, n_pages = tables(lens, 0, page, seed=1)
    c = make_pool(kvq, fmt, H, D, page, n_pages, kg, vg, seed=2)
    before = {n: c.plane(n).clone() for n in ("k_codes", "v_codes") + (("k_meta", "v_meta") if fmt != "fp16" else ())}
    T = sum(new) + 3   # three rows behind the last sequence
    k, v = rand((T, H, D), g, DT[dtype], 3.0), rand((T, H, D), g, DT[dtype])
    cu = i32([0] + list(np.cumsum(new)))
    ko, vo = (torch.full((T, H, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    c.append(k, v, dev(table), i32(lens), cu_tokens=cu, k_out=ko, v_out=vo)
    assert c.status() == 0 and c.launches == 1
    where = [(table[b, (held[b] + j) // page], (held[b] + j) % page) for b in range(4) for j in range(new[b])]
    ids, rows = (np.array(x) for x in zip(*where))
    n = len(where)
    for side, x, out, group in (("k", k, ko, min(kg, D)), ("v", v, vo, min(vg, D))):
        x64 = host(x)[:n]
        if fmt == "fp16":
            want = {side + "_codes": x64.astype(np.float16)}
            hat = x64.astype(np.float16).astype(np.float64)
        else:
            codes, meta, hat = coded(x64, 8 if fmt == "aff8" else 4, group)
            want = {side + "_codes": codes, side + "_meta": meta}
        for name, w in want.items():
            whole = before[name].cpu().numpy()
            whole[ids, :, rows] = w
            np.testing.assert_array_equal(_bits(c.plane(name).cpu().numpy()), _bits(whole), err_msg=name)
        # u * s + z in fp32 (one rounding of a value of at most 2 |z| + ...: 2^-23 of the range), then the type's
        rng = np.abs(hat).max()
        tol = torch.finfo(DT[dtype]).eps / 2 * np.abs(hat) + 2.0 ** -23 * rng
        assert np.all(np.abs(host(out)[:n] - hat) <= tol)
        assert torch.all(out[n:] == 7.0)


@pytest.mark.parametrize("fmt", ["fp16", "aff8", "aff4"])
@pytest.mark.parametrize("inter,rot,norm", [(False, 128, True), (True, 64, False), (False, 96, False)])
def test_append_rotated(kvq, fmt, inter, rot, norm):
    # keys leave as the rotation's bytes (rope_qk in fp32), coded by the append's rules: storing the
    # separately rotated fp32 keys gives the same pool
    g = torch.Generator().manual_seed(rot)
    H, Hq, D, page, prefix = 2, 6, 128, 32, 100
    new, held = [33, 1, 64], [31, 500, 0]
    lens = [a + b for a, b in zip(new, held)]
    table, _, n_pages = tables(lens, 0, page, seed=3)
    T = sum(new)
    q, k, v = rand((T, Hq, D), g, torch.float32), rand((T, H, D), g, torch.float32, 2.0), rand((T, H, D), g, torch.float32)
    wq, wk = (rand((D,), g, torch.float32), rand((D,), g, torch.float32)) if norm else (None, None)
    rope = kvq.Rope(rot, 10000.0, interleaved=inter)
    cu = i32([0] + list(np.cumsum(new)))
    pos = i32([prefix + held[b] + j for b in range(3) for j in range(new[b])])
    qr, kr = kvq.rope_qk(q, k, pos, rope, q_norm=wq, k_norm=wk)
    a, b = (make_pool(kvq, fmt, H, D, page, n_pages, seed=4) for _ in range(2))
    kw = dict(cu_tokens=cu, rope=rope, q_norm=wq, k_norm=wk)
    qo = a.append(k, v, dev(table), i32(lens), q=q, prefix_len=i32([prefix]), **kw)
    b.append(kr, v, dev(table), i32(lens), cu_tokens=cu)
    assert torch.equal(qo, qr) and torch.equal(a.buf, b.buf)
    # explicit positions in place of the derived ones
    p = make_pool(kvq, fmt, H, D, page, n_pages, seed=4)
    p.append(k, v, dev(table), i32(lens), positions=pos, **kw)
    assert torch.equal(a.buf, p.buf)


@pytest.mark.parametrize("B", [1, 3, 64, 300])
def test_append_one_token_each(kvq, B):
    # a decode step: no cu_tokens; rows of length 0 (padding) write nothing, here or in q_out
    g = torch.Generator().manual_seed(B)
    H, Hq, D, page = 2, 4, 64, 16
    lens = [0 if b % 5 == 4 else 1 + 7 * b % 50 for b in range(B)]
    table, _, n_pages = tables(lens, 0, page, seed=5)
    c = make_pool(kvq, "aff8", H, D, page, n_pages, seed=6)
    before = c.plane("k_codes").clone()
    q, k, v = rand((B, Hq, D), g, torch.bfloat16), rand((B, H, D), g, torch.bfloat16), rand((B, H, D), g, torch.bfloat16)
    qo = torch.full_like(q, 9.0)
    c.append(k, v, dev(table), i32(lens), q=q, q_out=qo)
    assert c.status() == 0
    codes, _, _ = coded(host(k), 8, 64)
    want = before.cpu().numpy()
    for b, n in enumerate(lens):
        if n:
            want[table[b, (n - 1) // page], :, (n - 1) % page] = codes[b]
    np.testing.assert_array_equal(c.plane("k_codes").cpu().numpy(), want)
    live = torch.tensor([n > 0 for n in lens]).cuda()
    assert torch.equal(qo[live], q[live]) and torch.all(qo[~live] == 9.0)


def test_append_many_sequences_find_their_tokens(kvq):
    # every length of a 4096-sequence batch, empty ones among them
    rng = np.random.default_rng(0)
    new = rng.integers(0, 4, 4096)
    page, H, D = 16, 1, 64
    table, _, n_pages = tables(list(new), 0, page, seed=7)
    c = make_pool(kvq, "fp16", H, D, page, n_pages, fill=False)
    T = int(new.sum())
    k = torch.arange(T, dtype=torch.float32).mul(0.25)[:, None, None].expand(T, H, D).contiguous().cuda()
    c.append(k, k, dev(table), i32(new.tolist()), cu_tokens=i32([0] + list(np.cumsum(new))))
    got = c.plane("k_codes").cpu().numpy()
    t = 0
    for b, n in enumerate(new):
        for j in range(n):
            assert (got[table[b, 0], 0, j] == np.float16(0.25 * t)).all()
            t += 1


def test_append_bad_pages(kvq):
    # ids outside the pool and lengths beyond the table: those rows are left out and the status says so
    H, D, page = 2, 64, 16
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        c = make_pool(kvq, "aff4", H, D, page, 6, seed=8)
        before = c.buf[256:].clone()
        k = torch.ones((1, H, D), dtype=torch.bfloat16, device="cuda")
        c.append(k, k, i32([[bad, 0]]), i32([5]))
        assert c.status() == kvq.DEV_BAD_PAGE and torch.equal(c.buf[256:], before)
        c.clear_status()
        c.append(k, k, i32([[1, 0]]), i32([33]))
        assert c.status() == kvq.DEV_BAD_PAGE and torch.equal(c.buf[256:], before)
        c.clear_status()
        c.append(k, k, i32([[1, 0]]), i32([32]))
        assert c.status() == 0 and not torch.equal(c.buf[256:], before)


def test_append_strided_projection(kvq):
    g = torch.Generator().manual_seed(11)
    B, Hq, H, D, page = 5, 4, 2, 128, 64
    qkv = rand((B, (Hq + 2 * H) * D + 1), g, torch.bfloat16)
    for off in (0, 1):
        q, k, v = (qkv[:, off + a * D:off + b * D].view(B, -1, D) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
        lens = [1, 64, 65, 2, 3]
        table, _, n = tables(lens, 0, page)
        a, b = (make_pool(kvq, "aff4", H, D, page, n, fill=False) for _ in range(2))
        rope = kvq.Rope(D)
        qa = a.append(k, v, dev(table), i32(lens), q=q, rope=rope)
        qb = b.append(k.contiguous(), v.contiguous(), dev(table), i32(lens), q=q.contiguous(), rope=rope)
        assert torch.equal(qa, qb) and torch.equal(a.buf, b.buf)


# ---------------------------------------------------------------- attention --

def run_attention(kvq, fmt, H, G, D, page, lens, prefix, dtype, kg=64, vg=64, seed=0, scale=0.0, qscale=1.0):
    table, pre, n_pages = tables(lens, prefix, page, seed=seed)
    c = make_pool(kvq, fmt, H, D, page, n_pages, kg, vg, seed=seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    q = rand((len(lens), H * G, D), g, DT[dtype], qscale)
    kw = dict(prefix_pages=dev(pre), prefix_len=i32([prefix])) if prefix else {}
    out = c.decode_attn(q, dev(table), i32(lens), softmax_scale=scale, **kw)
    assert c.status() == 0
    want, vmax, smax = reference(q, values(c, "k"), values(c, "v"), table, lens, pre, prefix, page,
                                 scale if scale > 0 else None)
    check_attention(out, want, vmax, smax, f"{fmt} H{H} G{G} D{D} page{page} prefix{prefix}")
    return c, q, out


@pytest.mark.parametrize("fmt", ["fp16", "aff8", "aff4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 131])
def test_attention_formats(kvq, fmt, D, page, prefix):
    for dtype in ("bf16", "fp16"):
        run_attention(kvq, fmt, 2, 4, D, page, [1, 64, 0, 65, 200, 16, 127], prefix, dtype, seed=page)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("H", [1, 3])
def test_attention_head_groups(kvq, G, H):
    for prefix in (0, 300):
        run_attention(kvq, "aff4", H, G, 128, 64, [100, 3, 64], prefix, "bf16", seed=G)
        run_attention(kvq, "fp16", H, G, 64, 16, [77, 130], prefix, "fp16", seed=G)


@pytest.mark.parametrize("kg,vg", [(32, 32), (32, 128), (128, 32), (64, 128), (128, 128)])
@pytest.mark.parametrize("fmt", ["aff8", "aff4"])
def test_attention_groups(kvq, fmt, kg, vg):
    run_attention(kvq, fmt, 2, 4, 128, 64, [129, 1, 300], 200, "fp16", kg, vg, seed=kg + vg)
    run_attention(kvq, fmt, 2, 5, 64, 32, [129, 1, 300], 77, "bf16", kg, vg, seed=kg + vg)


@pytest.mark.parametrize("B", [1, 2, 17, 33, 70])
@pytest.mark.parametrize("fmt", ["fp16", "aff8", "aff4"])
def test_attention_shared_prefix_batches(kvq, B, fmt):
    lens = [(37 * b) % 90 for b in range(B)]
    run_attention(kvq, fmt, 2, 4, 128, 64, lens, 1000, "bf16", seed=B)
    run_attention(kvq, fmt, 1, 7, 64, 16, lens, 513, "bf16", seed=B)


@pytest.mark.parametrize("fmt", ["fp16", "aff4"])
def test_attention_long(kvq, fmt):
    run_attention(kvq, fmt, 1, 4, 128, 64, [5000, 9, 0, 20011], 0, "bf16", seed=1)
    run_attention(kvq, fmt, 1, 8, 128, 128, [3, 1, 0, 64], 20011, "bf16", seed=2)


def test_attention_empty_rows_are_zero(kvq):
    c, _, out = run_attention(kvq, "aff8", 2, 3, 128, 64, [0, 5, 0], 0, "bf16")
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0)
    # negative lengths count as none, and a prefix of length 0 as no prefix
    q = torch.ones((2, 6, 128), dtype=torch.bfloat16, device="cuda")
    out = c.decode_attn(q, i32([[0], [0]]), i32([-3, 0]), prefix_pages=i32([1, 2]), prefix_len=i32([0]))
    assert torch.all(out == 0)
    out = c.decode_attn(q, i32([[0], [0]]), i32([0, 0]), prefix_pages=i32([1, 2]), prefix_len=i32([-9]))
    assert torch.all(out == 0) and c.status() == 0
    # a table without columns
    out = c.decode_attn(q, torch.zeros((2, 0), dtype=torch.int32, device="cuda"), i32([0, 0]))
    assert torch.all(out == 0) and c.status() == 0


@pytest.mark.parametrize("scale,qscale", [(0.3, 1.0), (0.02, 40.0), (1.0, 3.0)])
def test_attention_scales_and_sharp_softmax(kvq, scale, qscale):
    run_attention(kvq, "aff8", 2, 4, 128, 64, [200, 1, 70], 150, "bf16", scale=scale, qscale=qscale)
    run_attention(kvq, "fp16", 2, 4, 64, 16, [200, 1, 70], 150, "bf16", scale=scale, qscale=qscale)


def test_attention_ignores_rows_past_the_lengths(kvq):
    # NaN, infinities and the types' largest values in rows behind the lengths of every page reach nothing
    for fmt in ("fp16", "aff8", "aff4"):
        for page, prefix in ((64, 100), (16, 35), (128, 130)):
            lens = [3, 0, 66, 17]
            table, pre, n_pages = tables(lens, prefix, page, seed=9)
            c = make_pool(kvq, fmt, 2, 64, page, n_pages, seed=10)
            q = rand((4, 8, 64), torch.Generator().manual_seed(1), torch.bfloat16)
            args = (q, dev(table), i32(lens))
            kw = dict(prefix_pages=dev(pre), prefix_len=i32([prefix]))
            clean = c.decode_attn(*args, **kw)
            live = np.zeros((n_pages, page), dtype=bool)
            for row, n in [(pre, prefix)] + list(zip(table, lens)):
                ids, rows = opos.page_rows(row, n, page)
                live[ids, rows] = True
            dead = dev(~live)
            for bad in (float("nan"), float("inf"), -65504.0):
                for side in "kv":
                    x = c.plane(side + ("_codes" if fmt == "fp16" else "_meta"))
                    x.transpose(1, 2)[dead] = bad
                assert torch.equal(c.decode_attn(*args, **kw), clean), (fmt, page, bad)


def test_attention_bad_pages(kvq):
    # rows of pages outside the pool, or past the table, are left out and the status says so
    H, D, page = 2, 128, 64
    c = make_pool(kvq, "aff4", H, D, page, 6, seed=12)
    q = rand((1, 8, D), torch.Generator().manual_seed(2), torch.bfloat16)
    kv, vv = values(c, "k"), values(c, "v")
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        for where in (0, 1, 2):
            row = [3, 1, 5]
            row[where] = bad
            out = c.decode_attn(q, i32([row]), i32([150]))
            assert c.status() == kvq.DEV_BAD_PAGE
            c.clear_status()
            n = [64, 64, 22]
            keep = [i for i in range(3) if i != where]
            k = np.concatenate([kv[row[i], :, :n[i]] for i in keep], 1)
            v = np.concatenate([vv[row[i], :, :n[i]] for i in keep], 1)
            pk, pv = k[None].transpose(0, 2, 1, 3), v[None].transpose(0, 2, 1, 3)   # one page of all rows
            want, vm, sm = reference(q, pk.transpose(0, 2, 1, 3), pv.transpose(0, 2, 1, 3), [[0]], [k.shape[1]], [], 0,
                                     k.shape[1])
            check_attention(out, want, vm, sm)
            out = c.decode_attn(q, i32([[2]]), i32([0]), prefix_pages=i32(row), prefix_len=i32([150]))
            assert c.status() == kvq.DEV_BAD_PAGE
            c.clear_status()
            check_attention(out, want, vm, sm)
    short = c.decode_attn(q, i32([[4]]), i32([64]))
    assert c.status() == 0
    assert torch.equal(c.decode_attn(q, i32([[4]]), i32([100])), short) and c.status() == kvq.DEV_BAD_PAGE
    c.clear_status()
    none = c.decode_attn(q, i32([[-1]]), i32([64]))
    assert torch.all(none == 0) and c.status() == kvq.DEV_BAD_PAGE


def test_attention_is_the_same_every_time(kvq):
    for fmt in ("fp16", "aff4"):
        c, q, out = run_attention(kvq, fmt, 2, 4, 128, 64, [500, 3, 64, 1000], 700, "bf16", seed=21)
        table, pre, _ = tables([500, 3, 64, 1000], 700, 64, seed=21)
        for _ in range(5):
            again = c.decode_attn(q, dev(table), i32([500, 3, 64, 1000]), prefix_pages=dev(pre), prefix_len=i32([700]))
            assert torch.equal(again, out)


def test_attention_pages_shared_between_sequences(kvq):
    # two sequences over the same pages, and one page twice in a row
    c = make_pool(kvq, "aff8", 1, 64, 16, 5, seed=13)
    q = rand((2, 4, 64), torch.Generator().manual_seed(3), torch.bfloat16)
    q[1] = q[0]
    out = c.decode_attn(q, i32([[2, 3, 2], [2, 3, 2]]), i32([48, 48]))
    assert torch.equal(out[0], out[1])
    kv, vv = values(c, "k"), values(c, "v")
    table = np.array([[2, 3, 2], [2, 3, 2]])
    want, vm, sm = reference(q, kv, vv, table, [48, 48], [], 0, 16)
    check_attention(out, want, vm, sm)


def test_steps_together_and_replayed(kvq):
    # the prefix appended as a sequence of its own, then decode steps (norm, rotation, append, attention)
    # in one captured graph that follows the lengths, against float64 over what the pool holds
    H, G, D, page, B, prefix = 2, 4, 128, 64, 3, 150
    g = torch.Generator().manual_seed(31)
    rope = kvq.Rope(D, 10000.0)
    n_pages = 3 + B * 2
    pre, table = np.arange(3, dtype=np.int32), (3 + np.arange(B * 2, dtype=np.int32)).reshape(B, 2)
    c = make_pool(kvq, "aff4", H, D, page, n_pages, fill=False)
    pk, pv = rand((prefix, H, D), g, torch.bfloat16), rand((prefix, H, D), g, torch.bfloat16)
    c.append(pk, pv, dev(pre[None]), i32([prefix]), cu_tokens=i32([0, prefix]), rope=rope)
    w = rand((D,), g, torch.bfloat16)
    q, k, v = (torch.empty((B, h, D), dtype=torch.bfloat16, device="cuda") for h in (H * G, H, H))
    lens, tab, plen, pp = i32([0, 70, 20]), dev(table), i32([prefix]), dev(pre)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(max(16, c.workspace_bytes(B, H * G, 3)), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        c.append(k, v, tab, lens, q=q, rope=rope, prefix_len=plen, q_out=qr, q_norm=w, k_norm=w)
        c.decode_attn(qr, tab, lens, prefix_pages=pp, prefix_len=plen, out=out, workspace=ws)

    step()
    lens.copy_(i32([0, 70, 20]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    f, _ = opos.frequencies(D, 10000.0)
    for i in range(4):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        now = [n + i + 1 for n in (0, 70, 20)]
        assert lens.tolist() == now and c.status() == 0
        # the rotated queries are those of the formula, and attention is over the pool's values
        want_q = opos.rotate(opos.head_norm(host(q), host(w), 1e-6), np.array([prefix + n - 1 for n in now]), f)
        assert np.abs(host(qr) - want_q).max() <= 2.0 ** -8 * np.abs(want_q).max()
        want, vm, sm = reference(qr, values(c, "k"), values(c, "v"), table, now, pre, prefix, page)
        check_attention(out, want, vm, sm, f"step {i}")


def test_two_streams_with_their_own_workspaces(kvq):
    H, G, D, page, lens, prefix = 2, 4, 128, 64, [900, 3, 400], 500
    table, pre, n = tables(lens, prefix, page, seed=41)
    c = make_pool(kvq, "aff4", H, D, page, n, seed=42)
    q = rand((3, H * G, D), torch.Generator().manual_seed(4), torch.bfloat16)
    q2 = q * 0.5
    args = (dev(table), i32(lens))
    kw = dict(prefix_pages=dev(pre), prefix_len=i32([prefix]))
    want, want2 = c.decode_attn(q, *args, **kw), c.decode_attn(q2, *args, **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(max(16, c.workspace_bytes(3, H * G, len(pre))), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s, x, w in zip(streams, (q, q2), ws):
            outs.append(c.decode_attn(x, *args, workspace=w, stream=s, **kw))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, (want, want2)[i % 2])


def test_refusals_with_a_pool(kvq):
    c = make_pool(kvq, "aff4", 2, 128, 64, 4, fill=False)
    k = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    t, n = i32([[0]]), i32([1])
    with pytest.raises(ValueError, match="must be"):
        c.append(k, k.float(), t, n)
    with pytest.raises(ValueError, match="page_table"):
        c.append(k, k, i32([[0], [1]]), n)
    with pytest.raises(ValueError, match="cu_tokens"):
        c.append(k, k, t, n, cu_tokens=i32([0]))
    with pytest.raises(kvq.KvqError, match="heads"):
        c.append(k[:, :1], k[:, :1], t, n)
    with pytest.raises(kvq.KvqError, match="rot_dim"):
        make_pool(kvq, "fp16", 2, 64, 64, 1, fill=False).append(k[..., :64], k[..., 64:], t, n, rope=kvq.Rope(128))
    with pytest.raises(kvq.KvqError, match="one token per sequence"):
        c.append(k.expand(2, 2, 128), k.expand(2, 2, 128), t, n)
    with pytest.raises(kvq.KvqError, match="bf16 or fp16"):
        c.decode_attn(q.float(), t, n)
    with pytest.raises(kvq.KvqError, match="8 query heads"):
        c.decode_attn(torch.zeros((1, 18, 128), dtype=torch.bfloat16, device="cuda"), t, n)
    with pytest.raises(kvq.KvqError, match="multiple"):
        c.decode_attn(q[:, :3].contiguous(), t, n)
    with pytest.raises(ValueError, match="prefix_len"):
        c.decode_attn(q, t, n, prefix_pages=i32([1]))
    with pytest.raises(ValueError, match="one row per sequence"):
        c.decode_attn(q.expand(2, 8, 128).contiguous(), t, n)
    if c.workspace_bytes(64, 16, 100) > 16:
        with pytest.raises(kvq.KvqError, match="workspace"):
            c.decode_attn(torch.zeros((64, 16, 128), dtype=torch.bfloat16, device="cuda"), i32([[0]] * 64), i32([1] * 64),
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="CUDA tensor"):
        c.decode_attn(q, t.cpu(), n)
    assert c.status() == 0


def test_wait_that_runs_out_reports_and_recovers(kvq):
    # a tile that never arrives: the bounded waits give up, the status says so, the next call is right
    H, G, D, page, lens, prefix = 2, 4, 64, 16, [100, 5], 40
    table, pre, n = tables(lens, prefix, page, seed=51)
    c = make_pool(kvq, "aff8", H, D, page, n, seed=52)
    q = rand((2, H * G, D), torch.Generator().manual_seed(5), torch.bfloat16)
    args, kw = (q, dev(table), i32(lens)), dict(prefix_pages=dev(pre), prefix_len=i32([prefix]))
    want = c.decode_attn(*args, **kw)
    torch.cuda.synchronize()
    kvq.kvq_test_stall_decode_tiles(True)
    try:
        c.decode_attn(*args, **kw)
        assert c.status() == kvq.DEV_TIMEOUT
    finally:
        kvq.kvq_test_stall_decode_tiles(False)
    c.clear_status()
    assert torch.equal(c.decode_attn(*args, **kw), want) and c.status() == 0


# Prefixes long enough, for their batches, to be taken once for all sequences (on up to 152 SMs).
SHARED = [
    # (B, H, G, D, page, prefix)
    (3, 8, 4, 64, 64, 11000),       # a dozen query rows per kv head, long runs
    (65, 4, 1, 128, 16, 1025),      # one row tile, a tile of one row at the end
    (33, 4, 4, 64, 32, 2100),       # rows just past one tile of 128
    (100, 4, 8, 128, 128, 800),     # four CTAs of rows
    (40, 8, 3, 128, 64, 897),
]


@pytest.mark.parametrize("fmt,kg,vg", [("fp16", 0, 0), ("aff8", 128, 32), ("aff4", 64, 64), ("aff4", 32, 128)])
@pytest.mark.parametrize("shape", SHARED)
def test_attention_prefix_taken_once(kvq, shape, fmt, kg, vg):
    B, H, G, D, page, prefix = shape
    lens = [(37 * b) % 70 for b in range(B)]
    c, q, out = run_attention(kvq, fmt, H, G, D, page, lens, prefix, "bf16", kg or 64, vg or 64, seed=B)
    assert c.launches == 3   # prefix, own rows, merge
    table, pre, _ = tables(lens, prefix, page, seed=B)
    kw = dict(prefix_pages=dev(pre), prefix_len=i32([prefix]))
    assert torch.equal(c.decode_attn(q, dev(table), i32(lens), **kw), out)
    run_attention(kvq, fmt, H, G, D, page, lens, prefix, "fp16", kg or 64, vg or 64, seed=B, qscale=4.0)


def test_prefix_taken_once_follows_its_length(kvq):
    # the plan goes by the tables' width, the work by the length on the device: from nothing to the whole table
    B, H, G, D, page, most = 33, 4, 4, 64, 64, 2112
    lens = [(11 * b) % 40 for b in range(B)]
    table, pre, n = tables(lens, most, page, seed=61)
    c = make_pool(kvq, "aff8", H, D, page, n, seed=62)
    q = rand((B, H * G, D), torch.Generator().manual_seed(6), torch.bfloat16)
    plen = i32([0])
    for prefix in (0, 1, 127, 128, 129, 1000, 2111, 2112):
        plen.fill_(prefix)
        out = c.decode_attn(q, dev(table), i32(lens), prefix_pages=dev(pre), prefix_len=plen)
        want, vm, sm = reference(q, values(c, "k"), values(c, "v"), table, lens, pre, prefix, page)
        check_attention(out, want, vm, sm, f"prefix {prefix}")
    assert c.status() == 0
    plen.fill_(most + 1)
    again = c.decode_attn(q, dev(table), i32(lens), prefix_pages=dev(pre), prefix_len=plen)
    assert torch.equal(again, out) and c.status() == kvq.DEV_BAD_PAGE


def test_prefix_taken_once_ignores_rows_past_the_length_and_bad_pages(kvq):
    B, H, G, D, page, prefix = 33, 4, 4, 64, 64, 2100
    lens = [(13 * b) % 30 for b in range(B)]
    for fmt in ("fp16", "aff8", "aff4"):
        table, pre, n = tables(lens, prefix, page, seed=71)
        c = make_pool(kvq, fmt, H, D, page, n, seed=72)
        q = rand((B, H * G, D), torch.Generator().manual_seed(7), torch.bfloat16)
        args, kw = (q, dev(table), i32(lens)), dict(prefix_pages=dev(pre), prefix_len=i32([prefix]))
        clean = c.decode_attn(*args, **kw)
        live = np.zeros((n, page), dtype=bool)
        for row, m in [(pre, prefix)] + list(zip(table, lens)):
            ids, rows = opos.page_rows(row, m, page)
            live[ids, rows] = True
        for bad in (float("nan"), float("inf"), -65504.0):
            for side in "kv":
                c.plane(side + ("_codes" if fmt == "fp16" else "_meta")).transpose(1, 2)[dev(~live)] = bad
            assert torch.equal(c.decode_attn(*args, **kw), clean), (fmt, bad)
        # a page outside the pool is left out
        kv, vv = values(c, "k"), values(c, "v")
        hole = pre.copy()
        hole[5] = n
        out = c.decode_attn(*args, prefix_pages=dev(hole), prefix_len=i32([prefix]))
        assert c.status() == kvq.DEV_BAD_PAGE
        keep = np.delete(pre, 5)
        want, vm, sm = reference(q, kv, vv, table, lens, keep, prefix - page, page)
        check_attention(out, want, vm, sm, fmt)


@pytest.mark.parametrize("fmt", ["fp16", "aff8", "aff4"])
@pytest.mark.parametrize("B,G", [(33, 4), (33, 3)])   # two row tiles a CTA, and one
def test_prefix_taken_once_starts_with_dead_tiles(kvq, fmt, B, G):
    # whole tiles out of the pool in front of live ones, with scores too small to move a maximum: the first
    # live tile sets the row's reference.  Also every page but the last one, and every page.
    H, D, page, prefix = 4, 64, 64, 2100
    lens = [0] * B
    table, pre, n = tables(lens, prefix, page, seed=101)
    c = make_pool(kvq, fmt, H, D, page, n, seed=102)
    q = rand((B, H * G, D), torch.Generator().manual_seed(11), torch.bfloat16, 0.05)
    kv, vv = values(c, "k"), values(c, "v")
    for dead in (4, 16, len(pre) - 1, len(pre)):
        hole = pre.copy()
        hole[:dead] = -1
        out = c.decode_attn(q, dev(table), i32(lens), prefix_pages=dev(hole), prefix_len=i32([prefix]))
        assert c.status() == kvq.DEV_BAD_PAGE
        want, vm, sm = reference(q, kv, vv, table, lens, pre[dead:], max(prefix - dead * page, 0), page)
        check_attention(out, want, vm, sm, f"{fmt} {dead} dead pages")
    # the same as every other page
    hole = pre.copy()
    hole[::2] = n
    out = c.decode_attn(q, dev(table), i32(lens), prefix_pages=dev(hole), prefix_len=i32([prefix]))
    keep = pre[1::2]
    want, vm, sm = reference(q, kv, vv, table, lens, keep, len(keep) * page, page)
    check_attention(out, want, vm, sm, f"{fmt} odd pages")


def test_prefix_taken_once_wait_that_runs_out(kvq):
    B, H, G, D, page, prefix = 65, 4, 1, 64, 64, 1100
    lens = [5] * B
    for fmt in ("fp16", "aff4"):
        table, pre, n = tables(lens, prefix, page, seed=81)
        c = make_pool(kvq, fmt, H, D, page, n, seed=82)
        q = rand((B, H * G, D), torch.Generator().manual_seed(8), torch.bfloat16)
        args, kw = (q, dev(table), i32(lens)), dict(prefix_pages=dev(pre), prefix_len=i32([prefix]))
        want = c.decode_attn(*args, **kw)
        torch.cuda.synchronize()
        kvq.kvq_test_stall_decode_tiles(True)
        try:
            c.decode_attn(*args, **kw)
            assert c.status() == kvq.DEV_TIMEOUT
        finally:
            kvq.kvq_test_stall_decode_tiles(False)
        c.clear_status()
        assert torch.equal(c.decode_attn(*args, **kw), want) and c.status() == 0


def test_workspace_covers_smaller_calls(kvq):
    # bytes for "up to" n sequences and pages hold for fewer of either
    c = make_pool(kvq, "fp16", 8, 64, 64, 1, fill=False)
    for hq in (8, 32, 64):
        for pages in (0, 3, 40, 600):
            sizes = [c.workspace_bytes(n, hq, pages) for n in range(1, 400)]
            assert sizes == sorted(sizes)
            assert all(a <= b for a, b in zip(sizes[::37], [c.workspace_bytes(n, hq, pages + 100) for n in range(1, 400, 37)]))
    small = c.decode_attn(torch.zeros((64, 32, 64), dtype=torch.bfloat16, device="cuda"), i32([[0]] * 64), i32([1] * 64),
                          prefix_pages=i32([0] * 20), prefix_len=i32([1200]),
                          workspace=torch.empty(c.workspace_bytes(300, 32, 40), dtype=torch.uint8, device="cuda"))
    assert small.shape == (64, 32, 64) and c.status() == 0


def test_extreme_values(kvq):
    # queries from the ends of bf16's range, one key of -inf, values near fp16's largest
    B, H, D, page = 33, 4, 64, 64
    for prefix in (0, 2100):
        lens = [40] * B
        table, pre, n = tables(lens, prefix, page, seed=91)
        c = make_pool(kvq, "fp16", H, D, page, n, seed=92)
        c.plane("v_codes").mul_(1e4)
        q = rand((B, H * 4, D), torch.Generator().manual_seed(9), torch.float32)
        q[:, 0] *= 1e30
        q[:, 1] *= 1e-30
        q[:, 2] = 0
        q = q.to(torch.bfloat16)
        kw = dict(prefix_pages=dev(pre), prefix_len=i32([prefix])) if prefix else {}
        out = c.decode_attn(q, dev(table), i32(lens), **kw)
        want, vm, sm = reference(q, values(c, "k"), values(c, "v"), table, lens, pre, prefix, page)
        # (head 0's softmax is one key's: its smax bound says nothing, its values are checked as they are)
        check_attention(out[:, 1:], want[:, 1:], vm[:, 1:], sm[:, 1:], f"prefix {prefix}")
        assert np.abs(host(out[:, 0]) - want[:, 0]).max() <= 2.0 ** -8 * np.abs(want[:, 0]).max() + 1e4 * 2.0 ** -10


def test_groups_of_graphs_replay_together(kvq):
    # two captured calls of one pool, replayed on two streams at once, keep out of each other's workspace
    B, H, G, D, page, prefix = 33, 4, 4, 64, 64, 2100
    lens = [(17 * b) % 200 for b in range(B)]
    table, pre, n = tables(lens, prefix, page, seed=95)
    c = make_pool(kvq, "aff4", H, D, page, n, seed=96)
    t, l, pp, pl = dev(table), i32(lens), dev(pre), i32([prefix])
    qs = [rand((B, H * G, D), torch.Generator().manual_seed(i), torch.bfloat16) for i in (1, 2)]
    want = [c.decode_attn(q, t, l, prefix_pages=pp, prefix_len=pl) for q in qs]
    outs, graphs = [torch.empty_like(q) for q in qs], []
    for q, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.decode_attn(q, t, l, prefix_pages=pp, prefix_len=pl, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_pages_beyond_4_gib(kvq):
    # planes larger than 32 bits of bytes: the last pages of a 5 GiB plane hold what the first ones would
    H, D, page, n = 8, 128, 128, 20480
    c = make_pool(kvq, "fp16", H, D, page, n, fill=False)
    small = make_pool(kvq, "fp16", H, D, page, 4, fill=False)
    g = torch.Generator().manual_seed(97)
    k, v = rand((300, H, D), g, torch.bfloat16), rand((300, H, D), g, torch.bfloat16)
    q = rand((1, H * 4, D), g, torch.bfloat16)
    outs = []
    for pool, ids in ((c, [n - 1, 16500, n - 3]), (small, [3, 0, 1])):
        pool.append(k, v, i32([ids]), i32([300]), cu_tokens=i32([0, 300]))
        outs.append(pool.decode_attn(q, i32([ids]), i32([300])))
        assert pool.status() == 0
    assert torch.equal(outs[0], outs[1])
    for a, b in zip([n - 1, 16500, n - 3], [3, 0, 1]):
        assert torch.equal(c.plane("k_codes")[a], small.plane("k_codes")[b])


def test_prefix_beyond_4_gib_taken_once(kvq):
    H, D, page, n = 8, 128, 128, 20480
    c = make_pool(kvq, "fp16", H, D, page, n, fill=False)
    small = make_pool(kvq, "fp16", H, D, page, 12, fill=False)
    g = torch.Generator().manual_seed(98)
    k, v = rand((1100, H, D), g, torch.bfloat16), rand((1100, H, D), g, torch.bfloat16)
    B = 33
    q = rand((B, H * 4, D), g, torch.bfloat16)
    outs = []
    for pool, ids in ((c, list(range(n - 9, n))), (small, list(range(9)))):
        pool.append(k, v, i32([ids]), i32([1100]), cu_tokens=i32([0, 1100]))
        outs.append(pool.decode_attn(q, i32([[0]] * B), i32([0] * B), prefix_pages=i32(ids), prefix_len=i32([1100])))
        assert pool.status() == 0 and pool.launches == 1 + 3
    assert torch.equal(outs[0], outs[1])


def test_a_growing_batch_keeps_one_workspace(kvq):
    # a pool's own workspace grows with the batch; the smaller ones are given back
    c = make_pool(kvq, "fp16", 8, 64, 64, 1, fill=False)
    pages, plen = i32([0] * 40), i32([2500])
    q, out = torch.zeros((2, 400, 32, 64), dtype=torch.bfloat16, device="cuda")
    tab, lens = i32([[0]] * 400), i32([1] * 400)
    before = torch.cuda.memory_allocated()
    for n in range(2, 401, 2):
        c.decode_attn(q[:n], tab[:n], lens[:n], prefix_pages=pages, prefix_len=plen, out=out[:n])
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before <= c.workspace_bytes(400, 32, 40) + (2 << 20)


@pytest.mark.parametrize("fmt,G,dtype", [("aff8", 4, torch.bfloat16), ("aff4", 4, torch.bfloat16),
                                         ("aff4", 8, torch.bfloat16), ("aff8", 8, torch.float16)])
def test_extreme_queries_next_to_stored_codes(kvq, fmt, G, dtype):
    # the power of two that brings a query to its codes' size, at both ends of it
    B, H, D, page = 3, 2, 64, 32
    lens = [1, 40, 70]
    table, pre, n = tables(lens, 0, page, seed=101)
    c = make_pool(kvq, fmt, H, D, page, n, kgroup=64, vgroup=64, seed=102)
    q = rand((B, H * G, D), torch.Generator().manual_seed(10), torch.float32)
    bf = dtype is torch.bfloat16
    q[:, 0] *= 1e30 if bf else 1e4
    q[:, 1] *= 1e-37 if bf else 1e-6
    q[:, 2] = 0
    q = q.to(dtype)
    out = c.decode_attn(q, dev(table), i32(lens))
    want, vm, sm = reference(q, values(c, "k"), values(c, "v"), table, lens, pre, 0, page)
    # (head 0's softmax is one key's: its smax bound says nothing, a rounding of weight 1 and of the output remain)
    check_attention(out[:, 1:], want[:, 1:], vm[:, 1:], sm[:, 1:], fmt)
    err = np.abs(host(out[:, 0]) - want[:, 0])
    assert (err <= torch.finfo(dtype).eps * np.abs(want[:, 0]) + 2.0 ** -10 * np.abs(want[:, 0]).max()).all()
