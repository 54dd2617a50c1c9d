"""GPU parity of rope_qk (rotary positions, per-head norms) with float64.

Tolerance: the result of the fp32 arithmetic rounded once to the output
type, half a step of it (finfo.eps / 2).  In fp32 the angle is off by at
most 2^-24 pi (half a unit of a 24-bit half-turn, twice over for the cut to
32 bits and sincospif's own rounding), the products and their sum by a few
2^-24, the norm (a sum of D squares by E-term lanes and five shuffles, a square root
and a division) by under 16 of them: together under 32 * 2^-24 = 2^-19 of the pair's
two magnitudes."""
import numpy as np
import pytest
import torch

from kvq_helpers import host
from oracle import positions as opos

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def kvq():
    import bit_kv_cache_quant_gb300 as m

    return m


def expected(x, pos, weight, eps, rot, base, scaling, inter, mag=None, **p):
    """(float64 rows, magnitude of each channel's pair)."""
    x = host(x).astype(np.float64)
    if weight is not None:
        x = opos.head_norm(x, host(weight), eps)
    f, m = opos.frequencies(rot, base, scaling, **p)
    y = opos.rotate(x, pos, f, m if mag is None else mag, inter)
    # both channels of a pair, each way round: |a| + |b|
    both = np.abs(x)
    ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    ib = ia + (1 if inter else rot // 2)
    s = (both[..., ia] + both[..., ib]) * m
    both[..., ia], both[..., ib] = s, s
    return y, both


def check(got, want, both, dtype, what=""):
    slack = 2.0 ** -19 * both
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps   # half a step of subnormals at most
    tol = half * (np.abs(want) + slack) + slack + tiny
    err = np.abs(host(got).astype(np.float64) - want)
    assert np.all(err <= tol), f"{what}: {(err > tol).sum()} off, worst {(err / tol).max():.2f} of the tolerance"


def rand(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D,rot", [(32, 32), (32, 10), (64, 64), (64, 32), (128, 128), (128, 64), (128, 96), (128, 6),
                                   (256, 256), (256, 50)])
@pytest.mark.parametrize("inter", [False, True])
def test_rotation(kvq, dtype, D, rot, inter):
    g = torch.Generator().manual_seed(D + rot)
    T = 7
    q, k = rand((T, 5, D), g, DT[dtype]), rand((T, 2, D), g, DT[dtype])
    pos = torch.tensor([0, 1, -3, 4096, 1000003, 2 ** 31 - 1, 77], dtype=torch.int32)
    rope = kvq.Rope(rot, 10000.0, interleaved=inter)
    qo, ko = kvq.rope_qk(q, k, pos.cuda(), rope)
    for x, y in ((q, qo), (k, ko)):
        want, both = expected(x, pos.numpy(), None, 0, rot, 10000.0, "none", inter)
        check(y, want, both, DT[dtype])
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaling,p", [
    ("linear", dict(factor=4.0)), ("ntk", dict(factor=4.0)),
    ("yarn", dict(factor=16.0, original_max_position=4096, beta_fast=32.0, beta_slow=1.0)),
    ("llama3", dict(factor=8.0, original_max_position=8192, low_freq_factor=1.0, high_freq_factor=4.0)),
    ("factors", dict(factors=[1.0 + 0.5 * i for i in range(64)])),
])
def test_scalings_far_out(kvq, scaling, p):
    g = torch.Generator().manual_seed(1)
    q = rand((33, 3, 128), g, torch.float32)
    pos = torch.arange(33, dtype=torch.int32) * 65521
    qo, none = kvq.rope_qk(q, None, pos.cuda(), kvq.Rope(128, 500000.0, scaling=scaling, **p))
    assert none is None
    want, both = expected(q, pos.numpy(), None, 0, 128, 500000.0, scaling, False, **p)
    check(qo, want, both, torch.float32)


@pytest.mark.parametrize("T", [1, 2, 63, 1000, 5003])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128, 256])
def test_norm_and_rotation(kvq, T, dtype, D):
    g = torch.Generator().manual_seed(T)
    q, k = rand((T, 3, D), g, DT[dtype], 5.0), rand((T, 1, D), g, DT[dtype], 0.01)
    k[T // 2] = 0
    wq, wk = rand((D,), g, DT[dtype]), rand((D,), g, DT[dtype])
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    qo, ko = kvq.rope_qk(q, k, pos.cuda(), kvq.Rope(D, 10000.0), q_norm=wq, k_norm=wk, eps=1e-5)
    for x, y, w in ((q, qo, wq), (k, ko, wk)):
        want, both = expected(x, pos.numpy(), w, 1e-5, D, 10000.0, "none", False)
        check(y, want, both, DT[dtype])
    # the norm alone
    qn, _ = kvq.rope_qk(q, None, None, None, q_norm=wq, eps=1e-5)
    want = opos.head_norm(host(q), host(wq), 1e-5)
    check(qn, want, np.abs(want), DT[dtype])


@pytest.mark.parametrize("off", [0, 1, 2, 4])
@pytest.mark.parametrize("dtype", list(DT))
def test_strided_views_and_in_place(kvq, dtype, off):
    # q and k as slices of one projection (at `off` elements from its start), rotated in place: v and the
    # rest stay as they were, and the bytes are those of the out-of-place call
    g = torch.Generator().manual_seed(off)
    T, hq, hk, D = 19, 6, 2, 128
    wide = (hq + 2 * hk) * D + 8
    buf = rand((T * wide + 16,), g, DT[dtype])
    qkv = buf[off:off + T * wide].view(T, wide)
    q, k = qkv[:, :hq * D].view(T, hq, D), qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    rope = kvq.Rope(D, 10000.0)
    before = buf.clone()
    qo, ko = kvq.rope_qk(q, k, pos, rope)
    want, both = expected(q, pos.cpu().numpy(), None, 0, D, 10000.0, "none", False)
    check(qo, want, both, DT[dtype])
    assert torch.equal(buf, before)
    # heads before tokens
    qt = torch.empty((hq, T, D), dtype=DT[dtype], device="cuda")
    kvq.rope_qk(q, None, pos, rope, q_out=qt.transpose(0, 1))
    assert torch.equal(qt.transpose(0, 1), qo)
    kvq.rope_qk(q, k, pos, rope, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[off:off + T * wide].view(T, wide)[:, :(hq + hk) * D] = False
    assert torch.equal(buf[rest], before[rest])


def test_negative_positions_undo(kvq):
    g = torch.Generator().manual_seed(3)
    q = rand((50, 4, 64), g, torch.float32)
    pos = (torch.arange(50, dtype=torch.int32) * 99991).cuda()
    rope = kvq.Rope(64, 10000.0)
    there, _ = kvq.rope_qk(q, None, pos, rope)
    back, _ = kvq.rope_qk(there, None, -pos, rope)
    # two passes of the file's fp32 bound
    assert (back - q).abs().max().item() <= 2 * 2.0 ** -19 * 2 * q.abs().max().item()


def test_non_finite_rows_stay_in_their_row(kvq):
    g = torch.Generator().manual_seed(4)
    q = rand((4, 3, 128), g, torch.bfloat16)
    pos = torch.arange(4, dtype=torch.int32).cuda()
    rope = kvq.Rope(128)
    clean, _ = kvq.rope_qk(q, None, pos, rope)
    q[2, 1, 5] = float("nan")
    q[1, 0, 0] = float("inf")
    out, _ = kvq.rope_qk(q, None, pos, rope)
    keep = torch.ones((4, 3), dtype=torch.bool, device="cuda")
    keep[2, 1] = keep[1, 0] = False
    assert torch.equal(out[keep], clean[keep])
    assert out[2, 1].isnan().sum().item() == 2


def test_many_tokens_match_few(kvq):
    # the launch's shape goes by the number of tokens; the bytes do not
    g = torch.Generator().manual_seed(5)
    T = 20011
    q, k = rand((T, 8, 64), g, torch.bfloat16), rand((T, 2, 64), g, torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    w = rand((64,), g, torch.bfloat16)
    rope = kvq.Rope(64)
    qo, ko = kvq.rope_qk(q, k, pos, rope, q_norm=w)
    for a in (0, 9999, T - 5):
        qs, ks = kvq.rope_qk(q[a:a + 5], k[a:a + 5], pos[a:a + 5], rope, q_norm=w)
        assert torch.equal(qs, qo[a:a + 5]) and torch.equal(ks, ko[a:a + 5])


def test_empty_stream_and_graph(kvq):
    rope = kvq.Rope(128)
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    qo, ko = kvq.rope_qk(e, e, torch.empty(0, dtype=torch.int32, device="cuda"), rope)
    assert qo.shape == e.shape and ko.shape == e.shape
    g = torch.Generator().manual_seed(6)
    q = rand((9, 4, 128), g, torch.bfloat16)
    pos = torch.arange(9, dtype=torch.int32).cuda()
    want, _ = kvq.rope_qk(q, None, pos, rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = kvq.rope_qk(q, None, pos, rope, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.rope_qk(q, None, pos, rope, q_out=out)
    pos.add_(5)
    graph.replay()
    torch.cuda.synchronize()
    want, _ = kvq.rope_qk(q, None, pos, rope)
    assert torch.equal(out, want)
