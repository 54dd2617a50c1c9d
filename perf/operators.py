"""Timed cases of the rotary, paged-append and shared-prefix decode operators.

Each case is one call (`rope_qk`, `PagedKVCache.append`, `PagedKVCache.decode_attn`) on inputs as a serving
step has them in hand.  `run` computes the operators either from elementary torch operations in 32 bits
(64 for the rotation's angles), or, where `own` is true, through this package.  `exact` states the same
definitions in 64 bits.

The page pool is one buffer: 256 bytes of state, then the planes k_codes, k_meta, v_codes, v_meta, each
starting at a multiple of 256 bytes.  Codes are [page][kv head][row in page][bytes of a row]: fp16 values,
8-bit levels stored as u - 128, or nibbles with channel 2j in the low half of byte j.  Metadata is fp16
[page][kv head][row in page][group][scale, zero] (absent for fp16 rows).
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BITS = {"fp16": 16, "aff8": 8, "aff4": 4}

# name -> (kind, parameters) of the frequency scalings the cases use
SCALINGS = {
    "none": {},
    "linear": {"factor": 4.0},
    "llama3": {"factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original_max_position": 8192},
    "yarn": {"factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original_max_position": 4096},
}


def listed():
    return [
        # One decoding token: pure launch latency.
        dict(name="rope_token", op="rope", tokens=1, hq=32, hk=8, d=128, rot=128, inter=False, scaling="llama3",
             base=500000.0, first=8192, dtype="bf16"),
        # A 32K prompt of a 32/8-head layer: bandwidth.
        dict(name="rope_prompt_32k", op="rope", tokens=32768, hq=32, hk=8, d=128, rot=128, inter=False,
             scaling="llama3", base=500000.0, first=0, dtype="bf16"),
        # Interleaved pairs on half of each head, fp32, a chunk of odd length a million positions out.
        dict(name="rope_far_partial_fp32", op="rope", tokens=4097, hq=8, hk=8, d=64, rot=32, inter=True,
             scaling="linear", base=10000.0, first=1000003, dtype="fp32"),
        # Per-head norms before the rotation: one decode step of a batch of 64.
        dict(name="norm_rope_batch_64", op="norm_rope", tokens=64, hq=32, hk=8, d=128, rot=128, inter=False,
             scaling="none", base=1000000.0, first=4096, dtype="bf16"),
        # The same for a 16K prompt with YaRN frequencies, fp16.
        dict(name="norm_rope_prompt_16k", op="norm_rope", tokens=16384, hq=40, hk=8, d=128, rot=128, inter=False,
             scaling="yarn", base=10000.0, first=0, dtype="fp16"),
        # A decode step's append: one token for each of 64 sequences into 4-bit pages.
        dict(name="append_step_b64_aff4", op="append", batch=64, new=1, ragged=False, held=511, prefix=4096, hq=32,
             hk=8, d=128, rot=128, inter=False, scaling="llama3", base=500000.0, norm=False, page=64, fmt="aff4",
             group=64, dtype="bf16"),
        # Ragged prompts of a batch into fp16 pages of 16 rows.
        dict(name="append_ragged_b9_fp16", op="append", batch=9, new=1999, ragged=True, held=37, prefix=0, hq=16,
             hk=8, d=128, rot=64, inter=True, scaling="none", base=10000.0, norm=False, page=16, fmt="fp16", group=0,
             dtype="bf16"),
        # A 32K prompt, queries and keys normed and rotated, into 8-bit pages.
        dict(name="append_prompt_32k_aff8", op="append", batch=1, new=32768, ragged=False, held=0, prefix=0, hq=32,
             hk=8, d=128, rot=128, inter=False, scaling="none", base=1000000.0, norm=True, page=128, fmt="aff8",
             group=128, dtype="bf16"),
        # A small batch behind a short system prompt: latency.
        dict(name="attn_b4_prefix500_aff4", op="attn", batch=4, hq=32, hk=8, d=128, prefix=500, own_len=61, page=64,
             fmt="aff4", group=64, dtype="bf16"),
        # 64 requests about one 32K document, fp16 pages: the prefix is read and multiplied once for all.
        dict(name="attn_b64_prefix32k_fp16", op="attn", batch=64, hq=32, hk=8, d=128, prefix=32768, own_len=512,
             page=64, fmt="fp16", group=0, dtype="bf16"),
        # 120 samples from one 8K prompt, 4-bit pages, own parts up to 1K.
        dict(name="attn_b120_prefix8k_aff4", op="attn", batch=120, hq=40, hk=8, d=128, prefix=8191, own_len=1025,
             page=64, fmt="aff4", group=64, dtype="bf16"),
        # No prefix at all: 33 ragged sequences up to 16K, head_dim 64, 8-bit pages of 16 rows.
        dict(name="attn_b33_own16k_d64_aff8", op="attn", batch=33, hq=32, hk=8, d=64, prefix=0, own_len=16001,
             page=16, fmt="aff8", group=64, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "append", "attn"])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.randint(1, 8)
    d = rng.choice([64, 128])
    inter = rng.random() < 0.4
    rot = rng.choice([d, d, d // 2])
    scaling = rng.choice(sorted(SCALINGS))
    base = rng.choice([10000.0, 500000.0, 1000000.0])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["fp16", "aff8", "aff4"])
    group = 0 if fmt == "fp16" else rng.choice([32, 64, d])
    if op in ("rope", "norm_rope"):
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        row = (hq + hk) * d * (2 if dtype == "fp32" else 1)
        tokens = _log(rng, 1, min(32768, 32768 * 40 * 128 // row))
        return dict(op=op, tokens=tokens, hq=hq, hk=hk, d=d, rot=rot, inter=inter, scaling=scaling, base=base,
                    first=rng.choice([0, 1, 8191, 1000003]), dtype=dtype)
    if op == "append":
        batch = _log(rng, 1, 200)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 24000 * 40 // max(40, hq + 2 * hk) // batch))
        return dict(op=op, batch=batch, new=new, ragged=new > 1 and rng.random() < 0.6, held=rng.randint(0, 300),
                    prefix=rng.choice([0, 1000]), hq=hq, hk=hk, d=d, rot=rot, inter=inter, scaling=scaling,
                    base=base, norm=rng.random() < 0.5, page=page, fmt=fmt, group=group,
                    dtype=rng.choice(["bf16", "fp16"]))
    batch = _log(rng, 1, 128)
    prefix = 0 if rng.random() < 0.15 else _log(rng, 1, min(32768, 32768 * 64 * 32 * 128 // (batch * hq * d)))
    own_len = _log(rng, 1, max(1, min(16000, 60000 // batch)))
    return dict(op="attn", batch=batch, hq=hq, hk=hk, d=d, prefix=prefix, own_len=own_len, page=page, fmt=fmt,
                group=group, dtype=rng.choice(["bf16", "fp16"]))


# ------------------------------------------------------------------ lengths --

def _spread(n, most):
    """n lengths from 1 to `most`, evenly spread: their sum goes by the case alone."""
    return [most] if n == 1 else [1 + (most - 1) * i // (n - 1) for i in range(n)]


def _new_tokens(c):
    return _spread(c["batch"], c["new"]) if c["ragged"] else [c["new"]] * c["batch"]


def _groups(c):
    return 0 if c["fmt"] == "fp16" else c["d"] // c["group"]


def _row_bytes(c):
    return c["d"] * BITS[c["fmt"]] // 8


def work(c):
    if c["op"] in ("rope", "norm_rope"):
        size = 4 if c["dtype"] == "fp32" else 2
        rows = c["tokens"] * (c["hq"] + c["hk"])
        flops = rows * (3.0 * c["rot"] + (4.0 * c["d"] if c["op"] == "norm_rope" else 0.0))
        return {"bytes": 2.0 * rows * c["d"] * size + 4.0 * c["tokens"], "flops": flops}
    stored = _row_bytes(c) + 4 * _groups(c)
    if c["op"] == "append":
        size = 4 if c["dtype"] == "fp32" else 2
        t = sum(_new_tokens(c))
        row = c["d"] * size
        # q read and written, k and v read, stored, and what was stored written out
        moved = t * (2 * c["hq"] * row + 2 * c["hk"] * (2 * row + stored))
        return {"bytes": float(moved), "flops": t * ((c["hq"] + c["hk"]) * 3.0 * c["rot"] + 8.0 * c["hk"] * c["d"])}
    keys = sum(_spread(c["batch"], c["own_len"]))
    read = (c["prefix"] + keys) * 2 * c["hk"] * stored + 2 * c["batch"] * c["hq"] * c["d"] * 2
    return {"bytes": float(read), "flops": 4.0 * c["hq"] * c["d"] * (c["batch"] * c["prefix"] + keys)}


# ------------------------------------------------------------------- inputs --

def _frequencies(c):
    """(radians per position of each pair, factor on sines and cosines), in 64 bits."""
    rot, p = c["rot"], SCALINGS[c["scaling"]]
    freq, factor = [], 1.0
    for i in range(rot // 2):
        f = c["base"] ** (-2.0 * i / rot)
        if c["scaling"] == "linear":
            f /= p["factor"]
        elif c["scaling"] == "llama3":
            turns = p["original_max_position"] * f / (2.0 * math.pi)     # turns within the trained length
            lo, hi = p["low_freq_factor"], p["high_freq_factor"]
            keep = min(1.0, max(0.0, (turns - lo) / (hi - lo)))
            f = f * keep + f / p["factor"] * (1.0 - keep)
        elif c["scaling"] == "yarn":
            at = [rot * math.log(p["original_max_position"] / (b * 2.0 * math.pi)) / (2.0 * math.log(c["base"]))
                  for b in (p["beta_fast"], p["beta_slow"])]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = f * (1.0 - ramp) + f / p["factor"] * ramp
        freq.append(f)
    if c["scaling"] == "yarn":
        factor = 0.1 * math.log(p["factor"]) + 1.0
    return freq, factor


def _pool(c, pages, g):
    """A page pool of `pages` pages whose every row holds codes and metadata of normal values."""
    rows, rb, ng = (pages, c["hk"], c["page"]), _row_bytes(c), _groups(c)
    sizes, off = [], 256
    for n in (rb, 4 * ng, rb, 4 * ng):
        sizes.append((off, pages * c["hk"] * c["page"] * n))
        off = (off + pages * c["hk"] * c["page"] * n + 255) // 256 * 256
    buf = torch.zeros(off, dtype=torch.uint8, device="cuda")
    planes = {}
    for name, (o, n) in zip(("k_codes", "k_meta", "v_codes", "v_meta"), sizes):
        if not n:
            continue
        at = buf[o:o + n]
        if name.endswith("codes"):
            if c["fmt"] == "fp16":
                at = at.view(torch.float16).view(*rows, c["d"])
                at.normal_(generator=g)
            else:
                at = at.view(*rows, rb)
                at.random_(0, 256, generator=g)
        else:   # levels of a range of some five sigma, with ranges of keys spread wider
            at = at.view(torch.float16).view(*rows, ng, 2)
            width = torch.rand((*rows, ng), generator=g, device="cuda") * (2.0 if name[0] == "k" else 1.0) + 4.0
            at[..., 0] = width / (2 ** BITS[c["fmt"]] - 1)
            at[..., 1] = -0.5 * width
        planes[name] = at
    return buf, planes


def _tables(c, lens, g):
    """Pages of each sequence in a random order: (table of the sequences' own pages, the prefix's, pages)."""
    need = [(n + c["page"] - 1) // c["page"] for n in lens]
    shared = (c["prefix"] + c["page"] - 1) // c["page"]
    wide = max(1, max(need))
    order = torch.randperm(sum(need) + shared + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
    at = (torch.arange(wide, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None])
    table[at] = order[shared:shared + sum(need)]
    return table, order[:shared].clone(), sum(need) + shared + 1


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": dict(c)}
    if c["op"] != "attn":
        freq, factor = _frequencies(c)
        s["freq"], s["factor"] = torch.tensor(freq, dtype=torch.float64, device="cuda"), factor
        if c["op"] == "norm_rope" or c.get("norm"):
            s["q_norm"], s["k_norm"] = ((1.0 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dt)
                                        for _ in range(2))
    if c["op"] in ("rope", "norm_rope"):
        t, hq, hk, d = c["tokens"], c["hq"], c["hk"], c["d"]
        qkv = torch.randn((t, (hq + 2 * hk) * d), generator=g, device="cuda").to(dt)    # one projection's output
        s["q"], s["k"] = qkv[:, :hq * d].view(t, hq, d), qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["positions"] = (torch.arange(t, device="cuda") + c["first"]
                          + torch.randint(0, 64, (1,), generator=g, device="cuda")).to(torch.int32)
        s["q_out"], s["k_out"] = (torch.empty((t, h, d), dtype=dt, device="cuda") for h in (hq, hk))
    elif c["op"] == "append":
        hq, hk, d = c["hq"], c["hk"], c["d"]
        mix = torch.randperm(c["batch"], generator=g, device="cuda").tolist()
        new = [_new_tokens(c)[i] for i in mix]
        t = sum(new)
        lens = [c["held"] + n for n in new]
        s["page_table"], _, pages = _tables(c, lens, g)
        s["buf"], s["planes"] = _pool(c, pages, g)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["cu_tokens"] = None if c["new"] == 1 else torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        s["prefix_len"] = torch.tensor([c["prefix"]], dtype=torch.int32, device="cuda")
        qkv = torch.randn((t, (hq + 2 * hk) * d), generator=g, device="cuda")
        k = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        k += 2.0 * torch.randn((hk, d), generator=g, device="cuda")     # keys sit around a mean of their channel
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = (x.view(t, -1, d) for x in qkv.split((hq * d, hk * d, hk * d), dim=1))
        s["q_out"], s["k_out"], s["v_out"] = (torch.empty((t, h, d), dtype=dt, device="cuda") for h in (hq, hk, hk))
    else:
        mix = torch.randperm(c["batch"], generator=g, device="cuda").tolist()
        lens = [_spread(c["batch"], c["own_len"])[i] for i in mix]
        s["page_table"], s["prefix_pages"], pages = _tables(c, lens, g)
        s["buf"], s["planes"] = _pool(c, pages, g)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["prefix_len"] = torch.tensor([c["prefix"]], dtype=torch.int32, device="cuda")
        s["q"] = torch.randn((c["batch"], c["hq"], c["d"]), generator=g, device="cuda").to(dt)
        s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------- the plain forms --

def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, c, cos, sin):
    """x [T, H, D] in 32 bits, pairs of its first `rot` channels rotated; cos, sin [T, 1, rot / 2]."""
    y = x.clone()
    half = c["rot"] // 2
    a, b = (x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]) if c["inter"] else (x[..., :half], x[..., half:c["rot"]])
    first, second = a * cos - b * sin, b * cos + a * sin
    if c["inter"]:
        y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2] = first, second
    else:
        y[..., :half], y[..., half:c["rot"]] = first, second
    return y


def _plain_rows(s, positions):
    c = s["case"]
    angle = positions.double()[:, None, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()
    q, k = (_norm(s[n], s[n + "_norm"]) if n + "_norm" in s else s[n].float() for n in ("q", "k"))
    return _rotated(q, c, cos, sin), _rotated(k, c, cos, sin)


def _plain_quantised(x, c):
    """codes (as stored), metadata and the values they stand for, of rows x [T, H, D] in 32 bits."""
    levels = 2 ** BITS[c["fmt"]] - 1
    y = x.view(*x.shape[:-1], _groups(c), c["group"])
    zero = y.amin(-1, keepdim=True)
    # the definition's 32-bit quotient: torch would multiply by a rounded 1 / levels, which moves values at a border
    scale = ((y.amax(-1, keepdim=True) - zero).double() / levels).float().clamp_min(1e-5)
    u = ((y - zero) / scale).round().clamp(0, levels)
    s16, z16 = scale.half(), zero.half()
    hat = (u * s16.float() + z16.float()).view(x.shape)
    u = u.view(x.shape).to(torch.uint8)
    codes = u ^ 0x80 if levels == 255 else u[..., 0::2] | (u[..., 1::2] << 4)
    return codes, torch.cat((s16, z16), -1), hat


def _plain_append(s):
    c = s["case"]
    lens, cu = s["seq_lens"].long(), s["cu_tokens"]
    batch = lens.numel()
    count = torch.ones_like(lens) if cu is None else (cu[1:] - cu[:-1]).long()
    start = torch.arange(batch, device="cuda") if cu is None else cu[:-1].long()
    seq = torch.repeat_interleave(torch.arange(batch, device="cuda"), count, output_size=s["k"].shape[0])
    at = (lens - count)[seq] + torch.arange(s["k"].shape[0], device="cuda") - start[seq]
    q, k = _plain_rows(s, s["prefix_len"].long() + at)
    page, row = s["page_table"].long()[seq, at // c["page"]], at % c["page"]
    s["q_out"].copy_(q)
    for name, x in (("k", k), ("v", s["v"].float())):
        if c["fmt"] == "fp16":
            stored = x.half()
            s["planes"][name + "_codes"][page, :, row] = stored
            s[name + "_out"].copy_(stored)
        else:
            codes, meta, hat = _plain_quantised(x, c)
            s["planes"][name + "_codes"][page, :, row] = codes
            s["planes"][name + "_meta"][page, :, row] = meta
            s[name + "_out"].copy_(hat)


def _plain_values(s, name, pages):
    """Rows of `pages` [..., n] as [..., kv head, n * page, D] in 32 bits."""
    c = s["case"]
    x = s["planes"][name + "_codes"][pages]
    if c["fmt"] == "fp16":
        x = x.float()
    else:
        meta = s["planes"][name + "_meta"][pages].float()
        u = torch.stack((x & 15, x >> 4), -1).flatten(-2) if c["fmt"] == "aff4" else x ^ 0x80
        u = u.float().view(*u.shape[:-1], _groups(c), c["group"])
        x = (u * meta[..., 0:1] + meta[..., 1:2]).flatten(-2)
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_attention(s):
    c = s["case"]
    batch, hk, d = c["batch"], c["hk"], c["d"]
    g = c["hq"] // hk
    q = s["q"].float().view(batch, hk, g, d) * (d ** -0.5)
    table = s["page_table"].long().clamp_min(0)
    k, v = (_plain_values(s, n, table) for n in "kv")
    keys = torch.arange(k.shape[2], device="cuda")[None, None, None, :]
    score = (q @ k.transpose(-1, -2)).masked_fill(keys >= s["seq_lens"].view(-1, 1, 1, 1), -torch.inf)
    if c["prefix"]:
        pages = s["prefix_pages"].long()
        kp, vp = (_plain_values(s, n, pages)[:, :c["prefix"]] for n in "kv")
        rows = q.transpose(0, 1).reshape(hk, batch * g, d)
        shared = (rows @ kp.transpose(-1, -2)).view(hk, batch, g, -1).transpose(0, 1)
        top = torch.maximum(score.amax(-1, keepdim=True), shared.amax(-1, keepdim=True))
        p, pp = torch.exp(score - top), torch.exp(shared - top)
        both = (pp.transpose(0, 1).reshape(hk, batch * g, -1) @ vp).view(hk, batch, g, d).transpose(0, 1)
        out = (p @ v + both) / (p.sum(-1, keepdim=True) + pp.sum(-1, keepdim=True))
    else:
        p = torch.exp(score - score.amax(-1, keepdim=True))
        out = (p @ v) / p.sum(-1, keepdim=True)
    s["out"].copy_(out.reshape(batch, c["hq"], d))


# ------------------------------------------------------ the package's calls --

def _own_objects(s):
    """The rotation's table and the cache's handle, as a program makes them once."""
    import bit_kv_cache_quant_gb300 as kvq

    c = s["case"]
    if c["op"] != "attn":
        kind = c["scaling"]
        s["rope"] = kvq.Rope(c["rot"], c["base"], interleaved=c["inter"], scaling=kind, **SCALINGS[kind])
    if c["op"] in ("append", "attn"):
        fmt = ("fp16", 16, 0) if c["fmt"] == "fp16" else ("affine_token", BITS[c["fmt"]], c["group"])
        pages = s["planes"]["k_codes"].shape[0]
        s["cache"] = kvq.PagedKVCache(c["hk"], c["d"], c["page"], pages, *fmt, *fmt, buf=s["buf"])
    s["kvq"] = kvq


def _own_run(s):
    if "kvq" not in s:
        _own_objects(s)
    op = s["case"]["op"]
    if op in ("rope", "norm_rope"):
        s["kvq"].rope_qk(s["q"], s["k"], s["positions"], s["rope"], q_out=s["q_out"], k_out=s["k_out"],
                         q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS)
    elif op == "append":
        s["cache"].append(s["k"], s["v"], s["page_table"], s["seq_lens"], cu_tokens=s["cu_tokens"], q=s["q"],
                          rope=s["rope"], prefix_len=s["prefix_len"], q_out=s["q_out"], k_out=s["k_out"],
                          v_out=s["v_out"], q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS)
    else:
        s["cache"].decode_attn(s["q"], s["page_table"], s["seq_lens"], prefix_pages=s["prefix_pages"],
                               prefix_len=s["prefix_len"], out=s["out"])


def run(state):
    s = state
    c = s["case"]
    if own:
        _own_run(s)
    elif c["op"] in ("rope", "norm_rope"):
        q, k = _plain_rows(s, s["positions"])
        s["q_out"].copy_(q)
        s["k_out"].copy_(k)
    elif c["op"] == "append":
        _plain_append(s)
    else:
        _plain_attention(s)
    if c["op"] == "attn":
        return {"out": s["out"]}
    if c["op"] != "append":
        return {"q": s["q_out"], "k": s["k_out"]}
    # the pool where it holds values as they are; else its metadata, and the values of the new rows
    planes = ("k_codes", "v_codes") if c["fmt"] == "fp16" else ("k_meta", "v_meta")
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], **{n: s["planes"][n] for n in planes}}


# -------------------------------------------------- the definition, 64 bits --

def _exact_turned(c, x, weight, positions):
    """Row by row: mean square, weight, then each pair as a complex number times a power of the unit circle."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS) * weight.double()
    freq, factor = _frequencies(c)
    angle = torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    unit = torch.polar(torch.full_like(angle, factor), angle)[:, None, :]
    turn, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["inter"]:
        z = torch.view_as_complex(turn.reshape(*turn.shape[:-1], -1, 2).contiguous()) * unit
        turn = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(*[t.contiguous() for t in turn.chunk(2, -1)]) * unit
        turn = torch.cat((z.real, z.imag), -1)
    return torch.cat((turn, rest), -1)


def _exact_rows(c, plane, meta, pages):
    """The rows of `pages` [n] one page after another, as [kv head, n * page, D]."""
    raw = plane.index_select(0, pages)
    if c["fmt"] == "fp16":
        vals = raw.double()
    else:
        n = c["d"]
        u = torch.empty((*raw.shape[:-1], n), dtype=torch.float64, device="cuda")
        if c["fmt"] == "aff4":
            u[..., 0::2], u[..., 1::2] = (raw % 16).double(), torch.div(raw, 16, rounding_mode="floor").double()
        else:
            u.copy_((raw.to(torch.int32) + 128) % 256)
        m = meta.index_select(0, pages).double().repeat_interleave(c["group"], dim=-2)
        vals = u * m[..., 0] + m[..., 1]
    return vals.permute(1, 0, 2, 3).reshape(c["hk"], -1, c["d"])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("rope", "norm_rope"):
        return {n: _exact_turned(c, s[n], s.get(n + "_norm"), s["positions"]) for n in ("q", "k")}
    if c["op"] == "append":
        lens = s["seq_lens"].tolist()
        new = [1] * c["batch"] if s["cu_tokens"] is None else s["cu_tokens"].diff().tolist()
        seq = [b for b, n in enumerate(new) for _ in range(n)]
        at = [lens[b] - n + j for b, n in enumerate(new) for j in range(n)]
        seq, at = torch.tensor(seq, device="cuda"), torch.tensor(at, device="cuda")
        pos = at + c["prefix"]
        page = s["page_table"][seq, torch.div(at, c["page"], rounding_mode="floor")].long()
        row = at.remainder(c["page"])
        out = {"q": _exact_turned(c, s["q"], s.get("q_norm"), pos)}
        for n in "kv":
            x = _exact_turned(c, s["k"], s.get("k_norm"), pos) if n == "k" else s["v"].double()
            if c["fmt"] == "fp16":
                plane = s["planes"][n + "_codes"].double()
                plane[page, :, row] = x
                out[n], out[n + "_codes"] = x, plane
                continue
            # the formats code 32-bit values with a 32-bit scale and quotient: 64-bit results rounded to those
            r32 = lambda t: t.float().double()  # noqa: E731
            lv = 2 ** BITS[c["fmt"]] - 1
            parts = r32(x).split(c["group"], dim=-1)
            lo = torch.stack([p.min(-1).values for p in parts], -1)
            step = r32(r32(torch.stack([p.max(-1).values for p in parts], -1) - lo) / lv)
            step = step.clamp_min(float(torch.tensor(1e-5)))
            wide = [t.repeat_interleave(c["group"], -1) for t in (lo, step, lo.half().double(), step.half().double())]
            out[n] = torch.round(r32(r32(r32(x) - wide[0]) / wide[1])).clamp(0, lv) * wide[3] + wide[2]
            plane = s["planes"][n + "_meta"].double()
            plane[page, :, row] = torch.stack((step, lo), -1)
            out[n + "_meta"] = plane
        return out
    g, page = c["hq"] // c["hk"], c["page"]
    q, lens = s["q"].double(), s["seq_lens"].tolist()
    kv = [(s["planes"][n + "_codes"], s["planes"].get(n + "_meta")) for n in "kv"]
    shared = None
    if c["prefix"]:
        shared = [_exact_rows(c, *p, s["prefix_pages"].long())[:, :c["prefix"]] for p in kv]
    out = torch.empty_like(q)
    for b, n in enumerate(lens):
        mine = [_exact_rows(c, *p, s["page_table"][b, :(n + page - 1) // page].long())[:, :n] for p in kv]
        k, v = mine if shared is None else [torch.cat(x, 1) for x in zip(shared, mine)]
        rows = q[b].view(c["hk"], g, c["d"])
        w = torch.softmax(torch.bmm(rows, k.transpose(1, 2)) / math.sqrt(c["d"]), -1)
        out[b] = torch.bmm(w, v).view(c["hq"], c["d"])
    return {"out": out}
