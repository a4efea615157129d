"""The 8-bit paged KV cache's operators, and the append with the rotary embedding, as cases to measure.

Four operators of the decoder's attention path over a paged cache (pages of 16 tokens):

* ``append_rope``: the key and value rows of a step's new tokens into the bf16 pools, keys (and the step's query rows)
  normalised per head where the decoder does that, and rotated at their positions on the way.
* ``append_rope_fp8``: the same into pools of e4m3 values with one power-of-two scale (e8m0) per row and KV head.
* ``decode_attn_fp8``: attention of one new token per request over the 8-bit cache.
* ``expand_fp8``: pages of the 8-bit cache, by block table, as bf16 pages that chunked prefill reads.

Where ``own`` is false, ``run`` computes them in their plain form from elementary torch operations; where it is true, it
calls the library.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -80, 100  # range of a row's power-of-two scale
THETA = 1.0e6
EPS = 1.0e-6
NORM_SPREAD = 0.1  # spread of the norm weights around 1
CHANNEL_SPREAD = 0.5  # spread of the log of a channel's size: projections' channels differ in size


def listed():
    return [
        # one decode step of 16 requests: a token each, at the ends of contexts of 300 to 3000 tokens
        dict(name="append_step_bs16", op="append_rope", hq=16, hkv=8, d=128, tokens=16, prefix=3000, norm=True),
        # one chunk of a long prompt, straight behind 8192 cached tokens
        dict(name="append_chunk_4096", op="append_rope", hq=16, hkv=8, d=128, tokens=4096, prefix=8192, norm=True),
        # a ragged last chunk of another backbone, without norms
        dict(name="append_ragged_32q8kv", op="append_rope", hq=32, hkv=8, d=128, tokens=1777, prefix=4096, norm=False),
        # the same steps into the 8-bit cache
        dict(name="append_fp8_step_bs16", op="append_rope_fp8", hq=16, hkv=8, d=128, tokens=16, prefix=3000, norm=True),
        dict(name="append_fp8_chunk_4096", op="append_rope_fp8", hq=16, hkv=8, d=128, tokens=4096, prefix=8192, norm=True),
        # two requests of 37 and 200 tokens: the smallest step, bound by latency
        dict(name="decode_fp8_tiny", op="decode_attn_fp8", hq=16, hkv=8, d=128, batch=2, low=37, high=200, pad=0),
        # 16 concurrent clips with their prompts
        dict(name="decode_fp8_bs16", op="decode_attn_fp8", hq=16, hkv=8, d=128, batch=16, low=300, high=3000, pad=0),
        # one meeting of 38 minutes
        dict(name="decode_fp8_40k", op="decode_attn_fp8", hq=16, hkv=8, d=128, batch=1, low=40000, high=40000, pad=0),
        # 27 live requests in a bucket of 32, four query heads to a KV head, lengths far apart
        dict(name="decode_fp8_bs32_32q8kv", op="decode_attn_fp8", hq=32, hkv=8, d=128, batch=27, low=9, high=8000, pad=5),
        # small heads
        dict(name="decode_fp8_bs16_d64", op="decode_attn_fp8", hq=16, hkv=4, d=64, batch=16, low=300, high=3000, pad=0),
        # the cached prefix of one long prompt before its next chunk
        dict(name="expand_fp8_32k", op="expand_fp8", hq=16, hkv=8, d=128, batch=1, low=32768 + 4096, high=32768 + 4096, pad=0),
        # prefixes of several short prompts, ending inside their pages
        dict(name="expand_fp8_ragged", op="expand_fp8", hq=16, hkv=8, d=64, batch=6, low=100, high=2000, pad=1),
    ]


HEADS = [(16, 8, 128), (32, 8, 128), (64, 8, 128), (28, 4, 128), (40, 8, 128), (12, 4, 128), (16, 4, 64), (12, 2, 64), (8, 1, 64), (32, 32, 64)]
MOST_BYTES = 220e6  # a drawn case moves no more than the largest listed one


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append_rope", "append_rope_fp8", "decode_attn_fp8", "expand_fp8"])
    hq, hkv, d = rng.choice(HEADS)
    case = dict(op=op, hq=hq, hkv=hkv, d=d)
    if op.startswith("append"):
        case.update(tokens=_log_uniform(rng, 1, 6000), prefix=_log_uniform(rng, 1, 20000), norm=rng.random() < 0.5)
        while work(case)["bytes"] > MOST_BYTES:
            case["tokens"] = 1 + case["tokens"] // 2
        return case
    batch = _log_uniform(rng, 1, 40)
    high = _log_uniform(rng, 16, 60000)
    case.update(batch=batch, low=max(1, int(high * rng.uniform(0.05, 1.0))), high=high, pad=rng.choice([0, 0, 1, 3]))
    # the plain forms lay every request out at the longest one's length: bound that product
    while batch * case["high"] * hkv * d * 6 > MOST_BYTES:
        case["high"], case["low"] = 1 + case["high"] // 2, 1 + case["low"] // 2
    return case


def _lens(case):
    """The requests' lengths: spread over [low, high], its ends among them; padding rows of length 0 last."""
    n, low, high = case["batch"], case["low"], case["high"]
    r = np.random.default_rng(n * 1000003 + low * 1009 + high).integers(low, high, size=n, endpoint=True)
    r[0] = high
    r[-1] = low if n > 1 else high
    return np.concatenate([r, np.zeros(case["pad"], dtype=r.dtype)]).astype(np.int32)


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"].startswith("append"):
        t = case["tokens"]
        row_out = hkv * d * 2 if case["op"] == "append_rope" else hkv * (d + 1)
        # q and k and v read, q and k and v written, positions and slots, a table row per token
        moved = t * (2 * hq * d * 2 + 2 * hkv * d * 2 + 2 * row_out + 8) + t * d * 4
        return {"bytes": moved, "flops": t * (hq + hkv) * d * (8 if case["norm"] else 4)}
    total = int(_lens(case).sum())
    cache = 2 * total * hkv * (d + 1)
    if case["op"] == "decode_attn_fp8":
        rows = case["batch"] + case["pad"]
        return {"bytes": cache + 2 * rows * hq * d * 2 + 4 * (total // PAGE + 2 * rows), "flops": 4 * total * hq * d}
    return {"bytes": cache + 2 * total * hkv * d * 2, "flops": 2 * total * hkv * d}


# ------------------------------------------------------------------------------------------------ inputs
def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _table(max_pos, d):
    """cos and sin of position times theta^(-2i/d), in 64 bits, rounded once."""
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * THETA ** (
        -torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32).contiguous()


def _workspace(case, rows):
    """The workspace that a user's program keeps beside its cache (the library's calls take one; the plain form none)."""
    if own:
        import paged_kv_decode_gb300 as pkv

        if case["op"] == "decode_attn_fp8":
            return pkv.Workspace(pkv.decode_workspace_bytes(rows, -(-case["high"] // PAGE), 1, case["hq"], case["hkv"], case["d"]))
        return pkv.Workspace(pkv.PKV_STATUS_BYTES)
    return None


def _pages(rng, lens, spare):
    """A block table of pages in random order, `spare` of them left over."""
    need = -(-lens // PAGE)
    width = max(1, int(need.max()))
    order = rng.permutation(int(need.sum()) + spare)
    table = np.full((len(lens), width), order[-1], dtype=np.int32)
    table[np.arange(width)[None, :] < need[:, None]] = order[: int(need.sum())]
    return torch.from_numpy(table).cuda(), len(order)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = dict(case=dict(case))
    if case["op"].startswith("append"):
        t, prefix = case["tokens"], case["prefix"]
        # rows of one fused projection: q, k and v of a token side by side, channels of different size
        channel = torch.exp(CHANNEL_SPREAD * _normal(((hq + 2 * hkv) * d,), gen, torch.float32))
        s["qkv"] = (_normal((t, (hq + 2 * hkv) * d), gen, torch.float32) * channel).to(torch.bfloat16)
        s["q"] = s["qkv"][:, : hq * d].view(t, hq, d)
        s["k_new"] = s["qkv"][:, hq * d: (hq + hkv) * d].view(t, hkv, d)
        s["v_new"] = s["qkv"][:, (hq + hkv) * d:].view(t, hkv, d)
        if t <= 64:  # one token for each of t requests
            lens = rng.integers(max(1, prefix // 10), prefix + 1, size=t).astype(np.int64)
            positions = lens - 1
            pages = rng.permutation(4 * t + 64)[:t]
            slots = pages * PAGE + positions % PAGE
            num_pages = 4 * t + 64
        else:  # one request's chunk behind its prefix
            positions = prefix + np.arange(t, dtype=np.int64)
            first = prefix // PAGE
            num_pages = (prefix + t) // PAGE - first + 1 + 64
            slots = rng.permutation(num_pages)[positions // PAGE - first] * PAGE + positions % PAGE
        s["positions"] = torch.from_numpy(positions.astype(np.int32)).cuda()
        s["slots"] = torch.from_numpy(slots.astype(np.int32)).cuda()
        s["cos_sin"] = _table(int(positions.max()) + 1, d)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1 + NORM_SPREAD * _normal((d,), gen, torch.float32)).to(torch.bfloat16)
            s["k_weight"] = (1 + NORM_SPREAD * _normal((d,), gen, torch.float32)).to(torch.bfloat16)
        shape = (num_pages, hkv, PAGE, d)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda")
        s["k_pages"], s["v_pages"] = _normal(shape, gen), _normal(shape, gen)
        if case["op"] == "append_rope_fp8":
            s["k_pages"], k_exp = _quantise(s["k_pages"].float())
            s["v_pages"], v_exp = _quantise(s["v_pages"].float())
            s["kv_scales"] = torch.stack([k_exp, v_exp], dim=2).contiguous().view(torch.float8_e8m0fnu)
        s["workspace"] = _workspace(case, t)
        return s
    lens = _lens(case)
    s["block_table"], num_pages = _pages(rng, lens, 3)
    s["seq_lens"] = torch.from_numpy(lens).cuda()
    shape = (num_pages, hkv, PAGE, d)
    channel = torch.exp(CHANNEL_SPREAD * _normal((hkv, 1, d), gen, torch.float32))
    s["k_pages"], k_exp = _quantise(_normal(shape, gen, torch.float32) * channel)
    s["v_pages"], v_exp = _quantise(_normal(shape, gen, torch.float32))
    s["kv_scales"] = torch.stack([k_exp, v_exp], dim=2).contiguous().view(torch.float8_e8m0fnu)
    if case["op"] == "decode_attn_fp8":
        s["q"] = _normal((len(lens), hq, d), gen)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = d ** -0.5
    else:
        # a staging pool of the requests' own pages, in order
        width = s["block_table"].shape[1]
        s["out_table"] = torch.arange(len(lens) * width, dtype=torch.int32, device="cuda").view(len(lens), width)
        s["k_out"] = torch.zeros((len(lens) * width, hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    s["workspace"] = _workspace(case, len(lens))
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _quantise(x):
    """fp32 rows as e4m3 values times a power of two each: the least 2^e with max|x| <= 448 * 2^e."""
    most = x.abs().amax(dim=-1).double()
    m, e = torch.frexp(most / E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e).clamp(EXP_MIN, EXP_MAX)
    e = torch.where(most == 0, torch.full_like(e, EXP_MIN), e)
    y = (x * ((127 - e.int()) << 23).view(torch.float32)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)  # times 2^-e, exactly
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _norm_rotate(x, weight, cos, sin):
    """RMS norm of each head's row (where there is a weight), then the rotation of the pairs (i, i + d/2)."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    a, b = x.chunk(2, dim=-1)
    # 64 bits: values next to a border between two e4m3 steps
    a, b, c, s = a.double(), b.double(), cos.double()[:, None], sin.double()[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1).float()


def _plain_append(s):
    cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, dim=-1)
    q = _norm_rotate(s["q"], s["q_weight"], cos, sin)
    k = _norm_rotate(s["k_new"], s["k_weight"], cos, sin)
    s["q_out"].copy_(q)
    page, slot = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    if s["case"]["op"] == "append_rope":
        s["k_pages"][page, :, slot] = k.to(torch.bfloat16)
        s["v_pages"][page, :, slot] = s["v_new"]
        return
    k8, k_exp = _quantise(k)
    v8, v_exp = _quantise(s["v_new"].float())
    as_bytes = lambda x: x.view(torch.uint8)  # noqa: E731
    as_bytes(s["k_pages"])[page, :, slot] = as_bytes(k8)
    as_bytes(s["v_pages"])[page, :, slot] = as_bytes(v8)
    as_bytes(s["kv_scales"])[page, :, 0, slot] = k_exp
    as_bytes(s["kv_scales"])[page, :, 1, slot] = v_exp


def _rows(s, which, dtype=torch.float32):
    """The cached rows of every request in order, as the values they stand for: [batch, hkv, width * 16, d]."""
    table = s["block_table"].long()
    pool = s["k_pages" if which == 0 else "v_pages"]
    x = pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).to(dtype)
    e = s["kv_scales"].view(torch.uint8)[table][:, :, :, which].to(dtype) - 127
    x = x * torch.exp2(e)[..., None]
    b, w, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, w * p, d)


def _plain_decode(s):
    k, v = _rows(s, 0), _rows(s, 1)
    b, h, n, d = k.shape
    q = s["q"].float().view(b, h, -1, d)
    live = torch.arange(n, device="cuda")[None, :] < s["seq_lens"][:, None]
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    score = score.masked_fill(~live[:, None, None], -math.inf)
    most = score.amax(dim=-1, keepdim=True).clamp(min=-1e30)  # a request of length 0 has none
    p = torch.exp(score - most)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v.masked_fill(~live[:, None, :, None], 0.0)) / total.clamp(min=1e-30)
    s["out"].copy_(o.reshape(s["out"].shape))


def _plain_expand(s):
    b, w = s["block_table"].shape
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    live = torch.arange(w * PAGE, device="cuda")[None, :] < s["seq_lens"][:, None]
    live = live.view(b * w, 1, PAGE, 1)
    at = s["out_table"].view(-1).long()
    for_page = lambda x: x.view(b, hkv, w, PAGE, d).transpose(1, 2).reshape(b * w, hkv, PAGE, d)  # noqa: E731
    s["k_out"][at] = torch.where(live, for_page(_rows(s, 0)).to(torch.bfloat16), s["k_out"][at])
    s["v_out"][at] = torch.where(live, for_page(_rows(s, 1)).to(torch.bfloat16), s["v_out"][at])


def _outputs(s):
    op = s["case"]["op"]
    if op == "decode_attn_fp8":
        return {"out": s["out"]}
    if op == "expand_fp8":
        return {"k_out": s["k_out"], "v_out": s["v_out"]}
    # pools of 8 bits carry the types of the values that they stand for
    return {n: s[n] for n in ("q_out", "k_pages", "v_pages", "kv_scales") if n in s}


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import paged_kv_decode_gb300 as pkv

        if op == "append_rope":
            pkv.append_rope(s["k_new"], s["v_new"], s["positions"], s["slots"], s["cos_sin"], s["k_pages"], s["v_pages"],
                            s["workspace"], q=s["q"], q_out=s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        elif op == "append_rope_fp8":
            pkv.append_rope_fp8(s["k_new"], s["v_new"], s["positions"], s["slots"], s["cos_sin"], s["k_pages"], s["v_pages"],
                                s["kv_scales"], s["workspace"], q=s["q"], q_out=s["q_out"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=EPS)
        elif op == "decode_attn_fp8":
            pkv.decode_attn_fp8(s["q"], s["k_pages"], s["v_pages"], s["kv_scales"], s["block_table"], s["seq_lens"], s["out"],
                                s["scale"], s["workspace"])
        else:
            pkv.expand_fp8(s["k_pages"], s["v_pages"], s["kv_scales"], s["block_table"], s["seq_lens"], s["k_out"], s["v_out"],
                           s["out_table"], s["workspace"])
    elif op.startswith("append"):
        _plain_append(s)
    elif op == "decode_attn_fp8":
        _plain_decode(s)
    else:
        _plain_expand(s)
    return _outputs(s)


# ------------------------------------------------------------------------------------------------ in 64 bits
def _value(bytes8):
    """What the e4m3 codes 0..255 stand for, from the format's definition (7 exponent bias, no infinities)."""
    code = torch.arange(256, dtype=torch.float64, device="cuda")
    low, sign = code % 128, torch.where(code >= 128, -1.0, 1.0)
    e, m = torch.div(low, 8, rounding_mode="floor"), low % 8
    v = torch.where(e > 0, (1 + m / 8) * _power(e - 7), m / 8 * 2.0 ** -6)
    v = torch.where(low == 127, torch.full_like(v, math.nan), v) * sign
    return v[bytes8.long()]


def _power(e):
    """2^e in 64 bits, exactly, for whole numbers e."""
    return torch.from_numpy(np.ldexp(1.0, np.arange(-200, 201))).cuda()[e.long() + 200]


def _nearest8(x):
    """(the nearest e4m3 value, ties to even, of each row over its power of two; that power), in 64 bits."""
    most = x.abs().amax(dim=-1, keepdim=True)
    ladder = _power(torch.arange(EXP_MIN, EXP_MAX + 1, device="cuda"))
    at = torch.searchsorted(ladder * E4M3_MAX, most.contiguous()).clamp(max=len(ladder) - 1)
    power = ladder[at]
    y = x / power
    step = _power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX), power[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    d, op = case["d"], case["op"]
    if op.startswith("append"):
        p = s["positions"].double()[:, None]
        i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), p * THETA ** (-2 * i / d))[:, None]

        def rotated(x, weight):
            x = x.double()
            if weight is not None:
                x = x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt() * weight.double()
            z = torch.complex(x[..., : d // 2], x[..., d // 2:]) * turn
            return torch.cat([z.real, z.imag], -1)

        r = {"q_out": rotated(s["q"], s["q_weight"])}
        k, v = rotated(s["k_new"], s["k_weight"]), s["v_new"].double()
        at = s["slots"].long()

        def put(pool, rows):  # rows [tokens, hkv, ...] at their slots of [pages, hkv, 16, ...]
            flat = pool.transpose(1, 2).contiguous()
            flat.view(-1, *flat.shape[2:])[at] = rows
            return flat.transpose(1, 2).contiguous()

        if op == "append_rope":
            r["k_pages"], r["v_pages"] = put(s["k_pages"].double(), k), put(s["v_pages"].double(), v)
            return r
        (k, ks), (v, vs) = _nearest8(k), _nearest8(v)
        r["k_pages"] = put(_value(s["k_pages"].view(torch.uint8)), k)
        r["v_pages"] = put(_value(s["v_pages"].view(torch.uint8)), v)
        old = _power(s["kv_scales"].view(torch.uint8).int() - 127)
        r["kv_scales"] = torch.stack([put(old[:, :, 0], ks), put(old[:, :, 1], vs)], 2)
        return r

    lens = s["seq_lens"].tolist()
    hkv, scales = case["hkv"], s["kv_scales"].view(torch.uint8)

    def rows(b, pool, which):  # [hkv, length, d] of one request
        n = lens[b]
        page = s["block_table"][b, : -(-n // PAGE)].long()
        x = _value(pool.view(torch.uint8)[page]) * _power(scales[page][:, :, which].int() - 127)[..., None]
        return x.transpose(0, 1).reshape(hkv, -1, d)[:, :n]

    if op == "decode_attn_fp8":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        group = case["hq"] // hkv
        for b, n in enumerate(lens):
            if n:
                k, v = rows(b, s["k_pages"], 0), rows(b, s["v_pages"], 1)
                q = s["q"][b].double().view(hkv, group, d)
                p = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k) * s["scale"], -1)
                out[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(-1, d)
        return {"out": out}
    k_out, v_out = s["k_out"].double(), s["v_out"].double()
    for b, n in enumerate(lens):
        for pool, to, which in ((s["k_pages"], k_out, 0), (s["v_pages"], v_out, 1)):
            x = rows(b, pool, which).transpose(0, 1)  # [length, hkv, d]
            at = s["out_table"][b].long().repeat_interleave(PAGE)[:n]
            to[at, :, torch.arange(n, device="cuda") % PAGE] = x
    return {"k_out": k_out, "v_out": v_out}
