"""Speculative decoding over the paged KV cache, and forks of its pages, as cases to measure.

Three operators of the decoder's attention path over a paged cache (pages of 16 tokens), each on the bf16 cache and on the
8-bit one (e4m3 values, one power-of-two scale per row and KV head):

* ``tree_attn``: attention of a request's drafted tokens, the nodes of a tree (or of a chain), over its cached prefix and
  over the nodes that each one descends from. The nodes' rows lie in the cache, straight behind the prefix.
* ``keep_nodes``: once the drafts are verified, the rows of the accepted path's nodes move up to consecutive positions
  behind the prefix, in the pools of all layers.
* ``copy_pages``: whole pages to other pages of the pools of all layers: the pages that a forked request may not share.

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
MAX_NODES = 64
CHANNEL_SPREAD = 0.5  # spread of the log of a channel's size: projections' channels differ in size
SPARE = 3  # pages of a pool that no request has


def listed():
    return [
        # two requests of 37 and 200 tokens with four drafted tokens in a row: the smallest step, bound by latency
        dict(name="tree_tiny_chain", op="tree_attn", fp8=False, hq=16, hkv=8, d=128, batch=2, low=37, high=200, pad=0,
             few=4, most=4, chain=True),
        # 16 concurrent clips with their prompts, a tree of 16 nodes each
        dict(name="tree_bs16", op="tree_attn", fp8=False, hq=16, hkv=8, d=128, batch=16, low=300, high=3000, pad=0,
             few=16, most=16, chain=False),
        # one meeting of 38 minutes, a wide tree
        dict(name="tree_40k", op="tree_attn", fp8=False, hq=16, hkv=8, d=128, batch=1, low=40000, high=40000, pad=0,
             few=32, most=32, chain=False),
        # 27 live requests in a bucket of 32, four query heads to a KV head, lengths and trees far apart
        dict(name="tree_bs32_32q8kv", op="tree_attn", fp8=False, hq=32, hkv=8, d=128, batch=27, low=9, high=8000, pad=5,
             few=1, most=64, chain=False),
        # the 16 clips from the 8-bit cache
        dict(name="tree_fp8_bs16", op="tree_attn", fp8=True, hq=16, hkv=8, d=128, batch=16, low=300, high=3000, pad=0,
             few=16, most=16, chain=False),
        # the meeting from the 8-bit cache, eight drafted tokens in a row, small heads
        dict(name="tree_fp8_40k_d64", op="tree_attn", fp8=True, hq=16, hkv=4, d=64, batch=1, low=40000, high=40000, pad=0,
             few=8, most=8, chain=True),
        # what 16 clips keep of their trees, in the 28 layers of the decoder
        dict(name="keep_bs16", op="keep_nodes", fp8=False, hkv=8, d=128, layers=28, batch=16, high=3000, pad=0,
             most=16, depth=6),
        # 43 requests in a bucket of 48, deep trees, 8-bit cache
        dict(name="keep_fp8_bs48", op="keep_nodes", fp8=True, hkv=8, d=128, layers=28, batch=43, high=8000, pad=5,
             most=64, depth=16),
        # the last page of one request's prompt for its companion, in one layer
        dict(name="copy_one_page", op="copy_pages", fp8=False, hkv=8, d=128, layers=1, pages=1, pad=0),
        # the last pages of 16 prompts for their companions, in a bucket of 20, 8-bit cache
        dict(name="copy_fp8_bs16", op="copy_pages", fp8=True, hkv=8, d=128, layers=28, pages=16, pad=4),
        # a context of 4096 tokens for a request that goes its own way
        dict(name="copy_4096_tokens", op="copy_pages", fp8=False, hkv=8, d=128, layers=28, pages=256, pad=0),
    ]


HEADS = [(16, 8, 128), (32, 8, 128), (64, 8, 128), (28, 4, 128), (40, 8, 128), (12, 4, 128), (16, 4, 64), (12, 2, 64), (8, 1, 64), (32, 32, 64)]
MOST_BYTES = 220e6  # a drawn case moves no more than the largest listed one of attention
MOST_FLOPS = 200e9  # ... and multiplies no more


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["tree_attn", "tree_attn", "keep_nodes", "copy_pages"])
    hq, hkv, d = rng.choice(HEADS)
    case = dict(op=op, fp8=rng.random() < 0.4, hkv=hkv, d=d)
    if op == "copy_pages":
        case.update(layers=_log_uniform(rng, 1, 40), pages=_log_uniform(rng, 1, 300), pad=rng.choice([0, 0, 1, 3]))
        while work(case)["bytes"] > 4 * MOST_BYTES:
            case["pages"] = 1 + case["pages"] // 2
        return case
    most = _log_uniform(rng, 2 if op == "keep_nodes" else 1, MAX_NODES)
    if op == "keep_nodes":
        case.update(layers=_log_uniform(rng, 1, 40), batch=_log_uniform(rng, 1, 64), high=_log_uniform(rng, 16, 60000),
                    pad=rng.choice([0, 0, 1, 3]), most=most, depth=rng.randint(2, most))
        while case["layers"] * case["batch"] * hkv * d > 4e6:
            case["batch"] = 1 + case["batch"] // 2
        return case
    batch = _log_uniform(rng, 1, 40)
    high = _log_uniform(rng, 16, 60000)
    case.update(hq=hq, batch=batch, low=int(high * rng.choice([0.0, rng.uniform(0.05, 1.0)])), high=high,
                pad=rng.choice([0, 0, 1, 3]), few=rng.randint(1, most), most=most, chain=rng.random() < 0.3)
    # the plain forms lay every request out at the longest one's length: bound that product
    while batch * case["high"] * hkv * d * 6 > MOST_BYTES or batch * case["high"] * hq * d * 4 * most > MOST_FLOPS:
        case["high"], case["low"] = 1 + case["high"] // 2, case["low"] // 2
    return case


def _rng(case, salt):
    """The shape of a case's work goes by the case alone, its values by the seed."""
    return np.random.default_rng([salt, case["batch"], case["high"], case["most"]])


def _lens(case):
    """The requests' cached prefixes: spread over [low, high], its ends among them; padding rows last."""
    n, low, high = case["batch"], case["low"], case["high"]
    r = _rng(case, low).integers(low, high, size=n, endpoint=True)
    r[0] = high
    r[-1] = low if n > 1 else high
    return np.concatenate([r, np.zeros(case["pad"], dtype=r.dtype)]).astype(np.int32)


def _nodes(case):
    """The requests' numbers of nodes, likewise; padding rows have none."""
    n, few, most = case["batch"], case["few"], case["most"]
    r = _rng(case, 7).integers(few, most, size=n, endpoint=True)
    r[0] = most
    r[-1] = few if n > 1 else most
    return np.concatenate([r, np.zeros(case["pad"], dtype=r.dtype)]).astype(np.int32)


def _paths(case):
    """The accepted paths [rows, depth], -1 behind each one's end: the root, then nodes with rising numbers."""
    rng, rows, depth = _rng(case, case["depth"]), case["batch"] + case["pad"], case["depth"]
    order = np.argsort(rng.random((rows, case["most"] - 1)), axis=1)[:, : depth - 1] + 1
    n = np.where(np.arange(rows) < case["batch"], rng.integers(1, depth, size=rows, endpoint=True), 0)
    inside = np.arange(depth)[None, :] < n[:, None]
    # of the nodes drawn the first n - 1, in rising order
    order = np.sort(np.where(inside[:, 1:], order, case["most"]), axis=1)
    path = np.concatenate([np.zeros((rows, 1), dtype=order.dtype), order], axis=1)
    return np.where(inside, path, -1).astype(np.int32), n.astype(np.int32)


def work(case):
    hkv, d = case["hkv"], case["d"]
    row = hkv * (d + 1) if case["fp8"] else hkv * d * 2  # of K or of V, with its scale bytes
    if case["op"] == "copy_pages":
        return {"bytes": 4 * case["layers"] * case["pages"] * PAGE * row, "flops": 0}
    if case["op"] == "keep_nodes":
        path, n = _paths(case)
        moved = int(((path >= 0) & (path != np.arange(path.shape[1])[None, :])).sum())
        return {"bytes": 4 * case["layers"] * moved * row + 4 * (int(n.sum()) + 2 * len(n)), "flops": 0}
    nodes, lens, hq = _nodes(case).astype(np.int64), _lens(case).astype(np.int64), case["hq"]
    total = int((lens + nodes).sum())
    return {"bytes": 2 * total * row + int(nodes.sum()) * (2 * hq * d * 2 + 8) + 4 * (total // PAGE + 3 * len(lens)),
            "flops": 4 * int((nodes * (lens + nodes)).sum()) * hq * d}


# ------------------------------------------------------------------------------------------------ inputs
def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _cache(s, case, shape, gen):
    """Pools of rows whose channels (keys) differ in size: bf16, or quantised with their scales."""
    hkv, d = case["hkv"], case["d"]
    channel = torch.exp(CHANNEL_SPREAD * _normal((hkv, 1, d), gen, torch.float32))
    k, v = _normal(shape, gen, torch.float32) * channel, _normal(shape, gen, torch.float32)
    if case["fp8"]:
        (s["k_pages"], k_exp), (s["v_pages"], v_exp) = _quantise(k), _quantise(v)
        s["kv_scales"] = torch.stack([k_exp, v_exp], dim=-2).contiguous().view(torch.float8_e8m0fnu)
    else:
        s["k_pages"], s["v_pages"], s["kv_scales"] = k.to(torch.bfloat16), v.to(torch.bfloat16), None


def _workspace(case):
    """The workspace that a user's program keeps beside its cache (the library's calls take one; the plain form none)."""
    if own:
        import paged_kv_decode_gb300 as pkv

        if case["op"] == "tree_attn":
            return pkv.Workspace(pkv.tree_workspace_bytes(case["batch"] + case["pad"], case["most"], 1, case["hq"], case["hkv"], case["d"]))
        return pkv.Workspace(pkv.PKV_STATUS_BYTES)
    return None


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    hkv, d = case["hkv"], case["d"]
    s = dict(case=dict(case), workspace=_workspace(case))
    if case["op"] == "copy_pages":
        n, pad = case["pages"], case["pad"]
        pages = rng.permutation(2 * n + SPARE)
        _cache(s, case, (case["layers"], len(pages), hkv, PAGE, d), gen)
        s["src"] = _i32(np.concatenate([pages[:n], np.full(pad, -1)]))
        s["dst"] = _i32(np.concatenate([pages[n: 2 * n], np.full(pad, -1)]))
        return s
    if case["op"] == "keep_nodes":
        path, n = _paths(case)
        rows = len(n)
        prefix = rng.integers(max(0, case["high"] // 10), case["high"], size=rows, endpoint=True)
        prefix[0] = case["high"]
        width = (case["high"] + MAX_NODES) // PAGE + 1
        tail = MAX_NODES // PAGE + 1  # pages that a request's nodes can lie in; the pool has those alone
        pages = rng.permutation(rows * tail + SPARE)
        _cache(s, case, (case["layers"], len(pages), hkv, PAGE, d), gen)
        # (table entries of a request's other pages: a page of no request)
        table = np.full((rows, width + tail), pages[-1])
        table[np.arange(rows)[:, None], prefix[:, None] // PAGE + np.arange(tail)] = pages[: rows * tail].reshape(rows, tail)
        s["block_table"], s["prefix_lens"] = _i32(table[:, :width]), _i32(prefix)
        s["path"], s["path_lens"], s["idle_page"] = _i32(path), _i32(n), int(pages[-1])
        return s
    hq, lens, nodes = case["hq"], _lens(case), _nodes(case)
    rows, total = len(lens), int(nodes.sum())
    need = -(-(lens + nodes) // PAGE)
    order = rng.permutation(int(need.sum()) + SPARE)
    table = np.full((rows, max(1, int(need.max()))), order[-1])
    table[np.arange(table.shape[1])[None, :] < need[:, None]] = order[: int(need.sum())]
    s["block_table"], s["prefix_lens"] = _i32(table), _i32(lens)
    s["cu_nodes"] = _i32(np.concatenate([[0], np.cumsum(nodes)]))
    _cache(s, case, (len(order), hkv, PAGE, d), gen)
    s["q"] = _normal((total, hq, d), gen)
    s["out"] = torch.empty_like(s["q"])
    s["scale"], s["tree_mask"] = d ** -0.5, None
    if not case["chain"]:  # each node's ancestors and itself, a bit each; a node's parent is one of the eight before it
        mask = []
        for n in nodes.tolist():
            seen = []
            for i in range(n):
                seen.append((seen[int(rng.integers(max(0, i - 8), i))] if i else 0) | 1 << i)
            mask += seen
        s["tree_mask"] = torch.from_numpy(np.array(mask, dtype=np.uint64).view(np.int64)).cuda()
    # where the plain form finds a node: its request, its place in there
    s["row"] = torch.from_numpy(np.repeat(np.arange(rows), nodes)).cuda()
    s["node"] = torch.from_numpy(np.arange(total) - np.repeat(np.cumsum(nodes) - nodes, nodes)).cuda()
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


def _rows(s, which):
    """The cached rows of every request in order, as the values they stand for: [rows, hkv, width * 16, d]."""
    table = s["block_table"].long()
    pool = s["k_pages" if which == 0 else "v_pages"]
    if s["kv_scales"] is None:
        x = pool[table].float()
    else:
        x = pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(s["kv_scales"].view(torch.uint8)[table][:, :, :, which].float() - 127)[..., None]
    b, w, h, p, d = x.shape
    return x.transpose(1, 2).reshape(b, h, w * p, d)


def _plain_tree(s):
    """Scores of every request's nodes, laid out at the largest number of nodes, over every row of its table."""
    case = s["case"]
    hq, hkv, d, most = case["hq"], case["hkv"], case["d"], case["most"]
    k, v = _rows(s, 0), _rows(s, 1)
    b, _, n, _ = k.shape
    row, node = s["row"], s["node"]
    q = torch.zeros((b, most, hq, d), dtype=torch.float32, device="cuda")
    q[row, node] = s["q"].float()
    q = q.view(b, most, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)  # [b, hkv, heads * nodes, d]
    at = torch.arange(n, device="cuda") - s["prefix_lens"][:, None]  # a key's place among the nodes, negative in the prefix
    nodes = torch.arange(most, device="cuda")
    if s["tree_mask"] is None:
        seen = at[:, None, :] <= nodes[None, :, None]
    else:
        mask = torch.zeros((b, most), dtype=torch.int64, device="cuda")
        mask[row, node] = s["tree_mask"]
        bit = (mask[:, :, None] >> at.clamp(0, 63)[:, None, :]) & 1
        seen = (at[:, None, :] < 0) | ((bit == 1) & (at[:, None, :] < MAX_NODES))
    seen = seen & (at < (s["cu_nodes"][1:] - s["cu_nodes"][:-1])[:, None])[:, None, :]  # [b, nodes, n]
    score = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, -1, most, n)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=-1e30)  # a row that sees nothing has none
    p = score.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    live = (at < (s["cu_nodes"][1:] - s["cu_nodes"][:-1])[:, None])[:, None, :, None]
    o = torch.matmul(p.view(b, hkv, -1, n), v.masked_fill_(~live, 0.0)).view(b, hkv, -1, most, d) / total
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)[row, node])


def _pools(s):
    """Raw views of the pools (and of the scales): [layers, pages, hkv, 16, ...] each."""
    raw = [x.view(torch.uint8 if x.element_size() == 1 else torch.int16) for x in (s["k_pages"], s["v_pages"])]
    return raw if s["kv_scales"] is None else raw + [s["kv_scales"].view(torch.uint8).transpose(-1, -2)]


def _plain_keep(s):
    path, depth = s["path"].long(), s["path"].shape[1]
    step = torch.arange(depth, device="cuda")[None, :]
    live = (step < s["path_lens"][:, None]).view(-1)
    start = s["prefix_lens"].long()[:, None]
    to, at = start + step, start + path.clamp(min=0)

    def place(x):  # (page, slot); rows behind a path's end: a slot of the idle page, onto itself
        page = torch.gather(s["block_table"].long(), 1, x // PAGE).view(-1)
        return torch.where(live, page, torch.full_like(page, s["idle_page"])), torch.where(live, (x % PAGE).view(-1), 0)

    (to_page, to_slot), (at_page, at_slot) = place(to), place(at)
    for pool in _pools(s):
        pool[:, to_page, :, to_slot] = pool[:, at_page, :, at_slot]


def _plain_copy(s):
    n = s["case"]["pages"]
    src, dst = s["src"][:n].long(), s["dst"][:n].long()
    for pool in _pools(s):
        pool[:, dst] = pool[:, src]


def run(state):
    s = state
    op, scales = s["case"]["op"], s["kv_scales"]
    if own:
        import paged_kv_decode_gb300 as pkv

        if op == "copy_pages":
            pkv.copy_pages(s["src"], s["dst"], s["k_pages"], s["v_pages"], scales, workspace=s["workspace"])
        elif op == "keep_nodes":
            pkv.keep_nodes(s["path"], s["path_lens"], s["prefix_lens"], s["block_table"], s["k_pages"], s["v_pages"], scales,
                           workspace=s["workspace"])
        elif scales is None:
            pkv.tree_attn(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["prefix_lens"], s["cu_nodes"],
                          s["tree_mask"], s["out"], s["scale"], s["case"]["most"], s["workspace"])
        else:
            pkv.tree_attn_fp8(s["q"], s["k_pages"], s["v_pages"], scales, s["block_table"], s["prefix_lens"], s["cu_nodes"],
                              s["tree_mask"], s["out"], s["scale"], s["case"]["most"], s["workspace"])
    elif op == "copy_pages":
        _plain_copy(s)
    elif op == "keep_nodes":
        _plain_keep(s)
    else:
        _plain_tree(s)
    if op == "tree_attn":
        return {"out": s["out"]}
    return {n: s[n] for n in ("k_pages", "v_pages", "kv_scales") if s[n] is not None}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _value(bytes8):
    """What the e4m3 codes 0..255 stand for, from the format's definition (7 exponent bias, no infinities)."""
    code = torch.arange(256, dtype=torch.float64, device="cuda")
    low, sign = code % 128, torch.where(code >= 128, -1.0, 1.0)
    e, m = torch.div(low, 8, rounding_mode="floor"), low % 8
    v = torch.where(e > 0, (1 + m / 8) * _power(e - 7), m / 8 * 2.0 ** -6)
    v = torch.where(low == 127, torch.full_like(v, math.nan), v) * sign
    return v[bytes8.int()]


def _power(e):
    """2^e in 64 bits, exactly, for whole numbers e."""
    return torch.from_numpy(np.ldexp(1.0, np.arange(-200, 201))).cuda()[e.long() + 200]


def _moved(s, pairs):
    """The pools' values with every (page, rows) <- (page, rows) of the pairs carried out, read before any is written."""
    new = []
    for old in _pools(s):
        x = old.clone()
        for (page, rows), (from_page, from_rows) in pairs:
            x[:, page, :, rows] = old[:, from_page, :, from_rows]
        new.append(x)
    if s["kv_scales"] is None:
        return {"k_pages": new[0].view(torch.bfloat16).double(), "v_pages": new[1].view(torch.bfloat16).double()}
    return {"k_pages": torch.stack([_value(x) for x in new[0]]), "v_pages": torch.stack([_value(x) for x in new[1]]),
            "kv_scales": _power(new[2].transpose(-1, -2).int() - 127)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy_pages":
        n, whole = case["pages"], slice(0, PAGE)
        return _moved(s, [((b, whole), (a, whole)) for a, b in zip(s["src"][:n].tolist(), s["dst"][:n].tolist())])
    if case["op"] == "keep_nodes":
        path, n = s["path"].tolist(), s["path_lens"].tolist()
        prefix, table = s["prefix_lens"].tolist(), s["block_table"].tolist()
        place = lambda b, x: (table[b][x // PAGE], x % PAGE)  # noqa: E731
        pairs = [(place(b, prefix[b] + i), place(b, prefix[b] + path[b][i])) for b in range(len(n)) for i in range(n[b])]
        return _moved(s, pairs)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens, cu = s["prefix_lens"].tolist(), s["cu_nodes"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    masks = None if s["tree_mask"] is None else s["tree_mask"].tolist()

    def rows(b, pool, which, n):  # [hkv, n, d] of one request
        page = s["block_table"][b, : -(-n // PAGE)].long()
        if s["kv_scales"] is None:
            x = pool[page].double()
        else:
            x = _value(pool.view(torch.uint8)[page]) * _power(s["kv_scales"].view(torch.uint8)[page][:, :, which].int() - 127)[..., None]
        return x.transpose(0, 1).reshape(hkv, -1, d)[:, :n]

    for b, prefix in enumerate(lens):
        t = cu[b + 1] - cu[b]
        if not t:
            continue
        k, v = rows(b, s["k_pages"], 0, prefix + t), rows(b, s["v_pages"], 1, prefix + t)
        hidden = torch.zeros((t, prefix + t), dtype=torch.bool, device="cuda")
        hidden[:, prefix:] = torch.tensor([[j > i if masks is None else not masks[cu[b] + i] >> j & 1 for j in range(t)] for i in range(t)])
        q = s["q"][cu[b]: cu[b + 1]].double().view(t, hkv, hq // hkv, d)
        p = torch.einsum("thgd,hnd->hgtn", q, k) * s["scale"]
        p = torch.softmax(p.masked_fill_(hidden, -math.inf), -1)  # (every node sees itself)
        out[cu[b]: cu[b + 1]] = torch.einsum("hgtn,hnd->thgd", p, v).reshape(t, hq, d)
    return {"out": out}
