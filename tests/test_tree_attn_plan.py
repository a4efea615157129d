"""Tree attention's schedule on the device: the descriptors of cut items read back from the workspace and compared with the
schedule restated, captured calls replayed with other lengths, nodes, masks and tables (whole items, cut ones, none), four and
five query heads per KV head, and a captured step of many layers behind one another."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gb300 as pkv
from gpu_util import ensure_built, i32
from parity import bf16_to_f64
from test_tree_attn import GEOMS, REQS, THETA, Tree, _pieces, ancestors

GROUPS = {"32q8kv128": (32, 8, 128), "16q4kv64": (16, 4, 64), "40q8kv128": (40, 8, 128), "5q1kv64": (5, 1, 64)}


def _bits(t):
    return t.clone().view(torch.int16)


def _raw(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


# ---------------------------------------------------------------------------------------------- group sizes
@pytest.mark.gpu
@pytest.mark.parametrize("masks", ["tree", "any"])
@pytest.mark.parametrize("reqs", sorted(REQS))
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("geom", sorted(GROUPS))
def test_four_and_five_query_heads_to_a_kv_head(cuda_device, geom, fp8, reqs, masks):
    c = Tree(51, GROUPS[geom], REQS[reqs], cuda_device, fp8=fp8, masks=masks)
    c.step()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("geom", sorted(GROUPS))
def test_cut_items_of_several_row_tiles(cuda_device, geom):
    """More than 128 query rows a KV head (25 nodes of five heads fill 125 of a tile's rows), cut and whole, both caches; the
    8-bit one with the bits of its expanded pages."""
    reqs = [(5000, 64), (300, 26), (0, 51), (1200, 33)]
    c = Tree(52, GROUPS[geom], reqs, cuda_device)
    c.step()
    c.check()
    c = Tree(52, GROUPS[geom], reqs, cuda_device, fp8=True)
    got = _bits(c.step())
    c.check()
    k, v = (torch.zeros(c.pools[0].shape, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    pkv.expand_fp8(*c.pools, c.bt, i32([p + t for p, t in reqs], cuda_device), k, v, c.bt)
    out = torch.empty_like(c.out)
    pkv.tree_attn(c.q, k, v, c.bt, c.prefix, c.cu, c.mask, out, c.scale, c.most, c.ws)
    assert torch.equal(_bits(out), got)


# ---------------------------------------------------------------------------------------------- descriptors
def _expected_cuts(c, most, ctas):
    """{entry: (rows, first row, KV head, first CTA, last CTA)} of the cut items, and whether entries go by item."""
    grp = c.hq // c.hkv
    tile = 128 // grp
    items, names = [], []
    for b, (p, t) in enumerate(c.reqs):
        for h in range(c.hkv):
            for rt in range(-(-t // tile)):
                items.append(-(-(p + t) // 128))
                names.append((b, h, rt))
    tiles = -(-most // tile)
    by_item = len(c.reqs) * c.hkv * tiles <= ctas
    if not items:
        return {}, by_item
    pieces, last = _pieces(items, ctas)
    want = {}
    for cta, i, k0, k1 in pieces:
        if k0 == 0 and k1 < items[i]:
            b, h, rt = names[i]
            entry = (b * c.hkv + h) * tiles + rt if by_item else cta
            want[entry] = (grp * min(tile, c.reqs[b][1] - rt * tile), int(c.cu_np[b]) + rt * tile, h, cta, last[i])
    return want, by_item


PLANS = {"one": ("16q8kv128", [(20000, 32)], 32), "mixed": ("16q8kv128", [(300 + 171 * i, 16) for i in range(16)], 16),
         "by_cta": ("16q8kv128", [(40 + 101 * i, 1 + i % 16) for i in range(24)], 16),
         "row_tiles": ("28q4kv128", [(3000, 64), (40, 2), (0, 0), (1500, 30)], 64), "five": ("40q8kv128", [(7000, 60), (90, 26)], 64),
         "whole": ("14q2kv64", [(100, 9), (300, 3), (0, 0)], 16), "balanced": ("16q8kv128", [(1500, 8)] * 19, 8),
         "none": ("14q2kv64", [(700, 0), (0, 0)], 16)}


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", sorted(PLANS))
def test_descriptors_of_cut_items(cuda_device, case, fp8):
    name, reqs, most = PLANS[case]
    geom = {**GEOMS, **GROUPS}[name]
    c = Tree(53, geom, reqs, cuda_device, fp8=fp8, width=1300)
    ctas = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    c.ws.tensor[pkv.PKV_STATUS_BYTES:] = 0xFF
    pad = torch.zeros((1, *c.q.shape[1:]), dtype=torch.bfloat16, device=cuda_device)  # (a call has at least one row)
    c.step(q=torch.cat([c.q, pad]), out=torch.cat([c.out, pad]), tree_mask=None, max_nodes=most)
    torch.cuda.synchronize()
    raw = c.ws.tensor[pkv.PKV_STATUS_BYTES: pkv.PKV_STATUS_BYTES + 16 * ctas].cpu().numpy().view(np.int32).reshape(ctas, 4)
    want, by_item = _expected_cuts(c, most, ctas)
    entries = len(reqs) * geom[1] * -(-most // (128 // (geom[0] // geom[1]))) if by_item else ctas
    got = {i: (int(r), int(q), int(h), int(s) & 0xFFFF, int(s) >> 16) for i, (r, q, h, s) in enumerate(raw[:entries]) if r != 0}
    assert got == want
    assert bool(want) == (case not in ("whole", "balanced", "none"))
    assert by_item == (case != "by_cta")  # (19 requests of 8 heads are 152 items, an entry each)


# ---------------------------------------------------------------------------------------------- replays
REPLAYS = {
    # descriptors by item
    "few_items": ("14q2kv64", 40, [[(12000, 40), (700, 3), (0, 17)], [(100, 5), (30, 2), (60, 20)], [(0, 0), (9000, 33), (0, 0)],
                                   [(0, 0)] * 3, [(5000, 1), (5000, 40), (2000, 19)], [(3, 40), (0, 0), (12000, 1)]]),
    # descriptors by CTA, one row tile
    "many_items": ("16q8kv128", 16, [[(100 + 41 * i, 1 + i % 16) for i in range(24)], [(10 + 3 * i, 2) for i in range(24)],
                                     [(600, 16 * (i % 2)) for i in range(24)], [(5000, 9)] + [(0, 0)] * 23, [(0, 0)] * 24,
                                     [(500, 5)] * 24]),
    # descriptors by CTA, up to two row tiles an item
    "row_tiles": ("32q8kv128", 64, [[(1100 - 90 * i, 64 - 5 * i) for i in range(10)], [(40, 33)] * 10, [(3000, 64)] + [(0, 0)] * 9,
                                    [(64 * i, 64 * (i % 2)) for i in range(10)]]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", sorted(REPLAYS))
def test_captured_call_replayed_with_other_lengths(cuda_device, case, fp8):
    """One captured call; lengths, nodes, masks, tables, pools and queries change in place between replays, from long requests
    to short ones, to none, and back. Rows behind the last node stay as they were."""
    name, most, variants = REPLAYS[case]
    geom = {**GEOMS, **GROUPS}[name]
    need = lambda reqs: sum(-(-(p + t) // 16) for p, t in reqs)  # noqa: E731
    width = max(-(-(p + t) // 16) for reqs in variants for p, t in reqs)
    pages, room = max(need(r) for r in variants) + 2, max(sum(t for _, t in r) for r in variants) + 3

    def build(i):
        return Tree(60 + i, geom, variants[i], cuda_device, fp8=fp8, width=width, spare=pages - need(variants[i]))

    first = build(0)
    ws = first.ws
    assert ws.nbytes >= pkv.tree_workspace_bytes(len(variants[0]), most, pages, *geom)
    held = dict(q=torch.zeros((room, *first.q.shape[1:]), dtype=torch.bfloat16, device=cuda_device),
                out=torch.zeros((room, *first.q.shape[1:]), dtype=torch.bfloat16, device=cuda_device),
                tree_mask=torch.zeros(room, dtype=torch.int64, device=cuda_device), block_table=first.bt.clone(),
                prefix_lens=first.prefix.clone(), cu_nodes=first.cu.clone())
    pools = [x.clone() for x in first.pools]
    call = Tree.__new__(Tree)
    call.fp8, call.pools, call.scale, call.most, call.ws = fp8, pools, first.scale, most, ws
    for key in ("q", "out"):
        setattr(call, key, held[key])
    call.bt, call.prefix, call.cu, call.mask = held["block_table"], held["prefix_lens"], held["cu_nodes"], held["tree_mask"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call.step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call.step()
    for i in [*range(len(variants)), 1, 0]:
        t = build(i)
        n = int(t.cu_np[-1])
        held["q"].fill_(float("nan"))
        held["q"][:n] = t.q
        held["tree_mask"].fill_(-1)
        if n:
            held["tree_mask"][:n] = t.mask
        for key, x in (("block_table", t.bt), ("prefix_lens", t.prefix), ("cu_nodes", t.cu)):
            held[key].copy_(x)
        for x, y in zip(pools, t.pools):
            _raw(x).copy_(_raw(y))
        held["out"].fill_(3.5)
        graph.replay()
        t.ws = ws
        t.check(held["out"][:n])
        assert (held["out"][n:] == 3.5).all()
        if n:  # and an eager call's bits
            assert torch.equal(_bits(t.step(max_nodes=most)), _bits(held["out"][:n]))


# ---------------------------------------------------------------------------------------------- values
@pytest.mark.gpu
@pytest.mark.parametrize("power", [10, 20, 40, 100])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_every_row_of_huge_scores_is_a_mean_of_values(cuda_device, fp8, power):
    """Whatever the scores' size, an output is a weighted mean of value rows: finite and no larger than the largest of them
    (and half a step of bf16, of the weights and of the output, and the sums' last bits). Where one score is far ahead it is
    that row; most are."""
    c = Tree(54, GEOMS["16q8kv128"], [(1000, 6), (200, 1), (0, 3)], cuda_device, fp8=fp8, q_size=2.0 ** power)
    got = bf16_to_f64(c.step())
    assert np.isfinite(got).all()
    clear = rows = 0
    for b, (p, t) in enumerate(c.reqs):
        pages = c.table[b, : -(-(p + t) // 16)]
        flat = lambda x: x[pages].transpose(0, 2, 1, 3).reshape(-1, c.hkv, c.d)[: p + t]  # noqa: E731
        k, v = flat(c.k64), flat(c.v64)
        for i in range(t):
            n = int(c.cu_np[b]) + i
            q = bf16_to_f64(c.q[n])
            seen = np.array([True] * p + [bool(c.mask_np[n] >> j & 1) for j in range(t)])
            for h in range(c.hq):
                most = np.abs(v[seen, h // 2]).max(axis=0)
                assert (np.abs(got[n, h]) <= most * (1 + 2.0 ** -7 + 2.0 ** -13)).all()
                s = np.where(seen, k[:, h // 2] @ q[h], -np.inf) * c.scale
                order = np.argsort(s)
                slack = (c.d + 8) * 2.0 ** -23 * c.scale * (np.abs(k[:, h // 2]) @ np.abs(q[h])).max()
                rows += 1
                if seen.sum() < 2 or s[order[-1]] - s[order[-2]] > slack + 40:
                    clear += 1
                    want = v[order[-1], h // 2]
                    assert (np.abs(got[n, h] - want) <= 2.0 ** -8 * np.abs(want) + 1e-12).all()
    assert clear >= rows // 2


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [-1, 1])
def test_infinite_values_leave_other_nodes_and_columns_alone(cuda_device, sign):
    """An infinite value of one node: its column is infinite for the nodes that see it; all else keeps its bits."""
    c = Tree(55, GEOMS["16q8kv128"], [(700, 40), (90, 5)], cuda_device)
    clean = _bits(c.step())
    j = 3
    page, slot = int(c.table[0, (700 + j) // 16]), (700 + j) % 16
    # the column's clean sums are not those with a zero in this row: take it as zero, then as infinite
    c.pools[1][page, :, slot, 5] = 0.0
    zero = _bits(c.step())
    c.pools[1][page, :, slot, 5] = sign * float("inf")
    got = c.step()
    seen = np.array([i < 40 and bool(c.mask_np[i] >> j & 1) for i in range(45)])
    assert seen.any() and not seen[:40].all()
    assert torch.equal(_bits(got)[~seen], clean[~seen]) and torch.equal(_bits(got)[~seen], zero[~seen])
    x = bf16_to_f64(got)[seen]
    assert (x[..., 5] == sign * np.inf).all()
    rest = [i for i in range(c.d) if i != 5]
    assert torch.equal(_bits(got)[seen][..., rest], clean[seen][..., rest])
    assert c.ws.status() == 0


# ---------------------------------------------------------------------------------------------- a step of many layers
@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("reqs", [[(2000, 16), (700, 9), (31, 4)], [(90, 5), (200, 8)]], ids=["cut", "whole"])
def test_layers_in_one_graph(cuda_device, fp8, reqs):
    """Append with norm and rotation, tree attention, and the next layer's append of rows that come from its output: 12 layers
    in one captured graph, where each kernel starts while the one in front ends, then the kept rows and a copied page in all
    layers. Bit for bit the calls with a wait after each, for new inputs in place too."""
    ensure_built()
    dev, (hq, hkv, d), layers = cuda_device, GEOMS["16q8kv128"], 12
    rng = np.random.default_rng(56)
    gen = torch.Generator().manual_seed(56)
    total = sum(t for _, t in reqs)
    width = -(-max(p + t for p, t in reqs) // 16)
    pages = len(reqs) * width + 2
    table = rng.permutation(pages - 2).reshape(len(reqs), width)
    slots = [int(table[b, (p + i) // 16]) * 16 + (p + i) % 16 for b, (p, t) in enumerate(reqs) for i in range(t)]
    cu = np.concatenate([[0], np.cumsum([t for _, t in reqs])])
    masks = [m for _, t in reqs for m in ancestors(rng, t)]
    depth = [p + bin(m).count("1") - 1 for (p, m) in zip(np.repeat([p for p, _ in reqs], [t for _, t in reqs]), masks)]
    row = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(dev)  # noqa: E731
    weight, cos_sin = torch.ones(d, dtype=torch.bfloat16, device=dev), pkv.rope_cos_sin(THETA, 4096, d, dev)
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    pools = [row(layers, pages, hkv, 16, d).to(kind) for _ in range(2)]
    if fp8:
        pools.append(torch.full((layers, pages, hkv, 2, 16), 127, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu))
    start = [_raw(x).clone() for x in pools]
    x, q_rot = row(total, hq, d), torch.empty(layers, total, hq, d, dtype=torch.bfloat16, device=dev)
    out = torch.empty_like(q_rot)
    mask = torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64)).to(dev)
    bt, prefix, cu_d, pos, slot = (i32(a, dev) for a in (table, [p for p, _ in reqs], cu, depth, slots))
    path, n_path = i32([[0, 2, 3]] * len(reqs), dev), i32([3] * len(reqs), dev)
    src, dst = i32([int(table[0, 0]), int(table[-1, -1])], dev), i32([pages - 2, pages - 1], dev)
    ws = pkv.Workspace(pkv.tree_workspace_bytes(len(reqs), 16, pages, hq, hkv, d), dev)

    def step(wait):
        done = torch.cuda.synchronize if wait else lambda: None
        rows = x
        for at in range(layers):
            layer = [p[at] for p in pools]
            # (keys and values: heads of the layer's input)
            (pkv.append_rope_fp8 if fp8 else pkv.append_rope)(rows[:, :hkv], rows[:, hkv:], pos, slot, cos_sin, *layer, ws, q=rows,
                                                              q_out=q_rot[at], q_weight=weight, k_weight=weight)
            done()
            (pkv.tree_attn_fp8 if fp8 else pkv.tree_attn)(q_rot[at], *layer, bt, prefix, cu_d, mask, out[at], d ** -0.5, 16, ws)
            done()
            rows = out[at]
        pkv.keep_nodes(path, n_path, prefix, bt, *pools, workspace=ws)
        done()
        pkv.copy_pages(src, dst, *pools, workspace=ws)
        done()

    def fresh():
        for p, s in zip(pools, start):
            _raw(p).copy_(s)
        out.fill_(float("nan"))
        q_rot.fill_(float("nan"))
        torch.cuda.synchronize()

    def result():
        torch.cuda.synchronize()
        assert ws.status() == 0
        return [_raw(y).clone() for y in (out.view(torch.int16), q_rot.view(torch.int16), *[_raw(p) for p in pools])]

    fresh()
    step(True)
    want = result()
    assert np.isfinite(bf16_to_f64(out)).all()
    fresh()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(False)
    for turn in range(6):
        if turn == 3:  # other inputs in the same graph
            x.copy_(row(total, hq, d))
            fresh()
            step(True)
            want = result()
        fresh()
        graph.replay()
        for got, w in zip(result(), want):
            same = got.view(torch.int16) if got.dtype == torch.bfloat16 else got
            assert torch.equal(same, w.view(torch.int16) if w.dtype == torch.bfloat16 else w)
