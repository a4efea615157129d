"""Attention of drafted nodes over the paged cache (bf16 and 8-bit) against float64 numpy written from the definition, and
a speculative step as it is used: append, tree attention, keeping the accepted nodes, decode.

Tolerance (tree_bound), elementwise on |got - out|, from the call's roundings: bf16 output, half a step (2^-8 relative); the
softmax weights as bf16, 2^-8 each, so 2^-8 sum p |v|; the approximate exponentials and their arguments' last bits, 2^-14;
the fp32 score sums over d products, (d + 8) 2^-24 of scale * sum |q| |k|, which move numerator and denominator; the fp32
sums over n keys in steps of 16, one rounding or truncation (2^-23) a step, and their 16 joins."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_decode_gb300 as pkv
from fp8_util import cache_to, dequantise, random_cache
from gpu_util import ensure_built, i32
from paged_kv_decode_gb300 import _lib
from paged_kv_decode_gb300.build import build_library
from parity import bf16_to_f64

THETA = 1.0e6


# ---------------------------------------------------------------------------------------------- CPU
@pytest.fixture(scope="module")
def lib():
    build_library()
    return _lib.load()


def _desc(**kw):
    d = dict(num_q_heads=16, num_kv_heads=8, head_dim=128, page_size=16, num_pages=4)
    d.update(kw)
    return _lib.CacheDesc(**d)


@pytest.mark.parametrize("fp8", [False, True])
def test_host_argument_checks(lib, fp8):
    buf = ctypes.create_string_buffer(1024)
    p = (ctypes.addressof(buf) + 255) // 256 * 256  # never dereferenced: every call below ends on the host

    def call(desc=_desc(), q=p, kp=p, vp=p, sc=p, bt=p, pl=p, cu=p, mask=p, seqs=2, total=8, most=4, out=p, pages=4, ws=p,
             nb=1 << 30):
        f = lib.pkv_tree_attn_fp8 if fp8 else lib.pkv_tree_attn
        scales = (sc,) if fp8 else ()
        return f(q, kp, vp, *scales, bt, pl, cu, mask, seqs, total, most, out, 1.0, None,
                 None if desc is None else ctypes.byref(desc), pages, ws, nb)

    assert call(desc=None) == -1
    for bad in (_desc(head_dim=96), _desc(page_size=32), _desc(num_q_heads=36, num_kv_heads=4), _desc(num_q_heads=20)):
        assert call(desc=bad) == -3
    assert call(desc=_desc(num_pages=0)) == -2
    assert call(seqs=-1) == -2 and call(total=-1) == -2 and call(most=-1) == -2 and call(pages=0) == -2
    # (the end of the last tile of 128 keys, 128 ceil(16 pages / 128), is past 2^31 - 1 from 2^27 - 7 pages on)
    assert call(pages=(1 << 27) - 7, seqs=1) == -2 and call(seqs=1024, pages=1 << 18) == -2
    assert call(seqs=1025) == -3 and call(most=65) == -3
    assert call(ws=None) == -1 and call(nb=64) == -4
    assert call(seqs=0) == 0 and call(total=0) == 0 and call(most=0) == 0  # nothing to do, no device
    for name in ("q", "kp", "vp", "bt", "pl", "cu", "out"):
        assert call(**{name: None}) == -1, name
    for name in ("q", "kp", "vp", "out", "ws"):
        assert call(**{name: p + 8}) == -8, name
    assert call(mask=p + 4) == -8
    if fp8:
        assert call(sc=None) == -1 and call(sc=p + 8) == -8
    d = _desc()
    for bad in ((None, 1, 4), (ctypes.byref(_desc(head_dim=96)), 1, 4), (ctypes.byref(d), -1, 4),
                (ctypes.byref(d), 1025, 4), (ctypes.byref(d), 1, 65)):
        assert lib.pkv_tree_workspace_bytes(*bad) == 0


def _pieces(items, grid, cost=3, small=7):
    """The schedule of tree_attn.cu, restated: (cta, item, k0, k1) of every piece, for items of so many key tiles, and for
    each item the CTA with its last unit."""
    units, largest = sum(cost + n for n in items), cost + max(items)
    whole = largest <= small or 4 * largest * -(-len(items) // grid) * grid <= 5 * units
    size = [1 if whole else cost + n for n in items]
    units = sum(size)
    ctas = min(grid, units)
    quota, more = divmod(units, ctas)
    starts = np.concatenate([[0], np.cumsum(size)])
    got = []
    for c in range(ctas):
        lo = c * quota + min(c, more)
        hi = lo + quota + (c < more)
        for i, n in enumerate(items):
            a, b = max(lo, int(starts[i])), min(hi, int(starts[i + 1]))
            k0, k1 = (0, n) if whole else (max(0, a - int(starts[i]) - cost), max(0, b - int(starts[i]) - cost))
            if a < b and k1 > k0:
                got.append((c, i, k0, k1))
    split = more * (quota + 1)
    cta_of = lambda u: u // (quota + 1) if u < split else more + (u - split) // quota  # noqa: E731
    return got, [cta_of(int(s) - 1) for s in starts[1:]]


@pytest.mark.parametrize("grid", [1, 7, 152])
def test_shares_cover_the_items_and_records_are_distinct(grid):
    rng = np.random.default_rng(3)
    for items in ([1], [1] * 300, [313], [5, 1, 400, 2, 2, 60], rng.integers(1, 30, size=128).tolist(), [63] * 8, [4000] * 2,
                  [16] * 152, [4, 1, 3] * 90, [5] * 9):
        pieces, last = _pieces(items, grid)
        seen, slots, cuts = {}, set(), set()
        for c, i, k0, k1 in pieces:
            seen.setdefault(i, []).append((k0, k1, c))
            if (k0, k1) != (0, items[i]):  # a record: its slot is its own
                slot = (c, 1 if k0 == 0 else 0)
                assert slot not in slots
                slots.add(slot)
        for i, n in enumerate(items):
            parts = sorted(seen[i])
            assert parts[0][0] == 0 and parts[-1][1] == n and all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
            if len(parts) > 1:  # the CTAs that are joined: consecutive, each with a piece; one descriptor for each cut item
                assert [c for _, _, c in parts] == list(range(parts[0][2], last[i] + 1))
                assert parts[0][2] not in cuts
                cuts.add(parts[0][2])


# ---------------------------------------------------------------------------------------------- GPU
GEOMS = {"16q8kv128": (16, 8, 128), "64q8kv128": (64, 8, 128), "28q4kv128": (28, 4, 128), "12q4kv128": (12, 4, 128),
         "32q32kv64": (32, 32, 64), "8q1kv64": (8, 1, 64), "14q2kv64": (14, 2, 64), "12q2kv64": (12, 2, 64)}


def ancestors(rng, n, reach=8):
    seen = []
    for i in range(n):
        seen.append((seen[int(rng.integers(max(0, i - reach), i))] if i else 0) | 1 << i)
    return seen


class Tree:
    """Seeded requests (prefix, nodes), a permuted pool, every row that no request sees filled with NaN."""

    def __init__(self, seed, geom, reqs, dev, *, fp8=False, masks="tree", spare=2, width=None, q_size=1.0):
        ensure_built()
        self.hq, self.hkv, self.d = geom
        self.reqs, self.dev, self.fp8 = reqs, dev, fp8
        rng = np.random.default_rng(seed)
        need = [-(-(p + t) // 16) for p, t in reqs]
        order = rng.permutation(sum(need) + spare)
        self.pages = len(order)
        width = max([1] + need) if width is None else width
        self.table = np.full((len(reqs), width), self.pages + 99, dtype=np.int32)  # entries past a request's pages: never read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at: at + n]
            at += n
        shape = (self.pages, self.hkv, 16, self.d)
        live = np.zeros(shape[:3], dtype=bool)
        for b, (p, t) in enumerate(reqs):
            for i, page in enumerate(self.table[b, : need[b]]):
                live[page, :, : min(16, p + t - 16 * i)] = True
        if fp8:
            kc, vc, sc = random_cache(seed, self.pages, self.hkv, self.d)
            kc[~live], vc[~live] = 0x7F, 0xFF
            self.k64, self.v64 = dequantise(kc, sc[:, :, 0]), dequantise(vc, sc[:, :, 1])
            self.pools = cache_to(kc, vc, sc, dev)
        else:
            ch = np.exp(0.5 * rng.standard_normal((self.hkv, 1, self.d)))
            make = lambda x: torch.from_numpy(np.where(live[..., None], x, np.nan)).to(torch.bfloat16)  # noqa: E731
            k, v = make(rng.standard_normal(shape) * ch), make(rng.standard_normal(shape))
            self.k64, self.v64 = bf16_to_f64(k), bf16_to_f64(v)
            self.pools = (k.to(dev), v.to(dev))
        self.cu_np = np.concatenate([[0], np.cumsum([t for _, t in reqs])]).astype(np.int32)
        total = int(self.cu_np[-1])
        self.mask_np = None
        if masks == "tree":
            self.mask_np = [m for _, t in reqs for m in ancestors(rng, t)]
        elif masks == "any":  # any nodes of the request, also none, and bits past the last node
            self.mask_np = [int(rng.integers(0, 1 << 63)) << 1 | int(rng.integers(0, 2)) if rng.random() < 0.8 else 0
                            for _ in range(total)]
        self.set_masks(self.mask_np)
        self.q = torch.from_numpy(q_size * rng.standard_normal((total, self.hq, self.d))).to(torch.bfloat16).to(dev)
        self.out = torch.empty_like(self.q)
        self.scale = self.d ** -0.5
        self.bt, self.prefix, self.cu = i32(self.table, dev), i32([p for p, _ in reqs], dev), i32(self.cu_np, dev)
        self.most = max([1] + [t for _, t in reqs])
        self.ws = pkv.Workspace(pkv.tree_workspace_bytes(len(reqs), self.most, self.pages, *geom), dev)

    def set_masks(self, masks):
        self.mask_np = masks
        self.mask = None if masks is None else torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64)).to(self.dev)

    def step(self, **kw):
        a = dict(q=self.q, block_table=self.bt, prefix_lens=self.prefix, cu_nodes=self.cu, tree_mask=self.mask, out=self.out,
                 scale=self.scale, max_nodes=self.most, workspace=self.ws)
        a.update(kw)
        names = ("k_pages", "v_pages", "kv_scales")
        (pkv.tree_attn_fp8 if self.fp8 else pkv.tree_attn)(**dict(zip(names, self.pools)), **a)
        return a["out"]

    def want(self, b):
        """(out, sum p |v|, largest sum |q| |k| per head) of request b's nodes, in 64 bits."""
        p, t = self.reqs[b]
        pages = self.table[b, : -(-(p + t) // 16)]
        flat = lambda x: x[pages].transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.d)[: p + t]  # noqa: E731
        k, v = flat(self.k64), flat(self.v64)
        seen = np.ones((t, p + t), dtype=bool)
        for i in range(t):
            m = (2 << i) - 1 if self.mask_np is None else self.mask_np[self.cu_np[b] + i]
            seen[i, p:] = [bool(m >> j & 1) for j in range(t)]
        return tree64(bf16_to_f64(self.q[self.cu_np[b]: self.cu_np[b + 1]]), k, v, self.scale, seen)

    def check(self, out=None, only=None):
        torch.cuda.synchronize()
        assert self.ws.status() == 0
        got = bf16_to_f64(self.out if out is None else out)
        for b, (p, t) in enumerate(self.reqs):
            if t and (only is None or b in only):
                want, absolute, size = self.want(b)
                err = np.abs(got[self.cu_np[b]: self.cu_np[b + 1]] - want)
                bound = tree_bound(want, absolute, size, self.scale, self.d, p + t)
                assert (err <= bound).all(), (b, float((err / bound).max()))


def tree64(q, k, v, scale, seen):
    t, hq, d = q.shape
    n, hkv, _ = k.shape
    qg = q.reshape(t, hkv, hq // hkv, d)
    s = np.einsum("thgd,nhd->hgtn", qg, k) * scale
    s = np.where(seen, s, -np.inf)
    top = s.max(axis=-1, keepdims=True)
    w = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = w.sum(axis=-1, keepdims=True)
    w = w / np.where(total > 0, total, 1.0)
    out = np.einsum("hgtn,nhd->thgd", w, v).reshape(t, hq, d)
    absolute = np.einsum("hgtn,nhd->thgd", w, np.abs(v)).reshape(t, hq, d)
    size = np.einsum("thgd,nhd->hgtn", np.abs(qg), np.abs(k)).max(axis=-1).transpose(2, 0, 1).reshape(t, hq)
    return out, absolute, size


def tree_bound(out, absolute, size, scale, d, n):
    ds = (d + 8) * 2.0 ** -24 * abs(scale) * size[..., None]
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -14 + 2 * ds + (n / 16 + 16) * 2.0 ** -23) * absolute + 1e-37


REQS = {"ends": [(0, 1), (1, 1), (15, 1), (16, 3), (127, 1), (128, 1), (120, 8), (129, 2)],
        "wide": [(100, 64), (64, 64), (65, 63), (0, 64), (193, 33), (63, 2)],
        "ragged": [(37, 4), (5, 0), (200, 17), (0, 0), (0, 5), (1000, 9), (3, 0)],
        "one": [(700, 16)]}


@pytest.mark.gpu
@pytest.mark.parametrize("masks", ["tree", "chain", "any"])
@pytest.mark.parametrize("reqs", sorted(REQS))
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("geom", sorted(GEOMS))
def test_tree(cuda_device, geom, fp8, reqs, masks):
    c = Tree(11, GEOMS[geom], REQS[reqs], cuda_device, fp8=fp8, masks=masks)
    c.step()
    c.check()


CUT = {"long": ("16q8kv128", [(20000, 32)]), "small_heads": ("8q1kv64", [(9000, 7), (100, 60)]),
       "batch": ("16q8kv128", [(300 + 171 * i, 16) for i in range(16)]),
       "several_tiles": ("28q4kv128", [(3000, 64), (40, 2), (1500, 30)]),
       "two_tiles": ("64q8kv128", [(5000, 64), (300, 20), (0, 33), (4000, 40)]), "two_tiles_long": ("12q2kv64", [(16000, 64)]),
       "many": ("14q2kv64", [(i % 50, 1 + i % 3) for i in range(300)])}


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", sorted(CUT))
def test_cut_items_twice_on_one_workspace(cuda_device, case, fp8):
    geom, reqs = CUT[case]
    c = Tree(12, GEOMS[geom], reqs, cuda_device, fp8=fp8)
    first = c.step().clone()
    c.check()
    c.ws.tensor[256:] = 0xFF  # what calls leave behind the status header does not matter (NaN here)
    c.out.fill_(7.0)
    assert torch.equal(c.step().view(torch.int16), first.view(torch.int16))
    c.check()


def _bits(t):
    return t.clone().view(torch.int16)


@pytest.mark.gpu
@pytest.mark.parametrize("geom,reqs", [("16q8kv128", [(700, 16), (40, 3), (0, 64)]),
                                       ("14q2kv64", [(9000, 33), (17, 1)])], ids=str)
def test_8bit_gives_the_bits_of_expanded_pages(cuda_device, geom, reqs):
    c = Tree(21, GEOMS[geom], reqs, cuda_device, fp8=True)
    got = _bits(c.step())
    k, v = (torch.full(c.pools[0].shape, float("nan"), dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    lens = i32([p + t for p, t in reqs], cuda_device)
    pkv.expand_fp8(*c.pools, c.bt, lens, k, v, c.bt)
    out = torch.empty_like(c.out)
    pkv.tree_attn(c.q, k, v, c.bt, c.prefix, c.cu, c.mask, out, c.scale, c.most, c.ws)
    assert torch.equal(_bits(out), got)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_page_order_does_not_matter(cuda_device, fp8):
    c = Tree(22, GEOMS["16q8kv128"], [(3000, 9), (16, 16), (511, 2)], cuda_device, fp8=fp8)
    first = _bits(c.step())
    perm = np.random.default_rng(1).permutation(c.pages)
    back = np.argsort(perm)
    raw = lambda x: x.view(torch.uint8) if x.element_size() == 1 else x  # noqa: E731
    c.pools = [raw(x)[torch.from_numpy(perm).to(cuda_device)].contiguous().view(x.dtype) for x in c.pools]
    c.bt = i32(np.where(c.table < c.pages, back[np.minimum(c.table, c.pages - 1)], c.table), cuda_device)
    assert torch.equal(_bits(c.step()), first)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("geom,reqs", [("16q8kv128", [(300, 24), (120, 40), (0, 64)]), ("28q4kv128", [(2500, 64)]),
                                       ("8q1kv64", [(7000, 30)]), ("14q2kv64", [(60, 5), (3, 20)])], ids=str)
def test_rows_that_a_node_does_not_see_do_not_matter(cuda_device, geom, reqs, fp8):
    """NaN and infinities in a node's key and value rows: bit for bit the old output for the nodes that do not see it, no
    number where a node does."""
    c = Tree(23, GEOMS[geom], reqs, cuda_device, fp8=fp8)
    clean = _bits(c.step())
    sick = []  # (request, node): two in each, one of them the last but one
    for b, (p, t) in enumerate(reqs):
        for j in {t // 3, t - 2}:
            sick.append((b, j))
            page, slot = int(c.table[b, (p + j) // 16]), (p + j) % 16
            k, v = c.pools[0], c.pools[1]
            if fp8:
                k.view(torch.uint8)[page, :, slot] = 0x7F
                v.view(torch.uint8)[page, :, slot, ::3] = 0xFF
            else:
                k[page, :, slot] = float("inf")
                k[page, :, slot, 1] = float("nan")
                v[page, :, slot, 0::3] = float("inf")
                v[page, :, slot, 1::3] = float("nan")
    got = c.step()
    torch.cuda.synchronize()
    seen = np.zeros(int(c.cu_np[-1]), dtype=bool)
    for b, j in sick:
        for i in range(reqs[b][1]):
            seen[c.cu_np[b] + i] |= bool(c.mask_np[c.cu_np[b] + i] >> j & 1)
    assert seen.any() and not seen.all()
    assert torch.equal(_bits(got)[~seen], clean[~seen])
    assert not np.isfinite(bf16_to_f64(got)[seen]).all(axis=-1).any()
    assert c.ws.status() == 0


@pytest.mark.gpu
def test_infinite_value_rows_reach_those_that_see_them(cuda_device):
    """An infinite value is what the sum says: infinite in its column, and in no other, for the nodes that see the row."""
    reqs = [(700, 40)]
    c = Tree(24, GEOMS["16q8kv128"], reqs, cuda_device)
    clean = bf16_to_f64(c.step())
    p, j = 700, 3
    page, slot = int(c.table[0, (p + j) // 16]), (p + j) % 16
    c.pools[1][page, :, slot, 5] = -float("inf")
    got = bf16_to_f64(c.step())
    for i in range(40):
        want = clean[i].copy()
        if c.mask_np[i] >> j & 1:
            want[:, 5] = -np.inf
        assert np.array_equal(got[i][want != -np.inf], want[want != -np.inf]) or not (c.mask_np[i] >> j & 1)
        assert np.array_equal(np.isinf(got[i]), np.isinf(want))
        others = np.delete(got[i], 5, axis=1) - np.delete(want, 5, axis=1)
        # (the zero in the infinite value's place leaves the other columns' sums alone)
        assert (others == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("scale", [-0.05, 0.0, 1e-30, 2.0])
def test_any_scale(cuda_device, scale, fp8):
    c = Tree(25, GEOMS["12q4kv128"], [(130, 20), (0, 3)], cuda_device, fp8=fp8, masks="any")
    c.scale = scale
    c.step()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("power", [10, 20, 40])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_huge_scores_give_one_row(cuda_device, fp8, power):
    """Scores so far apart that one key takes all the weight: its value row, rounded once."""
    c = Tree(26, GEOMS["16q8kv128"], [(1000, 6), (200, 1)], cuda_device, fp8=fp8, q_size=2.0 ** power)
    c.step()
    torch.cuda.synchronize()
    got = bf16_to_f64(c.out)
    for b, (p, t) in enumerate(c.reqs):
        pages = c.table[b, : -(-(p + t) // 16)]
        flat = lambda x: x[pages].transpose(0, 2, 1, 3).reshape(-1, c.hkv, c.d)[: p + t]  # noqa: E731
        k, v = flat(c.k64), flat(c.v64)
        for i in range(t):
            q = bf16_to_f64(c.q[c.cu_np[b] + i])
            seen = np.array([True] * p + [bool(c.mask_np[c.cu_np[b] + i] >> j & 1) for j in range(t)])
            for h in range(c.hq):
                s = np.where(seen, k[:, h // 2] @ q[h], -np.inf) * c.scale
                order = np.argsort(s)
                # fp32 sums are off by at most (d + 8) 2^-24 of sum |q| |k|: take rows that are clear of it
                slack = (c.d + 8) * 2.0 ** -23 * c.scale * (np.abs(k[:, h // 2]) @ np.abs(q[h])).max()
                if s[order[-1]] - s[order[-2]] > slack + 40:
                    want = v[order[-1], h // 2]
                    assert (np.abs(got[c.cu_np[b] + i, h] - want) <= 2.0 ** -8 * np.abs(want) + 1e-12).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_rows_of_no_request_are_left(cuda_device, fp8):
    c = Tree(27, GEOMS["16q8kv128"], [(100, 5), (37, 0), (60, 3)], cuda_device, fp8=fp8)
    n = int(c.cu_np[-1])
    q = torch.cat([c.q, torch.full((4, *c.q.shape[1:]), float("nan"), dtype=torch.bfloat16, device=cuda_device)])
    out = torch.full_like(q, 3.5)
    mask = torch.cat([c.mask, torch.full((4,), -1, dtype=torch.int64, device=cuda_device)])
    c.step(q=q, out=out, tree_mask=mask)
    c.check(out[:n])
    assert (out[n:] == 3.5).all()
    # nothing to do: no rows, no requests, no nodes
    empty = q[:0].contiguous()
    c.step(q=empty, out=empty.clone(), tree_mask=mask[:0].contiguous(), cu_nodes=torch.zeros_like(c.cu))
    c.step(block_table=c.bt[:0].contiguous(), prefix_lens=c.prefix[:0].contiguous(), cu_nodes=c.cu[:1].contiguous())
    out.fill_(3.5)
    c.step(q=q, out=out, tree_mask=mask, cu_nodes=torch.zeros_like(c.cu))
    torch.cuda.synchronize()
    assert (out == 3.5).all() and c.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_bad_pages_and_lengths_are_reported(cuda_device, fp8):
    reqs = [(300, 5), (1000, 20), (37, 2), (2000, 9)]
    c = Tree(28, GEOMS["16q8kv128"], reqs, cuda_device, fp8=fp8)
    want = _bits(c.step())
    out_of_bounds = pkv.ERR_CODES["PKV_ERR_OUT_OF_BOUNDS"]

    def run(others, **kw):
        out = torch.full_like(c.out, 3.5)
        c.step(out=out, **kw)
        torch.cuda.synchronize()
        assert c.ws.status() == out_of_bounds
        with pytest.raises(pkv.PkvError):
            c.ws.check()
        assert c.ws.status() == 0
        for b in others:
            assert torch.equal(_bits(out)[c.cu_np[b]: c.cu_np[b + 1]], want[c.cu_np[b]: c.cu_np[b + 1]]), b
        return out

    table = c.table.copy()
    table[1, 3], table[3, 0] = c.pages, -1
    run([0, 2], block_table=i32(table, cuda_device))
    for b, p in ((1, -1), (1, c.bt.shape[1] * 16 - 19), (0, 2 ** 31 - 1)):
        prefix = np.array([p for p, _ in reqs])
        prefix[b] = p
        # (whole items or shares: where the others are cut may differ, so their bits may; the bound holds)
        out = torch.full_like(c.out, 3.5)
        c.step(out=out, prefix_lens=i32(prefix, cuda_device))
        torch.cuda.synchronize()
        assert c.ws.status() == out_of_bounds
        pkv.workspace_init(c.ws.tensor)
        c.check(out, only=[i for i in range(4) if i != b])
        assert (out[c.cu_np[b]: c.cu_np[b + 1]] == 3.5).all()
    for cu, bad in (([0, 5, 25, 24, 33], 2), ([0, 5, 25, 27, 99], 3), ([-1, 5, 25, 27, 36], 0)):
        out = torch.full_like(c.out, 3.5)
        c.step(out=out, cu_nodes=i32(cu, cuda_device))
        torch.cuda.synchronize()
        assert c.ws.status() == out_of_bounds
        pkv.workspace_init(c.ws.tensor)
        if cu[3] < cu[2]:
            out[cu[3]] = c.out[cu[3]]  # by this table row 24 belongs to requests 1 and 3: what it holds says nothing
        c.check(out, only=[b for b in range(2 if bad == 2 else 4) if b != bad])
    out = torch.full_like(c.out, 3.5)
    c.step(out=out, max_nodes=9)  # request 1 has 20
    torch.cuda.synchronize()
    assert c.ws.status() == out_of_bounds
    pkv.workspace_init(c.ws.tensor)
    c.check(out, only=[0, 2, 3])
    assert (out[5:25] == 3.5).all()
    c.check(c.step())


@pytest.mark.gpu
def test_captured_graphs_share_a_workspace(cuda_device):
    """Two captured calls of different sizes and caches on one workspace, replayed in turn with new inputs in place."""
    a = Tree(29, GEOMS["16q8kv128"], [(3000, 16), (700, 16), (40, 2)], cuda_device)
    b = Tree(30, GEOMS["14q2kv64"], [(12000, 40)], cuda_device, fp8=True)
    b.ws = a.ws
    side = torch.cuda.Stream()
    graphs = []
    for c in (a, b):
        with torch.cuda.stream(side):
            c.step()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.step()
            c.step()
        graphs.append(g)
    for turn in range(3):
        for c, g in zip((a, b), graphs):
            c.out.fill_(float("nan"))
            c.q.copy_(torch.randn(c.q.shape, device=cuda_device))
            g.replay()
            c.check()
    lens = [p for p, _ in a.reqs]
    a.reqs = [(p // 2, t) for p, t in a.reqs]  # shorter prefixes: other shares in the same graph
    a.set_masks([m for _, t in a.reqs for m in ancestors(np.random.default_rng(5), t)])
    a.prefix.copy_(i32([p for p, _ in a.reqs], cuda_device))
    assert lens != [p for p, _ in a.reqs]
    eager = Tree.step(a).clone()
    a.check()
    assert torch.isfinite(eager).all()


@pytest.mark.gpu
def test_two_streams_at_once_and_the_stream_argument(cuda_device):
    a = Tree(31, GEOMS["16q8kv128"], [(5000, 32), (900, 7)], cuda_device)
    b = Tree(32, GEOMS["32q32kv64"], [(600, 9)] * 6, cuda_device, fp8=True)
    want = [_bits(a.step()), _bits(b.step())]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        a.step(stream=s[0])
        b.step(stream=s[1])
    torch.cuda.synchronize()
    assert torch.equal(_bits(a.out), want[0]) and torch.equal(_bits(b.out), want[1])
    assert a.ws.status() == 0 and b.ws.status() == 0


@pytest.mark.gpu
def test_binding_refuses_bad_tensors(cuda_device):
    c = Tree(33, GEOMS["16q8kv128"], [(100, 4), (20, 3)], cuda_device)
    f = Tree(33, GEOMS["16q8kv128"], [(100, 4), (20, 3)], cuda_device, fp8=True)
    for x in (c, f):
        bad = [dict(q=x.q.float()), dict(q=x.q[:, :, :64]), dict(q=x.q[:, 0]), dict(out=x.out[:3]), dict(out=x.out.cpu()),
               dict(prefix_lens=x.prefix.long()), dict(prefix_lens=x.prefix[:1]), dict(cu_nodes=x.cu[:2]),
               dict(block_table=x.bt[:1]), dict(block_table=x.bt[0]), dict(tree_mask=x.mask.int()), dict(tree_mask=x.mask[:3]),
               dict(max_nodes=-1), dict(q=x.q.transpose(0, 1)), dict(q=None), dict(workspace=None), dict(scale="one")]
        for kw in bad:
            with pytest.raises((TypeError, ValueError, AttributeError, pkv.PkvError)):
                x.step(**kw)
        with pytest.raises(pkv.PkvError) as e:
            x.step(max_nodes=65)
        assert e.value.code == pkv.ERR_CODES["PKV_ERR_UNSUPPORTED"]
        with pytest.raises(pkv.PkvError) as e:
            x.step(workspace=pkv.Workspace(4096, cuda_device))
        assert e.value.code == pkv.ERR_CODES["PKV_ERR_WORKSPACE_TOO_SMALL"]
    with pytest.raises(TypeError):
        pkv.tree_attn(c.q, *f.pools[:2], c.bt, c.prefix, c.cu, c.mask, c.out, c.scale, 4, c.ws)
    with pytest.raises((TypeError, ValueError)):
        pkv.tree_attn_fp8(c.q, *f.pools[:2], None, c.bt, c.prefix, c.cu, c.mask, c.out, c.scale, 4, c.ws)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_pools_past_four_gigabytes(cuda_device, fp8):
    c = Tree(34, GEOMS["16q8kv128"], [(330, 12)], cuda_device, fp8=fp8)
    first = _bits(c.step())
    page_bytes = 16 * 128 * 8 * (1 if fp8 else 2)
    pages = (9 << 29) // page_bytes + 64  # 4.5 GiB
    at = np.linspace(0, pages - 1, c.pages).astype(np.int64)
    big = []
    for x in c.pools:
        y = torch.empty((pages, *x.shape[1:]), dtype=x.dtype, device=cuda_device)
        raw = (lambda z: z.view(torch.uint8)) if x.element_size() == 1 else (lambda z: z)
        raw(y)[torch.from_numpy(at).to(cuda_device)] = raw(x)
        big.append(y)
    c.pools = big
    c.bt = i32(np.where(c.table < c.pages, at[np.minimum(c.table, c.pages - 1)], c.table), cuda_device)
    assert torch.equal(_bits(c.step()), first) and c.ws.status() == 0


# ---------------------------------------------------------------------------------------------- a speculative step
@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64"])
def test_speculative_step(cuda_device, geom, fp8):
    """Three layers, three requests: the tree's rows appended at their depths, tree attention, the accepted nodes kept. The
    cache then holds, bit for bit, what appending the path token by token would have left, decode attention of every kept
    node agrees with its tree row, and a fork of each request goes on without touching its origin."""
    ensure_built()
    dev = cuda_device
    hq, hkv, d = GEOMS[geom]
    rng = np.random.default_rng(40)
    gen = torch.Generator().manual_seed(40)
    layers, reqs = 3, [(200, 12), (31, 7), (64, 20)]
    total = sum(t for _, t in reqs)
    width = 20
    pages = 3 * width + 8
    table = rng.permutation(pages)[: 3 * width].reshape(3, width)
    spare = [x for x in range(pages) if x not in table]
    parents, depth, masks = [], [], []
    for _, t in reqs:
        par = [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, t)]
        dep, seen = [], []
        for i, p in enumerate(par):
            dep.append(0 if p < 0 else dep[p] + 1)
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        parents.append(par)
        depth.append(dep)
        masks.append(seen)
    row = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(dev)  # noqa: E731
    q, k, v = row(layers, total, hq, d), row(layers, total, hkv, d), row(layers, total, hkv, d)
    cos_sin = pkv.rope_cos_sin(THETA, 512, d, dev)
    ws = pkv.Workspace(pkv.tree_workspace_bytes(3, 20, pages, hq, hkv, d), dev)
    dws = pkv.Workspace(pkv.decode_workspace_bytes(3, width, pages, hq, hkv, d), dev)
    raw = lambda x: x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)  # noqa: E731

    def empty_pools():
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        pools = [torch.zeros(layers, pages, hkv, 16, d, dtype=torch.uint8 if fp8 else kind, device=dev).view(kind)
                 for _ in range(2)]
        return pools + ([torch.full((layers, pages, hkv, 2, 16), 127, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)]
                        if fp8 else [])

    def append(pools, at, rows, positions, slots, q_out=None):
        kw = dict(q=q[at][rows].contiguous(), q_out=q_out) if q_out is not None else {}
        f = pkv.append_rope_fp8 if fp8 else pkv.append_rope
        f(k[at][rows].contiguous(), v[at][rows].contiguous(), i32(positions, dev), i32(slots, dev), cos_sin,
          *[x[at] for x in pools], dws, **kw)

    slot = lambda b, p: int(table[b, p // 16]) * 16 + p % 16  # noqa: E731
    # prefixes: rows of their own, the same in every run
    pk, pv = row(layers, 300, hkv, d), row(layers, 300, hkv, d)

    def prefill(pools):
        for at in range(layers):
            n = 0
            for b, (p, _) in enumerate(reqs):
                f = pkv.append_rope_fp8 if fp8 else pkv.append_rope
                f(pk[at, n: n + p].contiguous(), pv[at, n: n + p].contiguous(), i32(range(p), dev),
                  i32([slot(b, i) for i in range(p)], dev), cos_sin, *[x[at] for x in pools], dws)
                n += p

    cu = np.concatenate([[0], np.cumsum([t for _, t in reqs])])
    pos = [p + x for b, (p, _) in enumerate(reqs) for x in depth[b]]
    slots = [slot(b, p + i) for b, (p, t) in enumerate(reqs) for i in range(t)]
    bt, prefix = i32(table, dev), i32([p for p, _ in reqs], dev)
    mask = torch.from_numpy(np.array([m for s in masks for m in s], dtype=np.uint64).view(np.int64)).to(dev)

    pools = empty_pools()
    prefill(pools)
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    for at in range(layers):
        append(pools, at, slice(0, total), pos, slots, q_rot[at])
        (pkv.tree_attn_fp8 if fp8 else pkv.tree_attn)(q_rot[at], *[x[at] for x in pools], bt, prefix, i32(cu, dev), mask,
                                                      out[at], d ** -0.5, 20, ws)
    # the accepted path: from the deepest node up
    paths = []
    for b in range(3):
        i, path = int(np.argmax(depth[b])), []
        while i >= 0:
            path.append(i)
            i = parents[b][i]
        paths.append(path[::-1])
    most = max(len(p) for p in paths)
    path = np.full((3, most), -1)
    for b, p in enumerate(paths):
        path[b, : len(p)] = p
    pkv.keep_nodes(i32(path, dev), i32([len(p) for p in paths], dev), prefix, bt, *pools, workspace=dws)

    # token by token into another cache
    straight = empty_pools()
    prefill(straight)
    dec = torch.empty_like(q)
    for step in range(most):
        live = [b for b in range(3) if step < len(paths[b])]
        rows = [int(cu[b]) + paths[b][step] for b in live]
        lens = i32([reqs[b][0] + step + 1 for b in live], dev)
        for at in range(layers):
            append(straight, at, rows, [reqs[b][0] + step for b in live], [slot(b, reqs[b][0] + step) for b in live])
            o = torch.empty(len(live), hq, d, dtype=torch.bfloat16, device=dev)
            (pkv.decode_attn_fp8 if fp8 else pkv.decode_attn)(q_rot[at][rows].contiguous(), *[x[at] for x in straight],
                                                              bt[live].contiguous(), lens, o, d ** -0.5, dws)
            dec[at, rows] = o
    torch.cuda.synchronize()
    assert ws.status() == 0 and dws.status() == 0
    for b, (p, _) in enumerate(reqs):
        for x, y in zip(pools, straight):
            for i in range(p + len(paths[b])):
                page, s = int(table[b, i // 16]), i % 16
                sel = (lambda z: raw(z)[:, page, ..., s]) if x.shape[-1] == 16 and x.dim() == 5 and x.shape[-2] == 2 else (
                    lambda z: raw(z)[:, page, :, s])
                assert torch.equal(sel(x), sel(y)), (b, i)
        rows = [int(cu[b]) + i for i in paths[b]]
        got, want = bf16_to_f64(out[:, rows]), bf16_to_f64(dec[:, rows])
        # both are within their bounds of the exact sums; values are at most some 5 in size, weights sum to 1
        assert np.abs(got - want).max() <= 2 * 2.0 ** -8 * np.abs(want).max() + 2 * (2.0 ** -8 + 2.0 ** -10) * 6.0

    # forks: the last page of each request on a page of its own, then one more row there
    ends = [p + len(x) for (p, _), x in zip(reqs, paths)]
    last = [int(table[b, (n - 1) // 16]) for b, n in enumerate(ends)]
    before = [raw(x).clone() for x in pools]
    pkv.copy_pages(i32(last, dev), i32(spare[:3], dev), *pools, workspace=dws)
    for at in range(layers):
        append(pools, at, [0, 1, 2], ends, [spare[b] * 16 + n % 16 if n % 16 else -1 for b, n in enumerate(ends)])
    torch.cuda.synchronize()
    for x, y in zip(pools, before):
        assert torch.equal(raw(x)[:, last], y[:, last])
        for b, n in enumerate(ends):
            got, want = raw(x)[:, spare[b]], y[:, last[b]]
            keep = n % 16 or 16
            if x.shape[-1] == 16 and x.shape[-2] == 2:
                assert torch.equal(got[..., :keep], want[..., :keep])
            else:
                assert torch.equal(got[:, :, :keep], want[:, :, :keep])
