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
    assert call(pages=(1 << 27) - 1, seqs=1) == -2 and call(seqs=1024, pages=1 << 18) == -2
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
         "32q32kv64": (32, 32, 64), "8q1kv64": (8, 1, 64), "14q2kv64": (14, 2, 64)}


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
