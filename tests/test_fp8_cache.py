"""The 8-bit paged KV cache: decode attention over it and its expansion to bf16 pages, against float64 numpy over the
values that the cache stands for (tests/fp8_util.py; the bound's terms are in decode_bound), and a whole request served
from it (prompt chunks, then steps)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_decode_gb300 as pkv
from fp8_util import (NAN_CODE, attention64, cache_to, codes_of, decode_bound, dequantise, fp32_noise, quantise,
                      random_cache, rotate64)
from gpu_util import bits, ensure_built, i32
from paged_kv_decode_gb300 import _lib
from paged_kv_decode_gb300 import workloads as W
from paged_kv_decode_gb300.build import build_library
from parity import bf16_to_f64
from test_schedule import ShareMap, assign_share, piece_index, simulate


# ---------------------------------------------------------------------------------------------- CPU
def test_reference_format():
    """The references' format: every code's value quantises to itself, borders and ties as the definition says."""
    from fp8_util import CODE_VALUES, to_codes

    codes = np.array([c for c in range(256) if not np.isnan(CODE_VALUES[c])])
    assert np.array_equal(to_codes(CODE_VALUES[codes]), codes)
    assert np.array_equal(CODE_VALUES[[0x7E, 0x08, 0x01, 0x38]], [448.0, 2.0 ** -6, 2.0 ** -9, 1.0])
    assert np.array_equal(to_codes(np.array([464.0, 1e9, np.inf, 1.0625, 1.1875])), [0x7E, 0x7E, 0x7E, 0x38, 0x3A])
    # torch's own conversion agrees on its range
    x = torch.linspace(-448, 448, 20001)
    assert np.array_equal(to_codes(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    _, s = quantise(np.array([[448.0], [448.1], [224.0], [0.0], [1e-40], [3e38]]))
    assert s.tolist() == [127, 128, 126, 47, 47, 227]


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _lib.load()


def _desc(**kw):
    d = dict(num_q_heads=16, num_kv_heads=8, head_dim=128, page_size=16, num_pages=4)
    d.update(kw)
    return _lib.CacheDesc(**d)


def test_decode_host_argument_checks(lib):
    buf = ctypes.create_string_buffer(1024)
    p = (ctypes.addressof(buf) + 255) // 256 * 256

    def call(desc=_desc(), q=p, kp=p, vp=p, sc=p, bt=p, sl=p, out=p, batch=2, width=4, ws=p, nb=64):
        return lib.pkv_decode_attn_fp8(q, kp, vp, sc, bt, sl, out, 1.0, None,
                                       None if desc is None else ctypes.byref(desc), batch, width, ws, nb, 0)

    assert call(desc=None) == -1
    for bad in (_desc(head_dim=96), _desc(page_size=32), _desc(num_q_heads=36, num_kv_heads=4)):
        assert call(desc=bad) == -3
    assert call(batch=-1) == -2 and call(width=0) == -2 and call(width=(1 << 27) - 1, batch=1) == -2
    assert call(batch=1025) == -3
    assert call(batch=1024, width=1 << 18) == -2
    assert call(ws=None) == -1
    for name in ("q", "kp", "vp", "sc", "bt", "sl", "out"):
        assert call(**{name: None}) == -1, name
    for name in ("q", "kp", "vp", "sc", "out", "ws"):
        assert call(**{name: p + 8}) == -8, name
    assert call(batch=0) == 0


def test_decode_append_host_argument_checks(lib):
    buf = ctypes.create_string_buffer(1024)
    p = (ctypes.addressof(buf) + 255) // 256 * 256

    def call(desc=_desc(), q=p, k=p, v=p, kp=p, vp=p, sc=p, bt=p, sl=p, table=p, max_pos=8, qw=p, kw=p, eps=1e-6, out=p,
             batch=2, width=4, ws=p, nb=64):
        return lib.pkv_decode_append_attn_fp8(q, k, v, kp, vp, sc, bt, sl, table, max_pos, qw, kw, eps, out, 1.0, None,
                                              None if desc is None else ctypes.byref(desc), batch, width, ws, nb, 0)

    assert call(desc=None) == -1
    for bad in (_desc(head_dim=96), _desc(page_size=32), _desc(num_q_heads=36, num_kv_heads=4)):
        assert call(desc=bad) == -3
    assert call(batch=-1) == -2 and call(width=0) == -2 and call(width=(1 << 27) - 1, batch=1) == -2
    assert call(batch=1025) == -3 and call(batch=1024, width=1 << 18) == -2
    assert call(max_pos=0) == -2 and call(eps=-1.0) == -2 and call(eps=float("nan")) == -2
    assert call(ws=None) == -1
    for name in ("q", "k", "v", "kp", "vp", "sc", "bt", "sl", "out"):
        assert call(**{name: None}) == -1, name
    for name in ("q", "k", "v", "kp", "vp", "sc", "table", "qw", "kw", "out", "ws"):
        assert call(**{name: p + 8}) == -8, name
    assert call(batch=0) == 0


def test_expand_host_argument_checks(lib):
    buf = ctypes.create_string_buffer(1024)
    p = (ctypes.addressof(buf) + 255) // 256 * 256

    def call(desc=_desc(), kp=p, vp=p, sc=p, bt=p, sl=p, ko=p, vo=p, ot=p, seqs=2, width=4, out_pages=4, ws=None, nb=0):
        return lib.pkv_expand_fp8(kp, vp, sc, bt, sl, seqs, width, ko, vo, ot, out_pages,
                                  None if desc is None else ctypes.byref(desc), None, ws, nb)

    assert call(desc=None) == -1 and call(desc=_desc(head_dim=32)) == -3
    assert call(seqs=-1) == -2 and call(width=0) == -2 and call(out_pages=0) == -2 and call(width=(1 << 27) - 1, seqs=1) == -2
    for name in ("kp", "vp", "sc", "bt", "sl", "ko", "vo", "ot"):
        assert call(**{name: None}) == -1, name
    for name in ("kp", "vp", "sc", "ko", "vo"):
        assert call(**{name: p + 8}) == -8, name
    assert call(ws=p, nb=8) == -4
    assert call(seqs=0) == 0


class Units(ShareMap):
    """The share map of the 8-bit decode kernel: units of 32 tokens; shares of at least one unit and at most 2 sqrt(units
    of a pair) holders per pair; with the counted merge (one request, lam 0) a multiple of the pairs."""

    def __init__(self, seq_lens, grid, lam, hkv=8):
        super().__init__([(int(s) + 31) // 32 * 16 for s in seq_lens], grid, lam, hkv)  # as many pages as units
        self.n = min(grid, max(1, self.T))
        pairs = sum(1 for p in self.pages if p) * hkv
        if pairs:
            u = self.T // pairs
            h = int(2 * np.sqrt(np.float32(u)))
            if lam == 0:
                self.n = pairs * max(1, min(h, u, grid // pairs))
            elif pairs < 64:
                self.n = min(self.n, pairs * max(1, h))


UNIT_MIXES = [[37, 200], [1], [33], [32] * 7, [9000], [0, 700, 0, 33, 1, 2900, 0], list(range(1, 65)),
              [3, 8000, 5, 900], [1, 2, 3, 4, 5, 6, 7, 8, 4000], list(W.config_seq_lens(2))[:6]]


def _halves_finish(lo, hi, starts, halves, round_units, ring=3):
    """One CTA of `halves` producers with 4 consumers each: unit f of the share goes to consumer (f - lo) % (4 halves),
    a producer walks its own units 32 at a time in rounds, consumers meet at piece boundaries. True if all is read; a
    stage's previous use must lie in an earlier round (one barrier phase)."""
    cons = 4 * halves
    n = hi - lo
    piece = piece_index(lo, hi, starts) if n else []
    own = [[i for i in range(n) if i % cons // 4 == h] for h in range(halves)]
    rounds, round_of = [], {}
    for h in range(halves):
        rs = {}
        for o, i in enumerate(own[h]):
            rs.setdefault((o // 32, o % 32 // round_units), []).append(i)
        rounds.append([rs[k] for k in sorted(rs)])
        for r, lst in enumerate(rounds[h]):
            round_of.update({i: r for i in lst})
    back = cons * ring
    assert all(round_of[i - back] < round_of[i] for i in range(back, n))
    issued, done = [False] * n, [False] * n
    at, nxt, now = [0] * halves, [c for c in range(cons)], 0
    while not all(done):
        moved = False
        for h in range(halves):
            # a round goes out as a whole once all its stages are free
            while at[h] < len(rounds[h]) and all(i < back or done[i - back] for i in rounds[h][at[h]]):
                for i in rounds[h][at[h]]:
                    issued[i] = True
                at[h] += 1
                moved = True
        for c in range(cons):
            while nxt[c] < n and issued[nxt[c]] and piece[nxt[c]] == now:
                done[nxt[c]] = moved = True
                nxt[c] += cons
        if now < (piece[-1] if n else 0) and all(done[i] for i in range(n) if piece[i] == now):
            now += 1
            moved = True
        if not moved:
            return False
    return True


@pytest.mark.parametrize("lam", [0, 8])
@pytest.mark.parametrize("grid", [7, 152, 304])
def test_decode_shares_tile_the_units_and_cannot_deadlock(lam, grid):
    """Every unit in one share, the holders of a (request, KV head) consecutive and non-empty, and the copy schedule
    (rounds of 4 units) of every share finishes, with one producer and with two."""
    for lens in UNIT_MIXES:
        for hkv in (1, 8):
            if lam == 0 and (len(lens) > 1 or hkv > grid):
                continue  # the counted merge is for one request and few pairs
            sm = Units(lens, grid, lam, hkv)
            lo = [sm.lo(c) for c in range(sm.n + 1)]
            assert sm.n <= grid and lo[0] == 0 and lo[-1] == sm.T and all(a <= b for a, b in zip(lo, lo[1:]))
            starts = []
            for b, p in enumerate(sm.pages):
                for h in range(hkv if p else 0):
                    fs = sm.pref[b] + h * p
                    starts.append(fs)
                    for c in range(sm.cta(fs), sm.cta(fs + p - 1) + 1):
                        assert lo[c] < lo[c + 1] and lo[c] < fs + p and lo[c + 1] > fs
            for f in range(0, sm.T, 1 + sm.T // 200):
                assert lo[sm.cta(f)] <= f < lo[sm.cta(f) + 1]
            for c in range(sm.n):
                assert simulate(lo[c], lo[c + 1], starts, assign_share, 4)
            for c in range(0, sm.n, 1 + sm.n // 40):
                assert _halves_finish(lo[c], lo[c + 1], starts, 2, 4)


def test_two_producers_finish_on_one_share():
    """One CTA holding everything: runs of one-unit pieces, long pieces, and a mix."""
    for pieces in ([1] * 90, [200], [1, 1, 150, 1, 2, 3, 70, 1] * 2, list(range(1, 30))):
        starts = list(np.cumsum([0] + pieces[:-1]))
        assert _halves_finish(0, sum(pieces), starts, 2, 4) and _halves_finish(0, sum(pieces), starts, 1, 4)
    with pytest.raises(AssertionError):  # a round larger than a half's stages would wait on itself
        _halves_finish(0, 200, [0], 2, 16)


# ---------------------------------------------------------------------------------------------- GPU
def _poison(kc, vc, sc, bt, lens, poison_page):
    """Codes of slots that no request may read become NaN, their scales the NaN byte."""
    free = np.ones((kc.shape[0], 16), dtype=bool)
    for b, n in enumerate(lens):
        j = np.arange(n)
        free[bt[b, j // 16], j % 16] = False
    page, slot = free.nonzero()
    for pool in (kc, vc):
        pool[page, :, slot] = NAN_CODE
    sc[page, :, :, slot] = 0xFF


class Cache:
    """A seeded 8-bit cache of requests of given lengths on pages in random order, and its decode call."""

    def __init__(self, seed, geom, lens, dev, *, width=None, edit=None):
        ensure_built()
        self.hq, self.hkv, self.d = geom
        self.lens = np.asarray(lens, dtype=np.int32)
        rng = np.random.default_rng(seed)
        self.bt, pages, poison = W.place_pages(rng, self.lens, 16, True, 2, width)
        self.kc, self.vc, self.sc = random_cache(seed, pages, self.hkv, self.d)
        if edit is not None:
            edit(self)
        _poison(self.kc, self.vc, self.sc, self.bt, self.lens, poison)
        self.k, self.v, self.s = cache_to(self.kc, self.vc, self.sc, dev)
        gen = torch.Generator().manual_seed(seed)
        self.q = torch.randn(len(self.lens), self.hq, self.d, generator=gen).to(torch.bfloat16).to(dev)
        self.out = torch.full_like(self.q, float("nan"))
        self.block_table, self.seq_lens = i32(self.bt, dev), i32(self.lens, dev)
        self.scale = self.d ** -0.5
        self.ws = pkv.Workspace(pkv.decode_workspace_bytes(len(self.lens), self.bt.shape[1], pages, self.hq, self.hkv,
                                                           self.d), dev)

    def step(self, stream=None):
        pkv.decode_attn_fp8(self.q, self.k, self.v, self.s, self.block_table, self.seq_lens, self.out, self.scale,
                            self.ws, stream)
        return self.out

    def rows(self, b, which):
        n = int(self.lens[b])
        pages = self.bt[b, : (n + 15) // 16]
        x = dequantise((self.kc if which == 0 else self.vc)[pages], self.sc[pages][:, :, which])
        return x.transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.d)[:n]

    def check(self, what=""):
        got, q = bf16_to_f64(self.out), bf16_to_f64(self.q)
        for b, n in enumerate(self.lens):
            if n == 0:
                assert (got[b] == 0).all(), f"{what}: request {b} is empty"
                continue
            k, v = self.rows(b, 0), self.rows(b, 1)
            out, absolute, size = attention64(q[b], k, v, self.scale)
            tol = decode_bound(out, absolute, size, self.scale, self.d, int(n), np.abs(v).max())
            err = np.abs(got[b] - out)
            assert (err <= tol).all(), f"{what}: request {b} of {n}: {err.max()} over by {(err - tol).max()}"
        assert self.ws.status() == 0


GEOMS = {"16q8kv128": (16, 8, 128), "32q32kv128": (32, 32, 128), "28q4kv128": (28, 4, 128), "12q4kv128": (12, 4, 128),
         "64q8kv128": (64, 8, 128), "16q8kv64": (16, 8, 64), "8q1kv64": (8, 1, 64), "32q32kv64": (32, 32, 64),
         "14q2kv64": (14, 2, 64)}
LENS = {"none": [0], "all_empty": [0, 0, 0], "one": [1], "page": [16], "page_and_one": [17], "odd": [15, 0, 33, 1, 0], "tiny": [37, 200],
        "mixed": [3, 700, 0, 64, 1999, 16, 1, 310]}


@pytest.mark.gpu
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("geom", sorted(GEOMS))
def test_decode(cuda_device, geom, lens):
    c = Cache(21, GEOMS[geom], LENS[lens], cuda_device)
    c.step()
    torch.cuda.synchronize()
    c.check(f"{geom} {lens}")


@pytest.mark.gpu
@pytest.mark.parametrize("geom,lens,width", [("16q8kv128", W.config_seq_lens(2), None), ("16q8kv64", [3000] * 16, None),
                                             ("16q8kv128", [20000], None), ("16q8kv128", [900], 4096),
                                             ("8q1kv64", [9001], None), ("32q32kv64", W.config_seq_lens(5)[:12], 600),
                                             ("16q8kv64", [20000], None), ("8q1kv64", [9001], 9000),
                                             ("28q4kv128", [7000], 2100), ("28q4kv128", [5000, 40], None),
                                             ("8q1kv64", [9000, 15000], None), ("8q1kv64", [9000, 15000, 1], 3000),
                                             ("12q4kv128", [3, 0, 2500], 4000), ("64q8kv128", [17000], None),
                                             ("8q1kv64", [1], 9000)])
def test_decode_long_and_split(cuda_device, geom, lens, width):
    """Contexts split over many CTAs, by both merges and both launch shapes (a wide table takes the one-CTA shape)."""
    c = Cache(22, GEOMS[geom], lens, cuda_device, width=width)
    first = c.step().clone()
    torch.cuda.synchronize()
    c.check(geom)
    c.out.fill_(float("nan"))
    c.step()  # the workspace was left ready
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), c.out.view(torch.int16))
    assert c.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64"])
@pytest.mark.parametrize("batch", [70, 1024])
def test_decode_many_short_requests(cuda_device, geom, batch):
    """More (request, KV head) pairs than CTAs, many of one unit: shares of several whole pairs."""
    lens = np.random.default_rng(batch).integers(0, 70, size=batch)
    c = Cache(33, GEOMS[geom], lens, cuda_device)
    c.step()
    torch.cuda.synchronize()
    c.check(geom)


@pytest.mark.gpu
def test_decode_captured_graphs_share_a_workspace(cuda_device):
    """Two captured steps of different sizes on one workspace, replayed in turn on one stream, inputs changed between."""
    a = Cache(34, GEOMS["16q8kv128"], [700, 31, 0, 1200], cuda_device)
    b = Cache(35, GEOMS["16q8kv128"], [9000], cuda_device)
    big = a.ws if a.ws.nbytes >= b.ws.nbytes else b.ws
    a.ws = b.ws = big
    graphs = []
    for c in (a, b):
        c.step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.step()
        graphs.append(g)
    gen = torch.Generator().manual_seed(36)
    for _ in range(3):
        for c, g in ((a, graphs[0]), (b, graphs[1]), (a, graphs[0])):
            c.q.copy_(torch.randn(c.q.shape, generator=gen).to(torch.bfloat16))
            c.out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            c.check("replay")
    # fewer live requests than at capture: the rows behind them come back as zeros
    a.lens = np.array([700, 0, 0, 1200], dtype=np.int32)
    a.seq_lens.copy_(i32(a.lens, cuda_device))
    graphs[0].replay()
    torch.cuda.synchronize()
    a.check("a padded replay")


@pytest.mark.gpu
def test_decode_rows_of_very_different_scales(cuda_device):
    """Value rows of zeros (they count in the softmax's sum and add nothing), scales at both ends of their range, key
    rows of zeros, and a request whose rows are all zeros."""

    def edit(c):
        rng = np.random.default_rng(5)
        c.vc[:, :, 3] = 0
        c.sc[:, :, 1, 3] = 47
        c.kc[:, :, 5] = 0
        c.sc[:, :, 0, 5] = 47
        c.sc[:, :, 1, 7] = rng.integers(47, 140, size=c.sc.shape[:2])
        pages = c.bt[2, : 4]
        c.vc[pages] = 0
        c.sc[pages, :, 1] = 47
        c.kc[pages] = 0
        pages = c.bt[3, : 4]  # a request of huge values (2^100 448): finite outputs
        c.sc[pages, :, 1] = 227

    c = Cache(23, GEOMS["16q8kv128"], [1000, 37, 64, 50], cuda_device, edit=edit)
    c.step()
    torch.cuda.synchronize()
    c.check("scales")
    assert (bf16_to_f64(c.out)[2] == 0).all()


def _check_weighted(c, extra=None):
    """The outputs against float64, with fp16's smallest weight taken relative to the largest contribution of a row,
    p_j max|v_j|: a weight is held to 2^-25 where the largest p_j 2^e_j is 2^14, and 448 * 2^e_j is at most twice the
    row's largest value: n * 2^-38 * max_j p_j max|v_j|. extra(q, k): more error of the scores, [hq, 1]."""
    got, q64 = bf16_to_f64(c.out), bf16_to_f64(c.q)
    for b, n in enumerate(c.lens):
        k, v = c.rows(b, 0), c.rows(b, 1)
        out, absolute, size = attention64(q64[b], k, v, c.scale)
        s = np.einsum("hgd,nhd->hgn", q64[b].reshape(c.hkv, -1, c.d), k) * c.scale
        p = np.exp(s - s.max(axis=-1, keepdims=True))
        p /= p.sum(axis=-1, keepdims=True)
        top = (p * np.abs(v).max(axis=-1).T[:, None]).max(axis=-1).reshape(-1, 1)
        tol = decode_bound(out, absolute, size, c.scale, c.d, int(n), top)
        if extra is not None:
            tol += 2 * extra(q64[b], k) * absolute
        err = np.abs(got[b] - out)
        assert (err <= tol).all(), f"request {b} of {n}: {err.max()} over by {(err - tol).max()}"
    assert c.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("geom,lens", [("16q8kv128", [1000, 37, 64, 2900]), ("14q2kv64", [300, 20000]), ("8q1kv64", [9000])])
@pytest.mark.parametrize("exponent,key", [(40, 4), (100, 4), (60, 2), (32, 0), (36, 1), (-60, 4)])
def test_decode_value_rows_far_above_the_rest(cuda_device, geom, lens, exponent, key):
    """One value row of a request 2^exponent above the others, at a key of -2^key in every dimension that the (positive)
    queries score far below the others: it takes no precision from the rows that the softmax weighs."""

    def edit(c):
        for b, n in enumerate(c.lens):
            j = int(n) // 3
            page, slot = c.bt[b, j // 16], j % 16
            c.kc[page, :, slot], c.sc[page, :, 0, slot] = 0xB8, 127 + key  # e4m3 -1
            c.sc[page, :, 1, slot] = 127 + exponent - 8

    c = Cache(51, GEOMS[geom], lens, cuda_device, edit=edit)
    c.q = c.q.abs()
    c.step()
    torch.cuda.synchronize()
    _check_weighted(c)


@pytest.mark.gpu
def test_decode_exact_cases(cuda_device):
    """A context of one token gives that value row; identical keys give the mean, here of equal rows."""

    def edit(c):
        c.vc[:] = c.vc[0, 0, 0]
        c.sc[:, :, 1] = 120

    c = Cache(24, GEOMS["12q4kv128"], [1, 1, 16, 333], cuda_device, edit=edit)
    c.step()
    torch.cuda.synchronize()
    v = dequantise(c.vc[c.bt[0, 0], :, 0], c.sc[c.bt[0, 0], :, 1, 0])  # [hkv, d], exact in bf16
    got = bf16_to_f64(c.out)
    assert np.array_equal(got[0], np.repeat(v, 3, axis=0)) and np.array_equal(got[1], got[0])
    # equal rows: only the weights' fp16 roundings (2^-11) and the output's (2^-8) are left
    assert (np.abs(got[2:] - got[:1]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(got[:1])).all()


@pytest.mark.gpu
def test_decode_query_of_any_size(cuda_device):
    """Query rows of zeros, of one large value, tiny and huge ones (the scores' scale is taken out and put back)."""
    c = Cache(25, GEOMS["16q8kv128"], [300, 41], cuda_device)
    q = c.q.clone()
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -100
    q[0, 2, 1:] *= 2.0 ** -20
    q[1, 3] *= 2.0 ** 60
    q[1, 4, 5] = 1000.0
    c.q = q
    # huge scores: the first key by score takes everything; compare what float64 can say
    c.scale = c.scale * 2.0 ** -2
    c.step()
    torch.cuda.synchronize()
    got, q64 = bf16_to_f64(c.out), bf16_to_f64(q)
    for b, n in enumerate(c.lens):
        k, v = c.rows(b, 0), c.rows(b, 1)
        out, absolute, size = attention64(q64[b], k, v, c.scale)
        tol = decode_bound(out, absolute, size, c.scale, c.d, int(n), np.abs(v).max())
        assert (np.abs(got[b] - out) <= tol).all(), b


@pytest.mark.gpu
@pytest.mark.parametrize("power", [10, 20, 40, 80])
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64"])
def test_decode_huge_scores_give_one_row(cuda_device, geom, power):
    """Scores so far apart that the largest takes everything: its value row, to bf16's 2^-8 and the weight's 2^-11, for
    every head whose two largest scores differ by more than fp32's error in them and 64 (2^-92 in weight)."""
    c = Cache(53, GEOMS[geom], [700, 33, 1, 9000], cuda_device)
    c.q = c.q * 2.0 ** power
    c.step()
    torch.cuda.synchronize()
    got, q64 = bf16_to_f64(c.out), bf16_to_f64(c.q)
    clear = 0
    for b, n in enumerate(c.lens):
        k, v = c.rows(b, 0), c.rows(b, 1)
        for h in range(c.hq):
            g = h // (c.hq // c.hkv)
            s = k[:, g] @ q64[b, h] * c.scale
            at = np.argsort(s)
            error = (c.d + 8) * 2.0 ** -24 * c.scale * (np.abs(k[:, g]) @ np.abs(q64[b, h])).max()
            if n > 1 and s[at[-1]] - s[at[-2]] <= 64 + 2 * error:
                continue
            clear += 1
            want = v[at[-1], g]
            assert (np.abs(got[b, h] - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want)).all(), (b, h)
    assert clear >= 2 * c.hq and c.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64"])
@pytest.mark.parametrize("small", [-12, -20, -26])
def test_decode_query_with_one_large_dimension(cuda_device, geom, small):
    """Query rows of 2^small but for one dimension of 1, in which the keys are zero: the scores are the other dimensions'.
    A query value keeps bf16's 8 bits down to 2^-31 of its row's largest and is held to 2^-39 of it below."""

    def edit(c):
        c.kc[..., 3] = 0
        c.sc[:, :, 0] = c.sc[:, :, 0].astype(int) - small  # keys 2^-small larger

    c = Cache(52, GEOMS[geom], [700, 33, 1, 90], cuda_device, edit=edit)
    c.q = c.q * 2.0 ** small
    c.q[..., 3] = 1.0
    c.step()
    torch.cuda.synchronize()

    def lost(q, k):
        most = np.abs(q).max(axis=-1, keepdims=True) * 2.0 ** -39
        return c.scale * most * np.repeat(np.abs(k).sum(axis=-1).max(axis=0), c.hq // c.hkv)[:, None]

    _check_weighted(c, lost)


@pytest.mark.gpu
def test_decode_page_order_does_not_matter(cuda_device):
    c = Cache(26, GEOMS["16q8kv128"], [500, 77, 1200], cuda_device)
    a = c.step().clone()
    perm = np.random.default_rng(2).permutation(c.kc.shape[0])
    inv = np.argsort(perm).astype(np.int32)
    c.k, c.v, c.s = cache_to(c.kc[perm], c.vc[perm], c.sc[perm], cuda_device)
    c.block_table = i32(inv[c.bt], cuda_device)
    c.step()
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), c.out.view(torch.int16))


@pytest.mark.gpu
def test_decode_reports_bad_pages_and_lengths(cuda_device):
    c = Cache(27, GEOMS["16q8kv64"], [100, 60], cuda_device)
    for page, bad in ((2, c.kc.shape[0]), (3, -1), (6, 1 << 30)):  # first and second pages of their units
        bt = c.bt.copy()
        bt[0, page] = bad
        c.block_table = i32(bt, cuda_device)
        c.step()
        torch.cuda.synchronize()
        assert c.ws.status() == -7
        # the other request is not touched by it
        k, v, q = c.rows(1, 0), c.rows(1, 1), bf16_to_f64(c.q)[1]
        out, absolute, size = attention64(q, k, v, c.scale)
        tol = decode_bound(out, absolute, size, c.scale, c.d, 60, np.abs(v).max())
        assert (np.abs(bf16_to_f64(c.out)[1] - out) <= tol).all()
        pkv.workspace_init(c.ws.tensor)
    c.block_table = i32(c.bt, cuda_device)
    width = c.bt.shape[1]
    c.seq_lens = i32([100, width * 16 + 1], cuda_device)  # clamped to the table
    c.step()
    torch.cuda.synchronize()
    assert c.ws.status() == -7
    pkv.workspace_init(c.ws.tensor)
    c.seq_lens = i32(c.lens, cuda_device)
    c.step()
    torch.cuda.synchronize()
    c.check("after the errors")


@pytest.mark.gpu
def test_decode_on_two_streams_and_beside_the_bf16_call(cuda_device):
    """Two calls at once (a workspace each), then a bf16 decode call on one of the workspaces and back."""
    a = Cache(28, GEOMS["16q8kv128"], [2000, 31, 800], cuda_device)
    b = Cache(29, GEOMS["16q8kv128"], [64, 1500], cuda_device)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.step(s1)
        b.step(s2)
    torch.cuda.synchronize()
    a.check("stream 1")
    b.check("stream 2")
    case = W.decode_case(5, [2000, 31, 800], pending_append=False)
    out = torch.empty_like(case.q[0]).to(cuda_device)
    pkv.decode_attn(case.q[0].to(cuda_device), case.k_pages[0].to(cuda_device), case.v_pages[0].to(cuda_device),
                    i32(case.block_table, cuda_device), i32(case.seq_lens, cuda_device), out, a.scale, a.ws)
    a.out.fill_(float("nan"))
    a.step()
    torch.cuda.synchronize()
    a.check("after the bf16 call")
    want = oracle.decode(case.q[0], case.k_pages[0], case.v_pages[0], case.block_table, case.seq_lens, a.scale)
    assert np.abs(bf16_to_f64(out) - want).max() <= 1e-2


@pytest.mark.gpu
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64"])
@pytest.mark.parametrize("lens", [[1, 16, 17, 32, 33], [500, 0, 1777, 48, 64], [9000]])
def test_decode_early_prefetch_behind_the_append(cuda_device, geom, lens):
    """Ten layers of append and decode with early prefetch, replayed as one graph, with each layer's new rows over
    poison: the outputs and caches are the ones of the same calls without it, bit for bit."""
    hq, hkv, d = GEOMS[geom]
    layers, n = 10, len(lens)
    c = Cache(30, GEOMS[geom], lens, cuda_device)
    gen = torch.Generator().manual_seed(31)
    rows = torch.randn(layers, n, hq + 2 * hkv, d, generator=gen).to(torch.bfloat16).to(cuda_device)
    pos = i32(np.maximum(c.lens, 1) - 1, cuda_device)
    j = np.maximum(c.lens, 1) - 1
    slots = np.where(c.lens > 0, c.bt[np.arange(n), j // 16] * 16 + j % 16, -1)
    for b in range(n):  # the new rows' slots hold NaN until the append has run
        if slots[b] >= 0:
            c.k.view(torch.uint8)[slots[b] // 16, :, slots[b] % 16] = NAN_CODE
            c.s.view(torch.uint8)[slots[b] // 16, :, :, slots[b] % 16] = 0xFF
    slots = i32(slots, cuda_device)
    table = pkv.rope_cos_sin(1e6, int(c.lens.max()), d, cuda_device)

    def run(early):
        caches = [(c.k.clone(), c.v.clone(), c.s.clone()) for _ in range(layers)]
        q_rot = torch.empty(layers, n, hq, d, dtype=torch.bfloat16, device=cuda_device)
        outs = torch.full_like(q_rot, float("nan"))

        def chain():
            for i in range(layers):
                q, k, v = rows[i, :, :hq], rows[i, :, hq: hq + hkv], rows[i, :, hq + hkv:]
                pkv.append_rope_fp8(k, v, pos, slots, table, *caches[i], c.ws, q=q, q_out=q_rot[i])
                pkv.decode_attn_fp8(q_rot[i], *caches[i], c.block_table, c.seq_lens, outs[i], c.scale, c.ws,
                                    early_prefetch=early)

        if early:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                chain()
            graph.replay()
            graph.replay()
        else:
            chain()
        torch.cuda.synchronize()
        assert c.ws.status() == 0
        return outs, caches

    want, want_caches = run(False)
    got, got_caches = run(True)
    assert torch.isfinite(got.float()).all() and torch.equal(got.view(torch.int16), want.view(torch.int16))
    for a, b in zip(got_caches, want_caches):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


class Step:
    """Layers of new rows for a cache's requests, each layer with its own copy of the cache: the fused step, or the
    append and the attention as two calls."""

    def __init__(self, c, layers, seed, dev, *, rope, norm):
        self.c, self.layers = c, layers
        n, (hq, hkv, d) = len(c.lens), (c.hq, c.hkv, c.d)
        gen = torch.Generator().manual_seed(seed)
        draw = lambda heads: torch.randn(layers, n, heads, d, generator=gen).to(torch.bfloat16).to(dev)  # noqa: E731
        self.q, self.k, self.v = draw(hq), draw(hkv), draw(hkv)
        j = np.maximum(c.lens, 1) - 1
        slots = np.where(c.lens > 0, c.bt[np.arange(n), j // 16] * 16 + j % 16, -1)
        for b in range(n):  # the new rows' slots hold NaN until a call has written them
            if slots[b] >= 0:
                c.k.view(torch.uint8)[slots[b] // 16, :, slots[b] % 16] = NAN_CODE
                c.v.view(torch.uint8)[slots[b] // 16, :, slots[b] % 16] = NAN_CODE
                c.s.view(torch.uint8)[slots[b] // 16, :, :, slots[b] % 16] = 0xFF
        self.pos, self.slots = i32(j, dev), i32(slots, dev)
        self.table = pkv.rope_cos_sin(1e6, max(1, int(c.lens.max())), d, dev) if rope else None
        w = (1 + 0.2 * torch.randn(2, d, generator=gen)).to(torch.bfloat16).to(dev)
        self.qw, self.kw = (w[0].contiguous() if "q" in norm else None), (w[1].contiguous() if "k" in norm else None)
        self.caches = lambda: [(c.k.clone(), c.v.clone(), c.s.clone()) for _ in range(layers)]

    def two_calls(self, caches, outs):
        c = self.c
        q = torch.empty_like(self.q[0])
        for i in range(self.layers):
            pkv.append_rope_fp8(self.k[i], self.v[i], self.pos, self.slots, self.table, *caches[i], c.ws, q=self.q[i],
                                q_out=q, q_weight=self.qw, k_weight=self.kw)
            pkv.decode_attn_fp8(q, *caches[i], c.block_table, c.seq_lens, outs[i], c.scale, c.ws)

    def fused(self, caches, outs, early):
        c = self.c
        for i in range(self.layers):
            pkv.decode_append_attn_fp8(self.q[i], self.k[i], self.v[i], *caches[i], c.block_table, c.seq_lens, self.table,
                                       outs[i], c.scale, c.ws, q_weight=self.qw, k_weight=self.kw, early_prefetch=early)


STEP_LENS = [[1, 16, 17, 32, 33], [500, 0, 1777, 48, 64], [9000], [3, 700, 31, 32, 1999, 15, 1, 310, 5, 6, 7, 8, 40, 900]]


@pytest.mark.gpu
@pytest.mark.parametrize("rope,norm", [(True, "qk"), (True, ""), (False, "k"), (False, "")])
@pytest.mark.parametrize("lens", STEP_LENS, ids=str)
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64", "28q4kv128", "64q8kv128", "8q1kv64"])
def test_fused_step_has_the_two_calls_bits(cuda_device, geom, lens, rope, norm):
    """Outputs, rows and scales of the fused step, eager and as a replayed chain of layers with early prefetch."""
    c = Cache(40, GEOMS[geom], lens, cuda_device, width=2500 if lens == [9000] else None)
    st = Step(c, 3, 41, cuda_device, rope=rope, norm=norm)
    want, want_caches = torch.full_like(st.q, float("nan")), st.caches()
    st.two_calls(want_caches, want)
    got, got_caches = torch.full_like(st.q, float("nan")), st.caches()
    st.fused(got_caches, got, False)
    chain, chain_caches = torch.full_like(st.q, float("nan")), st.caches()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.fused(chain_caches, chain, True)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert c.ws.status() == 0
    assert torch.isfinite(want.float()).all()
    for out, caches in ((got, got_caches), (chain, chain_caches)):
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        for a, b in zip(caches, want_caches):
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.gpu
def test_fused_step_against_float64(cuda_device):
    """The fused step's outputs against float64 over the rows that it left in the cache."""
    c = Cache(42, GEOMS["16q8kv128"], [333, 1, 90, 0, 1600], cuda_device)
    st = Step(c, 1, 43, cuda_device, rope=True, norm="qk")
    caches = st.caches()
    out = torch.full_like(st.q, float("nan"))
    st.fused(caches, out, False)
    torch.cuda.synchronize()
    c.kc, c.vc, c.sc = (codes_of(x) for x in caches[0])
    table = bf16_to_f64(st.table)
    got = bf16_to_f64(out)[0]
    for b, n in enumerate(c.lens):
        if n == 0:
            assert (got[b] == 0).all()
            continue
        cs = table[n - 1:n]
        y, size = rotate64(bf16_to_f64(st.q[0, b:b + 1]), bf16_to_f64(st.qw), cs, 1e-6)
        k, v = c.rows(b, 0), c.rows(b, 1)
        yk, _ = rotate64(bf16_to_f64(st.k[0, b:b + 1]), bf16_to_f64(st.kw), cs, 1e-6)
        top = np.abs(yk).max(axis=-1, keepdims=True)
        # half an e4m3 step (2^-4, or 2^-10 of a scale of at most top / 224), with room for fp32
        assert (np.abs(k[n - 1] - yk[0]) <= np.maximum(2.0 ** -4 * np.abs(yk[0]), 2.0 ** -10 / 224 * top[0]) * 1.001).all()
        out64, absolute, qk = attention64(y[0], k, v, c.scale)
        # the query's rounding to bf16 moves a score by at most 2^-8 of scale * sum |q||k|
        tol = decode_bound(out64, absolute, qk, c.scale, c.d, int(n), np.abs(v).max())
        tol += 2 * 2.0 ** -8 * c.scale * qk[:, None] * absolute
        assert (np.abs(got[b] - out64) <= tol).all(), b


@pytest.mark.gpu
def test_fused_step_reports_and_refuses(cuda_device):
    c = Cache(44, GEOMS["16q8kv128"], [40, 100, 7], cuda_device)
    st = Step(c, 1, 45, cuda_device, rope=True, norm="qk")
    caches, out = st.caches(), torch.empty_like(st.q)
    # a table that is too short: reported, clamped to its last row
    short = st.table[:60].contiguous()
    call = lambda **kw: pkv.decode_append_attn_fp8(  # noqa: E731
        **{**dict(q=st.q[0], k_new=st.k[0], v_new=st.v[0], k_pages=caches[0][0], v_pages=caches[0][1],
                  kv_scales=caches[0][2], block_table=c.block_table, seq_lens=c.seq_lens, cos_sin=st.table, out=out[0],
                  scale=c.scale, workspace=c.ws, q_weight=st.qw, k_weight=st.kw), **kw})
    call(cos_sin=short)
    torch.cuda.synchronize()
    assert c.ws.status() == -7
    pkv.workspace_init(c.ws.tensor)
    # the new row's page outside the pool: nothing is written there, the others are served
    caches = st.caches()
    before = [x.clone() for x in caches[0]]
    bt = c.bt.copy()
    bt[1, 6] = c.kc.shape[0]  # request 1's last page (100 tokens)
    call(k_pages=caches[0][0], v_pages=caches[0][1], kv_scales=caches[0][2], block_table=i32(bt, cuda_device))
    torch.cuda.synchronize()
    assert c.ws.status() == -7
    page = c.bt[1, 6]
    for x, y in zip(caches[0], before):
        assert torch.equal(x.view(torch.uint8)[page], y.view(torch.uint8)[page])
        assert not torch.equal(x.view(torch.uint8)[c.bt[0, 2]], y.view(torch.uint8)[c.bt[0, 2]])
    pkv.workspace_init(c.ws.tensor)
    for bad, error in ((dict(k_new=st.k[0].float()), TypeError), (dict(k_new=st.k[0][:2]), ValueError),
                       (dict(v_new=st.v[0][:, :4].contiguous()), ValueError), (dict(q=st.q[0][:2]), ValueError),
                       (dict(cos_sin=st.table[:, :64].contiguous()), ValueError), (dict(cos_sin=st.table[:0]), ValueError),
                       (dict(k_weight=st.kw[:64].contiguous()), ValueError), (dict(k_new=None), ValueError),
                       (dict(workspace=pkv.Workspace(256, cuda_device)), pkv.PkvError), (dict(eps=-1.0), pkv.PkvError)):
        with pytest.raises(error):
            call(**bad)
    call()
    torch.cuda.synchronize()
    assert c.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64", "12q4kv128"])
@pytest.mark.parametrize("lens", [[1], [16, 0, 17], [200, 37, 1000]])
def test_expand_is_exact(cuda_device, geom, lens):
    c = Cache(31, GEOMS[geom], lens, cuda_device)
    s, w = c.bt.shape
    pages = s * w + 3
    out_bt = np.random.default_rng(3).permutation(pages)[: s * w].reshape(s, w).astype(np.int32)
    full = lambda: torch.full((pages, c.hkv, 16, c.d), 0x4321, dtype=torch.int16, device=cuda_device).view(  # noqa: E731
        torch.bfloat16)
    ko, vo = full(), full()
    pkv.expand_fp8(c.k, c.v, c.s, c.block_table, c.seq_lens, ko, vo, i32(out_bt, cuda_device), c.ws)
    torch.cuda.synchronize()
    for which, got in ((0, ko), (1, vo)):
        want = full()
        wn = want.cpu()
        for b, n in enumerate(c.lens):
            x = torch.from_numpy(c.rows(b, which)).to(torch.bfloat16)  # [n, hkv, d], exact
            j = np.arange(n)
            wn[out_bt[b, j // 16], :, j % 16] = x
        assert np.array_equal(bits(got), bits(wn))
    assert c.ws.status() == 0


@pytest.mark.gpu
def test_binding_refuses_bad_tensors(cuda_device):
    c = Cache(37, GEOMS["16q8kv128"], [40, 20], cuda_device)
    ok = dict(q=c.q, k_pages=c.k, v_pages=c.v, kv_scales=c.s, block_table=c.block_table, seq_lens=c.seq_lens, out=c.out,
              scale=c.scale, workspace=c.ws)
    pkv.decode_attn_fp8(**ok)
    for bad, error in ((dict(q=c.q.float()), TypeError), (dict(k_pages=c.k.view(torch.uint8)), TypeError),
                       (dict(kv_scales=c.s.view(torch.uint8)), TypeError), (dict(v_pages=c.v[:-1]), ValueError),
                       (dict(kv_scales=c.s[:, :, :, :8].contiguous()), ValueError), (dict(out=c.out[:1]), ValueError),
                       (dict(q=c.q[:, :, :64].contiguous()), ValueError), (dict(q=c.q.transpose(0, 1)), ValueError),
                       (dict(seq_lens=c.seq_lens[:1]), ValueError), (dict(seq_lens=c.seq_lens.long()), TypeError),
                       (dict(block_table=c.block_table[:1]), ValueError), (dict(block_table=c.block_table[0]), ValueError),
                       (dict(q=c.q.cpu()), ValueError), (dict(out=None), ValueError),
                       (dict(workspace=pkv.Workspace(256, cuda_device)), pkv.PkvError),
                       (dict(workspace=None), pkv.PkvError)):
        with pytest.raises(error):
            pkv.decode_attn_fp8(**{**ok, **bad})
    pages = c.bt.size
    stage = torch.zeros(pages, 8, 16, 128, dtype=torch.bfloat16, device=cuda_device)
    ident = i32(np.arange(pages).reshape(c.bt.shape), cuda_device)
    ok = dict(k_pages=c.k, v_pages=c.v, kv_scales=c.s, block_table=c.block_table, seq_lens=c.seq_lens, k_out=stage,
              v_out=stage.clone(), out_block_table=ident)
    pkv.expand_fp8(**ok)
    for bad, error in ((dict(k_out=stage.float()), TypeError), (dict(k_out=stage[:1]), ValueError),
                       (dict(v_out=stage[:, :4].contiguous()), ValueError), (dict(out_block_table=ident[:1]), ValueError),
                       (dict(out_block_table=ident.long()), TypeError), (dict(seq_lens=c.seq_lens[:1]), ValueError)):
        with pytest.raises(error):
            pkv.expand_fp8(**{**ok, **bad})
    torch.cuda.synchronize()
    assert c.ws.status() == 0


@pytest.mark.gpu
def test_expand_reports_bad_pages(cuda_device):
    c = Cache(32, GEOMS["16q8kv128"], [40, 40], cuda_device)
    s, w = c.bt.shape
    ident = np.arange(s * w).reshape(s, w).astype(np.int32)
    for edit_src, page in ((True, c.kc.shape[0]), (True, -1), (False, s * w), (False, -2)):
        bt, ot = c.bt.copy(), ident.copy()
        (bt if edit_src else ot)[1, 1] = page
        ko = torch.zeros(s * w, c.hkv, 16, c.d, dtype=torch.bfloat16, device=cuda_device)
        vo = torch.zeros_like(ko)
        pkv.workspace_init(c.ws.tensor)
        pkv.expand_fp8(c.k, c.v, c.s, i32(bt, cuda_device), c.seq_lens, ko, vo, i32(ot, cuda_device), c.ws)
        torch.cuda.synchronize()
        assert c.ws.status() == -7
        assert (ko[ident[1, 1]] == 0).all() and (vo[ident[1, 1]] == 0).all()
        want = torch.from_numpy(c.rows(1, 0)[32:40]).to(torch.bfloat16)
        assert torch.equal(ko[ident[1, 2], :, :8].cpu().transpose(0, 1), want)
    pkv.workspace_init(c.ws.tensor)


@pytest.mark.gpu
def test_pools_past_four_gigabytes(cuda_device):
    """Pages whose byte offsets pass 2^32: append, decode and expansion at the pool's end (uninitialised elsewhere)."""
    ensure_built()
    hq, hkv, d, pages = 16, 8, 128, 270000
    k = torch.empty(pages, hkv, 16, d, dtype=torch.uint8, device=cuda_device).view(torch.float8_e4m3fn)
    v = torch.empty_like(k)
    s = torch.empty(pages, hkv, 2, 16, dtype=torch.uint8, device=cuda_device).view(torch.float8_e8m0fnu)
    assert k.numel() > 1 << 32
    n = 50
    gen = torch.Generator().manual_seed(9)
    rows = torch.randn(2, n, hkv, d, generator=gen).to(torch.bfloat16)
    bt = np.array([[pages - 1, pages - 7, 263000, pages - 2]], dtype=np.int32)
    j = np.arange(n)
    ws = pkv.Workspace(pkv.decode_workspace_bytes(1, 4), cuda_device)
    pkv.append_rope_fp8(rows[0].to(cuda_device), rows[1].to(cuda_device), None,
                        i32(bt[0, j // 16] * 16 + j % 16, cuda_device), None, k, v, s, ws)
    q = torch.randn(1, hq, d, generator=gen).to(torch.bfloat16).to(cuda_device)
    out = torch.empty_like(q)
    pkv.decode_attn_fp8(q, k, v, s, i32(bt, cuda_device), i32([n], cuda_device), out, d ** -0.5, ws)
    ko = torch.zeros(4, hkv, 16, d, dtype=torch.bfloat16, device=cuda_device)
    vo = torch.zeros_like(ko)
    pkv.expand_fp8(k, v, s, i32(bt, cuda_device), i32([n], cuda_device), ko, vo, i32([[3, 1, 0, 2]], cuda_device), ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    k64, v64 = (dequantise(*quantise(bf16_to_f64(r))) for r in rows)
    want, absolute, size = attention64(bf16_to_f64(q)[0], k64, v64, d ** -0.5)
    tol = decode_bound(want, absolute, size, d ** -0.5, d, n, np.abs(v64).max())
    assert (np.abs(bf16_to_f64(out)[0] - want) <= tol).all()
    got = bf16_to_f64(vo)[[3, 1, 0, 2]].transpose(0, 2, 1, 3).reshape(-1, hkv, d)
    assert np.array_equal(got[:n], v64) and (got[n:] == 0).all()


@pytest.mark.gpu
def test_a_request_served_from_the_8bit_cache(cuda_device):
    """A prompt in two chunks, then three steps beside a second request: norms, rotation, 8-bit append, expansion and
    chunked prefill, then append and decode attention captured in a graph and replayed. Everything against float64 over
    the rows that the cache holds, which are themselves checked against float64 rows."""
    ensure_built()
    dev = cuda_device
    hq, hkv, d, eps = 16, 8, 128, 1e-6
    scale = d ** -0.5
    gen = torch.Generator().manual_seed(41)
    rng = np.random.default_rng(41)
    lens0, chunks = [300, 77], [170, 130]  # request 0 is prefilled here in two chunks, request 1 is there already
    steps, width = 3, 32
    bt = rng.permutation(2 * width).reshape(2, width).astype(np.int32)
    pages = 2 * width
    kp, vp, sc = (torch.zeros(pages, hkv, 16, d, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                  torch.zeros(pages, hkv, 16, d, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                  torch.zeros(pages, hkv, 2, 16, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu))
    table = pkv.rope_cos_sin(1e6, 512, d, dev)
    table64 = bf16_to_f64(table)
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=gen)).to(torch.bfloat16).to(dev) for _ in range(2))
    status = pkv.Workspace(pkv.PKV_STATUS_BYTES, dev)
    slots_of = lambda b, pos: bt[b, pos // 16] * 16 + pos % 16  # noqa: E731
    project = lambda n: torch.randn(n, (hq + 2 * hkv) * d, generator=gen).to(torch.bfloat16).to(dev)  # noqa: E731

    def split(x):
        n = x.shape[0]
        return (x[:, : hq * d].view(n, hq, d), x[:, hq * d: (hq + hkv) * d].view(n, hkv, d),
                x[:, (hq + hkv) * d:].view(n, hkv, d))

    def cached(b, n):
        """Rows 0 .. n - 1 of request b as the cache holds them (float64), K and V."""
        j = np.arange(n)
        page, slot = bt[b, j // 16], j % 16
        s = codes_of(sc)[page, :, :, slot]
        return (dequantise(codes_of(kp)[page, :, slot], s[:, :, 0]), dequantise(codes_of(vp)[page, :, slot], s[:, :, 1]))

    def check_rows(b, pos, k, v):
        y, size = rotate64(bf16_to_f64(k), bf16_to_f64(kw), table64[pos], eps)
        n = int(pos.max()) + 1
        ck, cv = (x[pos] for x in cached(b, n))
        top = np.abs(y).max(axis=-1, keepdims=True)
        # half an e4m3 step: 2^-4, or 2^-10 of a scale that is at most top / 224
        tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 / 224 * top * (1 + 2.0 ** -10)) + fp32_noise(d, size)
        assert (np.abs(ck - y) <= tol * (1 + 2.0 ** -20)).all()
        assert np.array_equal(cv, dequantise(*quantise(bf16_to_f64(v))))

    # request 1's prompt: rows in the cache by one append without query rows
    x1 = project(lens0[1])
    _, k, v = split(x1)
    pos = np.arange(lens0[1])
    pkv.append_rope_fp8(k, v, i32(pos, dev), i32(slots_of(1, pos), dev), table, kp, vp, sc, status, k_weight=kw)
    # request 0: two chunks
    stage_k = torch.full((width, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=dev)
    stage_v = torch.full_like(stage_k, float("nan"))
    ident = i32(np.arange(width)[None], dev)
    at = 0
    for n in chunks:
        x = project(n)
        q, k, v = split(x)
        pos = np.arange(at, at + n)
        q_rot = torch.empty(n, hq, d, dtype=torch.bfloat16, device=dev)
        pkv.append_rope_fp8(k, v, i32(pos, dev), i32(slots_of(0, pos), dev), table, kp, vp, sc, status, q=q, q_out=q_rot,
                            q_weight=qw, k_weight=kw)
        pkv.expand_fp8(kp, vp, sc, i32(bt[:1], dev), i32([at + n], dev), stage_k, stage_v, ident, status)
        ws = pkv.Workspace(pkv.prefill_workspace_bytes(1, n), dev)
        out = torch.empty_like(q_rot)
        pkv.prefill_chunk_attn(q_rot, stage_k, stage_v, ident, i32([at], dev), i32([0, n], dev), out, scale, n, ws)
        torch.cuda.synchronize()
        check_rows(0, pos, k, v)
        ck, cv = cached(0, at + n)
        got, q64 = bf16_to_f64(out), bf16_to_f64(q_rot)
        for i in list(range(0, n, 37)) + [n - 1]:
            want, absolute, size = attention64(q64[i], ck[: at + i + 1], cv[: at + i + 1], scale)
            # prefill rounds the softmax weights to bf16: 2^-8 in the place of decode's 2^-11
            tol = decode_bound(want, absolute, size, scale, d, at + i + 1, np.abs(cv).max()) + 2.0 ** -8 * absolute
            assert (np.abs(got[i] - want) <= tol).all(), (at, i)
        at += n
        assert ws.status() == 0
    # steps of both requests, one graph
    qkv = torch.zeros(2, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device=dev)
    q, k, v = split(qkv)
    q_rot = torch.empty(2, hq, d, dtype=torch.bfloat16, device=dev)
    out = torch.empty_like(q_rot)
    pos_d, slot_d, len_d = i32([0, 0], dev), i32([-1, -1], dev), i32([1, 1], dev)
    table_d = i32(bt, dev)
    ws = pkv.Workspace(pkv.decode_workspace_bytes(2, width), dev)

    def step():
        pkv.append_rope_fp8(k, v, pos_d, slot_d, table, kp, vp, sc, ws, q=q, q_out=q_rot, q_weight=qw, k_weight=kw)
        pkv.decode_attn_fp8(q_rot, kp, vp, sc, table_d, len_d, out, scale, ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # slots -1: nothing is appended
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = list(lens0)
    for i in range(steps):
        qkv.copy_(project(2))
        p = np.array(lens)
        pos_d.copy_(i32(p, dev))
        slot_d.copy_(i32([slots_of(b, p[b]) for b in range(2)], dev))
        len_d.copy_(i32(p + 1, dev))
        graph.replay()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        got, q64 = bf16_to_f64(out), bf16_to_f64(q_rot)
        for b in range(2):
            check_rows(b, np.array([lens[b] - 1]), k[b:b + 1], v[b:b + 1])
            ck, cv = cached(b, lens[b])
            want, absolute, size = attention64(q64[b], ck, cv, scale)
            tol = decode_bound(want, absolute, size, scale, d, lens[b], np.abs(cv).max())
            assert (np.abs(got[b] - want) <= tol).all(), (i, b)
    assert ws.status() == 0 and status.status() == 0
