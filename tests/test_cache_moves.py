"""Rows and pages that move within the paged cache: keep_nodes and copy_pages against plain numpy, bit for bit, in bf16 and
8-bit pools of one layer, of stacked layers and of lists of layers; what a call does not name stays as it was."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_decode_gb300 as pkv
from gpu_util import ensure_built, i32
from paged_kv_decode_gb300 import _lib
from paged_kv_decode_gb300.build import build_library


# ---------------------------------------------------------------------------------------------- CPU: refusals
@pytest.fixture(scope="module")
def lib():
    build_library()
    return _lib.load()


def _desc(**kw):
    d = dict(num_q_heads=8, num_kv_heads=8, head_dim=128, page_size=16, num_pages=4)
    d.update(kw)
    return _lib.CacheDesc(**d)


def _array(*p):
    return (ctypes.c_void_p * len(p))(*p)


@pytest.mark.parametrize("op", ["keep", "copy"])
def test_host_argument_checks(lib, op):
    buf = ctypes.create_string_buffer(1024)
    p = (ctypes.addressof(buf) + 255) // 256 * 256  # never dereferenced: every call below ends on the host
    good = _array(p, p, p)

    def call(desc=_desc(), a=p, b=p, prefix=p, bt=p, n=2, most=4, pages=4, kp=good, vp=good, sc=None, layers=3, ws=None, nb=0):
        d = None if desc is None else ctypes.byref(desc)
        if op == "keep":
            return lib.pkv_keep_nodes(a, b, prefix, bt, n, most, pages, kp, vp, sc, layers, d, None, ws, nb)
        return lib.pkv_copy_pages(a, b, n, kp, vp, sc, layers, d, None, ws, nb)

    assert call(desc=None) == -1
    for bad in (_desc(head_dim=96), _desc(page_size=32), _desc(num_q_heads=36, num_kv_heads=4), _desc(num_q_heads=20)):
        assert call(desc=bad) == -3
    assert call(desc=_desc(num_pages=0)) == -2
    assert call(n=-1) == -2 and call(layers=-1) == -2
    assert call(ws=p, nb=64) == -4
    assert call(n=0) == 0 and call(layers=0) == 0  # nothing to do, no device
    names = ("a", "b", "kp", "vp") + (("prefix", "bt") if op == "keep" else ())
    for name in names:
        assert call(**{name: None}) == -1, name
    assert call(kp=_array(p, None, p)) == -1 and call(vp=_array(p, p, None)) == -1 and call(sc=_array(p, None, p)) == -1
    assert call(kp=_array(p, p, p + 8)) == -8 and call(vp=_array(p + 4, p, p)) == -8 and call(sc=_array(p, p + 8, p)) == -8
    if op == "keep":
        assert call(most=-1) == -2 and call(pages=0) == -2 and call(pages=1 << 27) == -2
        assert call(n=1 << 20, pages=1 << 12) == -2
        assert call(most=65) == -3
        assert call(most=0) == 0


# ---------------------------------------------------------------------------------------------- GPU
class Pools:
    """Random bytes as the pools of some layers, and their copies as raw numpy [layers, pages, hkv, 16, ...]."""

    def __init__(self, seed, layers, pages, hkv, d, fp8, dev):
        ensure_built()
        rng = np.random.default_rng(seed)
        self.fp8, self.dev = fp8, dev
        shape = (layers, pages, hkv, 16, d)
        kind = np.uint8 if fp8 else np.int16
        draw = lambda s: rng.integers(np.iinfo(kind).min, np.iinfo(kind).max, size=s, endpoint=True, dtype=kind)  # noqa: E731
        self.raw = [draw(shape), draw(shape)]
        types = [torch.float8_e4m3fn if fp8 else torch.bfloat16] * 2
        if fp8:
            self.raw.append(draw((layers, pages, hkv, 2, 16)))
            types.append(torch.float8_e8m0fnu)
        self.t = [torch.from_numpy(r.copy()).to(dev).view(t) for r, t in zip(self.raw, types)]
        self.ws = pkv.Workspace(pkv.PKV_STATUS_BYTES, dev)

    def given(self, how):
        """The pools as a call takes them: stacked, a list, or the first layer alone."""
        form = {"stacked": lambda x: x, "list": list, "tuple": tuple, "one": lambda x: x[0]}[how]
        return [form(x) for x in self.t]

    def same(self, layers=None):
        torch.cuda.synchronize()
        for t, r in zip(self.t, self.raw):
            got = t.view(torch.uint8 if self.fp8 else torch.int16).cpu().numpy()
            assert np.array_equal(got, r)

    def move(self, pairs, layers=None):
        """The raw copies with row (page, slot) <- (page, slot) carried out, all read first."""
        for i, r in enumerate(self.raw):
            x = r if i < 2 else r.swapaxes(-1, -2)  # scales: rows last
            old = x.copy()
            for (p, s), (fp, fs) in pairs:
                x[:layers, p, :, s] = old[:layers, fp, :, fs]


SHAPES = [(8, 128), (4, 64), (1, 64), (32, 64), (2, 128), (5, 128)]


def _requests(seed, n, depth, most, pages_each=6):
    """(prefix, path, length, table) of n requests with rising paths, lengths from 0 to depth."""
    rng = np.random.default_rng(seed)
    pages = rng.permutation(n * pages_each)
    table = pages.reshape(n, pages_each).astype(np.int32)
    prefix = rng.integers(0, pages_each * 16 - most, size=n, endpoint=True).astype(np.int32)
    length = rng.integers(0, depth, size=n, endpoint=True).astype(np.int32)
    length[0], length[-1] = depth, 0 if n > 1 else depth
    path = np.full((n, depth), -7, dtype=np.int32)  # behind the path's end: never read
    for s in range(n):
        path[s, : length[s]] = np.sort(rng.permutation(most)[: length[s]])
    return prefix, path, length, table


def _pairs(prefix, path, length, table):
    at = lambda s, x: (table[s, x // 16], x % 16)  # noqa: E731
    return [(at(s, prefix[s] + i), at(s, prefix[s] + path[s, i])) for s in range(len(prefix)) for i in range(length[s])]


@pytest.mark.gpu
@pytest.mark.parametrize("n,depth,most", [(1, 1, 1), (1, 64, 64), (3, 5, 16), (17, 8, 64), (5, 33, 40), (200, 4, 9)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_keep_nodes(cuda_device, shape, fp8, n, depth, most):
    prefix, path, length, table = _requests(5, n, depth, most)
    p = Pools(6, 3, table.size, *shape, fp8, cuda_device)
    args = [i32(x, cuda_device) for x in (path, length, prefix, table)]
    pkv.keep_nodes(*args, *p.given("stacked"), workspace=p.ws)
    p.move(_pairs(prefix, path, length, table))
    p.same()
    assert p.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("how", ["list", "tuple", "one"])
def test_layers_may_be_given_in_any_form(cuda_device, how, fp8):
    prefix, path, length, table = _requests(7, 4, 6, 20)
    p = Pools(8, 70, table.size + 4, 2, 64, fp8, cuda_device)  # more layers than one launch takes
    some = 1 if how == "one" else None
    args = [i32(x, cuda_device) for x in (path, length, prefix, table)]
    pkv.keep_nodes(*args, *p.given(how))
    p.move(_pairs(prefix, path, length, table), some)
    src, dst = [3, -1, 0, 5], [table.size, 2, table.size + 3, -4]
    pkv.copy_pages(i32(src, cuda_device), i32(dst, cuda_device), *p.given(how), workspace=p.ws)
    p.move([((d, i), (s, i)) for s, d in zip(src, dst) if s >= 0 and d >= 0 for i in range(16)], some)
    p.same()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 7, 100])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("shape", SHAPES + [(65, 128)], ids=str)
def test_copy_pages(cuda_device, shape, fp8, n):
    order = np.random.default_rng(n).permutation(2 * n + 3)
    p = Pools(9, 2, len(order), *shape, fp8, cuda_device)
    src, dst = order[:n], order[n: 2 * n]
    src = np.where(np.arange(n) % 3 == 1, src[0], src)  # one page for several forks
    pkv.copy_pages(i32(src, cuda_device), i32(dst, cuda_device), *p.given("stacked"), workspace=p.ws)
    p.move([((d, i), (s, i)) for s, d in zip(src, dst) for i in range(16)])
    p.same()
    assert p.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_bad_entries_are_reported_and_skipped(cuda_device, fp8):
    prefix, path, length, table = _requests(10, 6, 6, 12)
    length[:] = 6
    path[:] = [0, 2, 3, 7, 9, 11]
    prefix[:] = 20
    path[1, 2] = 2       # does not rise: node 2 twice
    path[2, 0] = -1      # no node
    path[3, 5] = 1 << 20  # past the table
    table[4, 1] = table.size + 50  # positions 16 .. 31: a page outside the pool
    good = _pairs(prefix[:1], path[:1], length[:1], table[:1])
    at = lambda s, x: (table[s, x // 16], x % 16)  # noqa: E731
    for s, skip in ((1, {2}), (2, {0}), (3, {5}), (5, set())):
        good += [(at(s, prefix[s] + i), at(s, prefix[s] + path[s, i])) for i in range(6) if i not in skip]
    # request 4: prefix 20, nodes at 20 .. 31: all rows of the path lie in the bad page
    p = Pools(11, 2, table.size, 8, 128, fp8, cuda_device)
    pkv.keep_nodes(*[i32(x, cuda_device) for x in (path, length, prefix, table)], *p.given("stacked"), workspace=p.ws)
    p.move(good)
    p.same()
    with pytest.raises(pkv.PkvError):
        p.ws.check()
    # lengths past the path's room, negative ones, a negative prefix
    table[4, 1] = table[4, 2]
    path[:] = [0, 2, 3, 7, 9, 11]
    length[:] = [99, -1, 6, 6, 0, 0]
    prefix[3] = -5
    pkv.keep_nodes(*[i32(x, cuda_device) for x in (path, length, prefix, table)], *p.given("stacked"), workspace=p.ws)
    p.move(_pairs(prefix[[0, 2]], path[[0, 2]], np.array([6, 6]), table[[0, 2]]))
    p.same()
    assert p.ws.status() == pkv.ERR_CODES["PKV_ERR_OUT_OF_BOUNDS"]
    p.ws = pkv.Workspace(pkv.PKV_STATUS_BYTES, cuda_device)
    pkv.copy_pages(i32([0, table.size, 3], cuda_device), i32([1, 2, table.size + 7], cuda_device), *p.given("stacked"),
                   workspace=p.ws)
    p.move([((1, i), (0, i)) for i in range(16)])
    p.same()
    assert p.ws.status() == pkv.ERR_CODES["PKV_ERR_OUT_OF_BOUNDS"]


@pytest.mark.gpu
def test_nodes_that_stay_in_a_bad_page_are_reported(cuda_device):
    """A path that moves nothing, whose rows lie in a page outside the pool."""
    p = Pools(14, 1, 4, 8, 128, False, cuda_device)
    for table, status in (([[0, 4]], pkv.ERR_CODES["PKV_ERR_OUT_OF_BOUNDS"]), ([[0, 3]], 0)):
        p.ws = pkv.Workspace(pkv.PKV_STATUS_BYTES, cuda_device)
        pkv.keep_nodes(i32([[0, 1, 2]], cuda_device), i32([3], cuda_device), i32([16], cuda_device), i32(table, cuda_device),
                       *p.given("stacked"), workspace=p.ws)
        p.same()
        assert p.ws.status() == status


@pytest.mark.gpu
def test_binding_refuses_bad_tensors(cuda_device):
    prefix, path, length, table = _requests(12, 3, 4, 9)
    p = Pools(13, 2, table.size, 2, 64, True, cuda_device)
    k, v, sc = p.given("stacked")
    a = [i32(x, cuda_device) for x in (path, length, prefix, table)]
    half = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16, device=cuda_device)
    bad = [dict(kv_scales=None), dict(kv_scales=sc[:1]), dict(v_pages=v[:1]), dict(k_pages=k[:, :4]), dict(k_pages=[]),
           dict(k_pages=[k[0]], v_pages=[v[0], v[1]]), dict(k_pages=[k[0], k[1, :3].contiguous()]), dict(k_pages=k[0, 0]),
           dict(k_pages=half, v_pages=half), dict(k_pages=k.cpu()), dict(k_pages="pools"), dict(k_pages=[1, 2])]
    for kw in bad:
        pools = dict(k_pages=k, v_pages=v, kv_scales=sc)
        pools.update(kw)
        with pytest.raises((TypeError, ValueError, AttributeError)):
            pkv.keep_nodes(*a, **pools)
        with pytest.raises((TypeError, ValueError, AttributeError)):
            pkv.copy_pages(a[1], a[2], **pools)
    for i, x in ((0, path[:, :, None]), (0, path[:2]), (1, length[:2]), (2, prefix[:1]), (3, table[:1]), (3, table[0])):
        args = list(a)
        args[i] = i32(x, cuda_device)
        with pytest.raises(ValueError):
            pkv.keep_nodes(*args, k, v, sc)
    with pytest.raises(TypeError):
        pkv.keep_nodes(a[0].long(), *a[1:], k, v, sc)
    with pytest.raises(ValueError):
        pkv.copy_pages(a[1][:2], a[2], k, v, sc)
    with pytest.raises(ValueError):
        pkv.copy_pages(a[0], a[0], k, v, sc)
    with pytest.raises(pkv.PkvError) as e:
        pkv.keep_nodes(torch.zeros(3, 65, dtype=torch.int32, device=cuda_device), *a[1:], k, v, sc)
    assert e.value.code == pkv.ERR_CODES["PKV_ERR_UNSUPPORTED"]
    p.same()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_pools_past_four_gigabytes(cuda_device, fp8):
    """Pages and rows at both ends of pools whose byte offsets pass 32 bits."""
    ensure_built()
    pages = (5 << 30) // (16 * 128 * 8 * (1 if fp8 else 2))
    kind, raw = (torch.float8_e4m3fn, torch.uint8) if fp8 else (torch.bfloat16, torch.int16)
    k = torch.empty((pages, 8, 16, 128), dtype=kind, device=cuda_device)
    v = torch.empty_like(k)
    sc = torch.empty((pages, 8, 2, 16), dtype=torch.float8_e8m0fnu, device=cuda_device) if fp8 else None
    ends = [0, 1, 2, pages - 3, pages - 2, pages - 1]
    pools = [k, v] + ([sc] if fp8 else [])
    for i, pool in enumerate(pools):
        g = torch.Generator(device=cuda_device).manual_seed(i)
        pool.view(raw if i < 2 else torch.uint8)[ends] = torch.randint(0, 127, (6, *pool.shape[1:]), generator=g, device=cuda_device,
                                                                       dtype=raw if i < 2 else torch.uint8)
    read = lambda x: x.view(raw if x is not sc else torch.uint8)[ends].clone()  # noqa: E731
    old = [read(x) for x in pools]
    pkv.copy_pages(i32([0, pages - 1], cuda_device), i32([pages - 2, 1], cuda_device), k, v, sc)
    table = i32([[pages - 3, 2]], cuda_device)  # node 5 at position 17 (page 2, slot 1) to position 13
    pkv.keep_nodes(i32([[0, 5]], cuda_device), i32([2], cuda_device), i32([12], cuda_device), table, k, v, sc)
    torch.cuda.synchronize()
    for i, (x, o) in enumerate(zip(pools, old)):
        o[4], o[1] = o[0].clone(), o[5].clone()
        o = o if i < 2 else o.transpose(-1, -2)
        o[3][:, 13] = o[2][:, 1]
        assert torch.equal(read(x), o if i < 2 else o.transpose(-1, -2))
