"""Append with the rotary embedding and per-head norm, into the bf16 pools and into the 8-bit cache, against float64
numpy written from the definition (tests/fp8_util.py).

Tolerances: a bf16 result is within half a bf16 step (2^-8 relative) of the value, an e4m3 one within half an e4m3 step
(2^-4 relative, or 2^-10 of the row's scale where e4m3 is subnormal), both plus fp32's error in y (fp32_noise)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_decode_gb300 as pkv
from fp8_util import (CODE_VALUES, EXP_MAX, EXP_MIN, cache_to, codes_of, dequantise, fp32_noise, quantise, random_cache,
                      rotate64)
from gpu_util import bits, ensure_built, i32
from paged_kv_decode_gb300 import _lib
from paged_kv_decode_gb300.build import build_library
from parity import bf16_to_f64

THETA = 1.0e6
SENTINEL = 0x4321  # bf16 bits of slots that no call may write


# ---------------------------------------------------------------------------------------------- CPU: refusals
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
    row = 8 * 128

    def call(desc=_desc(), n=2, q=p, qs=16 * 128, k=p, ks=row, v=p, vs=row, pos=p, slots=p, table=p, max_pos=8, qw=p,
             kw=p, eps=1e-6, qo=p, kp=p, vp=p, sc=p, ws=None, nb=0):
        f = lib.pkv_append_rope_fp8 if fp8 else lib.pkv_append_rope
        scales = (sc,) if fp8 else ()
        return f(q, qs, k, ks, v, vs, pos, slots, n, table, max_pos, qw, kw, eps, qo, kp, vp, *scales,
                 None if desc is None else ctypes.byref(desc), None, ws, nb)

    assert call(desc=None) == -1
    for bad in (_desc(head_dim=96), _desc(page_size=32), _desc(num_q_heads=36, num_kv_heads=4), _desc(num_q_heads=20)):
        assert call(desc=bad) == -3
    assert call(desc=_desc(num_pages=0)) == -2
    assert call(desc=_desc(num_pages=(1 << 27) + 1)) == -3  # slots past 32 bits
    assert call(n=-1) == -2
    assert call(n=1 << 26) == -2  # 2^26 tokens of 32 rows
    assert call(eps=-1.0) == -2 and call(eps=float("nan")) == -2
    assert call(max_pos=0) == -2
    assert call(ks=row - 8) == -2 and call(vs=row - 8) == -2 and call(qs=row) == -2
    assert call(ks=row + 4) == -8 and call(vs=row + 4) == -8 and call(qs=16 * 128 + 4) == -8
    for name in ("k", "v", "slots", "kp", "vp", "pos"):
        assert call(**{name: None}) == -1, name
    assert call(q=None) == -1 and call(qo=None) == -1  # they come together
    if fp8:
        assert call(sc=None) == -1 and call(sc=p + 8) == -8
    for name in ("q", "k", "v", "table", "qw", "kw", "qo", "kp", "vp"):
        assert call(**{name: p + 8}) == -8, name
    assert call(ws=p, nb=64) == -4
    assert call(n=0) == 0  # nothing to do, no device


# ---------------------------------------------------------------------------------------------- GPU
GEOMS = {"16q8kv128": (16, 8, 128), "28q4kv128": (28, 4, 128), "12q4kv128": (12, 4, 128), "32q32kv64": (32, 32, 64),
         "8q1kv64": (8, 1, 64), "14q2kv64": (14, 2, 64)}


class Step:
    """Seeded inputs of one append: fused q/k/v rows, distinct slots over a permuted pool, positions."""

    def __init__(self, seed, geom, n, dev, *, norm="both", rope=True, gap=0, skip=()):
        ensure_built()
        hq, hkv, d = geom
        self.geom, self.n, self.dev = geom, n, dev
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        width = (hq + 2 * hkv) * d + gap
        ch = torch.exp(0.5 * torch.randn(width, generator=gen))
        self.qkv = (torch.randn(n, width, generator=gen) * ch).to(torch.bfloat16).to(dev)
        self.q = self.qkv[:, : hq * d].view(n, hq, d)
        self.k = self.qkv[:, hq * d: (hq + hkv) * d].view(n, hkv, d)
        self.v = self.qkv[:, (hq + hkv) * d: (hq + 2 * hkv) * d].view(n, hkv, d)
        self.num_pages = max(2, (2 * n + 15) // 16)
        slots = rng.permutation(self.num_pages * 16)[:n].astype(np.int32)
        for t in skip:
            slots[t] = -1 - t
        self.slots_np = slots
        self.slots = i32(slots, dev)
        self.max_pos = 777
        self.pos_np = rng.integers(0, self.max_pos, size=n).astype(np.int32)
        self.pos_np[0] = self.max_pos - 1
        self.pos = i32(self.pos_np, dev)
        self.table = pkv.rope_cos_sin(THETA, self.max_pos, d, dev) if rope else None
        w = (1 + 0.2 * torch.randn(2, d, generator=gen)).to(torch.bfloat16).to(dev)
        self.qw = w[0].contiguous() if norm in ("both", "q") else None
        self.kw = w[1].contiguous() if norm in ("both", "k") else None
        self.q_out = torch.empty(n, hq, d, dtype=torch.bfloat16, device=dev)
        self.ws = pkv.Workspace(pkv.PKV_STATUS_BYTES, dev)

    def pools16(self):
        _, hkv, d = self.geom
        full = lambda: torch.full((self.num_pages, hkv, 16, d), SENTINEL, dtype=torch.int16, device=self.dev).view(  # noqa: E731
            torch.bfloat16)
        return full(), full()

    def pools8(self):
        _, hkv, d = self.geom
        full = lambda shape, b, t: torch.full(shape, b, dtype=torch.uint8, device=self.dev).view(t)  # noqa: E731
        shape = (self.num_pages, hkv, 16, d)
        return (full(shape, 0x55, torch.float8_e4m3fn), full(shape, 0x56, torch.float8_e4m3fn),
                full((self.num_pages, hkv, 2, 16), 0x33, torch.float8_e8m0fnu))

    def want(self, x, w):
        cs = None if self.table is None else bf16_to_f64(self.table)[self.pos_np]
        return rotate64(bf16_to_f64(x), None if w is None else bf16_to_f64(w), cs, 1e-6)

    def append(self, pools, **kw):
        args = dict(q=self.q, q_out=self.q_out, q_weight=self.qw, k_weight=self.kw)
        args.update(kw)
        f = pkv.append_rope_fp8 if len(pools) == 3 else pkv.append_rope
        f(self.k, self.v, self.pos, self.slots, self.table, *pools, self.ws, **args)
        torch.cuda.synchronize()

    def split(self, pool):
        """(rows written [tokens with a slot, hkv, ...], everything else) of a pool [P, hkv, 16, ...] as numpy."""
        flat = pool.swapaxes(1, 2).reshape(-1, pool.shape[1], *pool.shape[3:])
        keep = self.slots_np >= 0
        rest = np.ones(len(flat), dtype=bool)
        rest[self.slots_np[keep]] = False
        return flat[self.slots_np[keep]], flat[rest]


def _check_bf16(got, y, size, d, what):
    err, tol = np.abs(got - y), 2.0 ** -8 * np.abs(y) + fp32_noise(d, size) + 2.0 ** -134
    assert (err <= tol).all(), f"{what}: {err.max()} over by {(err - tol).max()}"


def _check_fp8(codes, scales, y, size, d, what):
    """Rows of codes / scale bytes stand for y: the scale is the row's, each value within half a step."""
    e = scales.astype(np.int64) - 127
    noise = fp32_noise(d, size)
    top, off = np.abs(y).max(axis=-1), noise.max(axis=-1)
    assert (top <= 448.0 * np.ldexp(1.0, e) + off).all(), what
    assert ((top + off > 224.0 * np.ldexp(1.0, e)) | (e == EXP_MIN)).all(), what
    err = np.abs(dequantise(codes, scales) - y)
    tol = np.maximum(2.0 ** -4 * np.abs(y), np.ldexp(2.0 ** -10, e)[..., None]) + noise
    assert (err <= tol * (1 + 2.0 ** -20)).all(), f"{what}: over by {(err - tol).max()}"


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["none", "both", "k"])
@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("geom", sorted(GEOMS))
def test_bf16_pools(cuda_device, geom, n, norm):
    g = GEOMS[geom]
    st = Step(7, g, n, cuda_device, norm=norm, gap=8 * (n % 2), skip=(1,) if n > 1 else ())
    pools = st.pools16()
    st.append(pools)
    assert st.ws.status() == 0
    _check_bf16(bf16_to_f64(st.q_out), *st.want(st.q, st.qw), g[2], "q")
    keep = st.slots_np >= 0
    rows, rest = st.split(pools[0].cpu().view(torch.int16).numpy())
    y, size = st.want(st.k, st.kw)
    _check_bf16(bf16_to_f64(torch.from_numpy(rows.copy()).view(torch.bfloat16)), y[keep], size[keep], g[2], "k")
    assert (rest == SENTINEL).all()
    rows, rest = st.split(pools[1].cpu().view(torch.int16).numpy())
    assert np.array_equal(rows.view(np.uint16), bits(st.v)[keep]) and (rest == SENTINEL).all()


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["none", "both"])
@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("geom", sorted(GEOMS))
def test_fp8_pools(cuda_device, geom, n, norm):
    g = GEOMS[geom]
    st = Step(8, g, n, cuda_device, norm=norm, gap=8 * (n % 2), skip=(1,) if n > 1 else ())
    kp, vp, sc = st.pools8()
    st.append((kp, vp, sc))
    assert st.ws.status() == 0
    _check_bf16(bf16_to_f64(st.q_out), *st.want(st.q, st.qw), g[2], "q")
    keep = st.slots_np >= 0
    scales = codes_of(sc)
    kr, krest = st.split(codes_of(kp))
    ks, ksrest = st.split(scales[:, :, 0, :, None])
    y, size = st.want(st.k, st.kw)
    _check_fp8(kr, ks[..., 0], y[keep], size[keep], g[2], "k")
    # value rows are quantised from their bf16 values alone: bit for bit
    vr, vrest = st.split(codes_of(vp))
    vs, vsrest = st.split(scales[:, :, 1, :, None])
    want, want_s = quantise(bf16_to_f64(st.v)[keep])
    assert np.array_equal(vr, want) and np.array_equal(vs[..., 0], want_s)
    assert (krest == 0x55).all() and (vrest == 0x56).all() and (ksrest == 0x33).all() and (vsrest == 0x33).all()


@pytest.mark.gpu
@pytest.mark.parametrize("geom", ["16q8kv128", "14q2kv64"])
def test_long_chunk(cuda_device, geom):
    """5000 tokens: the grid-stride loop's later rounds, and q_out in q's own place."""
    g = GEOMS[geom]
    st = Step(9, g, 5000, cuda_device)
    q = st.q.contiguous()
    y, size = st.want(q, st.qw)
    pools = st.pools16()
    st.append(pools, q=q, q_out=q)
    _check_bf16(bf16_to_f64(q), y, size, g[2], "q in place")
    rows, _ = st.split(pools[0].cpu().view(torch.int16).numpy())
    _check_bf16(bf16_to_f64(torch.from_numpy(rows.copy()).view(torch.bfloat16)), *st.want(st.k, st.kw), g[2], "k")
    pools8 = st.pools8()
    st.append(pools8)
    kr, _ = st.split(codes_of(pools8[0]))
    ks, _ = st.split(codes_of(pools8[2])[:, :, 0, :, None])
    _check_fp8(kr, ks[..., 0], *st.want(st.k, st.kw), g[2], "k")
    assert st.ws.status() == 0


@pytest.mark.gpu
def test_same_bits_as_the_fused_decode_call_and_the_plain_append(cuda_device):
    """Without norms the key rows are decode_append_rope_attn's bits; without table too, append's."""
    geom = GEOMS["16q8kv128"]
    st = Step(10, geom, 9, cuda_device, norm="none")
    lens = np.minimum(st.pos_np, 200).astype(np.int32) + 1
    width = 13
    bt = np.random.default_rng(1).permutation(9 * width).reshape(9, width).astype(np.int32)
    shape = (9 * width, 8, 16, 128)
    zero = lambda: torch.zeros(shape, dtype=torch.bfloat16, device=cuda_device)  # noqa: E731
    kp, vp, kp2, vp2 = zero(), zero(), zero(), zero()
    ws = pkv.Workspace(pkv.decode_workspace_bytes(9, width), cuda_device)
    out = torch.empty_like(st.q_out)
    pkv.decode_append_rope_attn(st.q.contiguous(), st.k.contiguous(), st.v.contiguous(), kp, vp, i32(bt, cuda_device),
                                i32(lens, cuda_device), st.table, out, 128 ** -0.5, ws)
    slots = bt[np.arange(9), (lens - 1) // 16] * 16 + (lens - 1) % 16
    pkv.append_rope(st.k, st.v, i32(lens - 1, cuda_device), i32(slots, cuda_device), st.table, kp2, vp2)
    assert np.array_equal(bits(kp), bits(kp2)) and np.array_equal(bits(vp), bits(vp2))
    # and the attention over them with the rotated queries is the fused call's, which rotates its own
    pkv.append_rope(st.k, st.v, i32(lens - 1, cuda_device), i32(slots, cuda_device), st.table, kp2, vp2, q=st.q,
                    q_out=st.q_out)
    out2 = torch.empty_like(out)
    pkv.decode_attn(st.q_out, kp2, vp2, i32(bt, cuda_device), i32(lens, cuda_device), out2, 128 ** -0.5, ws)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    kp3, vp3 = zero(), zero()
    nan_k, nan_v = st.k.contiguous(), st.v.contiguous()
    nan_k.view(torch.int16)[2, 3, 5] = 0x7F81  # a NaN payload survives the plain copy
    pkv.append(nan_k, nan_v, i32(slots, cuda_device), kp3, vp3)
    kp4, vp4 = zero(), zero()
    pkv.append_rope(nan_k, nan_v, None, i32(slots, cuda_device), None, kp4, vp4)
    assert np.array_equal(bits(kp3), bits(kp4)) and np.array_equal(bits(vp3), bits(vp4))


@pytest.mark.gpu
def test_fp8_rows_of_every_size(cuda_device):
    """Zero rows, rows on the border between two scales, subnormal, huge and non-finite values: bit for bit."""
    d, hkv = 128, 8
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, hkv, d))
    x[0] = 0.0
    x[1, :, 0] = 448.0 * np.ldexp(1.0, np.arange(hkv) - 4)  # the largest value on the border: the lower scale
    x[2, :, 0] = 450.0  # one bf16 step above it: the next scale
    x[3] *= 1e-30
    x[4] *= np.ldexp(1.0, -130)
    x[5] *= 1e30
    x[6, :, 7] = 3.3e38
    x[7] = np.ldexp(1.0, rng.integers(-40, 20, size=(hkv, d)))  # a wide row: e4m3's subnormals and zeros
    x[8, :, 3] = np.inf
    x[9, :, 4] = -np.inf
    x[10, :, 5] = np.nan
    x[11] = np.inf
    x[12, :, ::2] = -0.0
    x[13] = (rng.integers(16, 32, size=(hkv, d)) + 0.5) / 16  # ties between two e4m3 values
    v = torch.from_numpy(x).to(torch.bfloat16)
    ensure_built()
    n, pages = 64, 8
    kp, vp, sc = cache_to(*random_cache(1, pages, hkv, d), cuda_device)
    slots = np.random.default_rng(4).permutation(pages * 16)[:n].astype(np.int32)
    vd = v.to(cuda_device)
    pkv.append_rope_fp8(vd, vd, None, i32(slots, cuda_device), None, kp, vp, sc)
    torch.cuda.synchronize()
    want, want_s = quantise(bf16_to_f64(v))
    for pool, which in ((kp, 0), (vp, 1)):
        got = codes_of(pool)[slots // 16, :, slots % 16]
        got_s = codes_of(sc)[slots // 16, :, which, slots % 16]
        assert np.array_equal(got_s, want_s)
        same = (got == want) | (np.isnan(CODE_VALUES[got]) & np.isnan(CODE_VALUES[want]))
        assert same.all()
    assert want_s.min() == EXP_MIN + 127 and want_s.max() == EXP_MAX + 127


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_bad_slots_and_positions_are_reported_and_skipped(cuda_device, fp8):
    st = Step(11, GEOMS["12q4kv128"], 20, cuda_device, norm="none")
    good = (st.pools8 if fp8 else st.pools16)()
    st.append(good)
    assert st.ws.status() == 0
    # a slot past the pool: that token's rows are not written, the others are
    slots, pos = st.slots_np.copy(), st.pos_np.copy()
    st.slots_np = slots.copy()
    st.slots_np[4] = -1
    bad = slots.copy()
    bad[4] = st.num_pages * 16
    st.slots = i32(bad, cuda_device)
    pools = (st.pools8 if fp8 else st.pools16)()
    st.append(pools)
    assert st.ws.status() == -7
    view = lambda p: p.cpu().view(torch.uint8 if fp8 else torch.int16).numpy()  # noqa: E731
    canary = {0: 0x55, 1: 0x56} if fp8 else {0: SENTINEL, 1: SENTINEL}
    for i in (0, 1):
        rows, rest = st.split(view(pools[i]))
        assert np.array_equal(rows, np.delete(view(good[i]).swapaxes(1, 2).reshape(-1, *rows.shape[1:])[slots], 4, 0))
        assert (rest == canary[i]).all()
    # positions outside the table are clamped and reported
    pkv.workspace_init(st.ws.tensor)
    st.slots_np, st.slots = slots, i32(slots, cuda_device)
    far = pos.copy()
    far[2], far[3] = st.max_pos + 5, -1
    st.pos = i32(far, cuda_device)
    q_far = st.q_out
    pools = (st.pools8 if fp8 else st.pools16)()
    st.append(pools)
    assert st.ws.status() == -7
    got, q_got = [view(p) for p in pools[:2]], bits(q_far)
    pkv.workspace_init(st.ws.tensor)
    st.pos = i32(np.clip(far, 0, st.max_pos - 1), cuda_device)
    pools = (st.pools8 if fp8 else st.pools16)()
    st.append(pools)
    assert st.ws.status() == 0
    assert all(np.array_equal(a, view(p)) for a, p in zip(got, pools)) and np.array_equal(q_got, bits(st.q_out))
    # a padding token (no slot) of a call without query rows may have any position
    st.slots = i32(np.where(np.arange(20) == 2, -1, slots), cuda_device)
    far[3] = 0
    st.pos = i32(far, cuda_device)
    st.append(pools, q=None, q_out=None, q_weight=None)
    assert st.ws.status() == 0


@pytest.mark.gpu
def test_binding_refuses_bad_tensors(cuda_device):
    st = Step(12, GEOMS["16q8kv128"], 4, cuda_device)
    p16, p8 = st.pools16(), st.pools8()
    ok = dict(q=st.q, q_out=st.q_out)
    with pytest.raises(TypeError):
        pkv.append_rope(st.k.float(), st.v, st.pos, st.slots, st.table, *p16, **ok)
    with pytest.raises(TypeError):
        pkv.append_rope(st.k, st.v, st.pos.long(), st.slots, st.table, *p16, **ok)
    with pytest.raises(TypeError):
        pkv.append_rope(st.k, st.v, st.pos, st.slots, st.table, *p8[:2], **ok)
    with pytest.raises(TypeError):
        pkv.append_rope_fp8(st.k, st.v, st.pos, st.slots, st.table, *p8[:2], p8[2].view(torch.uint8), **ok)
    with pytest.raises(ValueError):  # scales of another shape
        pkv.append_rope_fp8(st.k, st.v, st.pos, st.slots, st.table, *p8[:2], p8[2][:, :, :, :8].contiguous(), **ok)
    with pytest.raises(ValueError):  # a strided head
        pkv.append_rope(st.k.transpose(1, 2).contiguous().transpose(1, 2), st.v, st.pos, st.slots, st.table, *p16, **ok)
    with pytest.raises(ValueError):
        pkv.append_rope(st.k[:3], st.v, st.pos, st.slots, st.table, *p16, **ok)
    with pytest.raises(ValueError):
        pkv.append_rope(st.k, st.v, st.pos, st.slots, st.table, *p16, q=st.q)
    with pytest.raises(ValueError):
        pkv.append_rope(st.k, st.v, st.pos[:3], st.slots, st.table, *p16, **ok)
    with pytest.raises(ValueError):
        pkv.append_rope(st.k, st.v, st.pos, st.slots, st.table[:, :64].contiguous(), *p16, **ok)
    with pytest.raises(ValueError):
        pkv.append_rope(st.k, st.v, st.pos, st.slots, st.table, *p16, k_weight=st.kw[:64].contiguous(), **ok)
    with pytest.raises(ValueError):  # no CPU path
        pkv.append_rope(st.k.cpu(), st.v, st.pos, st.slots, st.table, *p16, **ok)
    with pytest.raises(pkv.PkvError):  # tokens 4 elements off a 16-byte boundary
        odd = torch.zeros(4, 8 * 128 + 4, dtype=torch.bfloat16, device=cuda_device)[:, : 8 * 128].view(4, 8, 128)
        pkv.append_rope(odd, st.v, st.pos, st.slots, st.table, *p16, **ok)
    assert all((p.view(torch.int16) == SENTINEL).all() for p in p16)
    # no tokens: nothing happens
    none = st.slots[:0]
    pkv.append_rope(st.k[:0], st.v[:0], none, none, st.table, *p16)
    assert all((p.view(torch.int16) == SENTINEL).all() for p in p16)
