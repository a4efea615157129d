"""One workspace shared by calls of different sizes: decode calls of any geometry, batch and merge, bf16 and 8-bit; prefill
and mixed-step calls of any number and length of chunks. Where a call's split scratch lies depends on its sizes, so nothing
that a call leaves uncleared may lie where another looks for zeros. Of decode only counted records stay behind; they have
every other 512 bytes of a workspace, behind the status header and the counters. Of prefill it is the records of cut query
tiles, right behind the status header."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gb300 as pkv
from gpu_util import DecodeOnDevice, ensure_built, i32
from paged_kv_decode_gb300 import workloads as W
from test_fp8_cache import GEOMS, Cache

pytestmark = pytest.mark.gpu


def _counted(ws):
    """Mask of the workspace's bytes that may hold counted records."""
    at = torch.arange(ws.nbytes, device=ws.tensor.device) - 512
    return (at >= 0) & (at // 512 % 2 == 0)


def _bf16(geom, lens, dev):
    g = W.Geometry(*GEOMS[geom])
    return DecodeOnDevice(W.decode_case(61, lens, geom=g, pending_append=False), 0, dev)


def _make(kind, geom, lens, dev, width=None):
    return _bf16(geom, lens, dev) if kind == "bf16" else Cache(61, GEOMS[geom], lens, dev, width=width)


def _bits(t):
    return t.clone().view(torch.int16)


BS16 = [3, 0, 2900, 700] * 4
CALLS = [("bf16", "64q8kv128", [9000], None), ("fp8", "64q8kv128", [9000], None),  # one request, counted
         ("bf16", "28q4kv128", [40000], None), ("fp8", "8q1kv64", [9001], 9000),  # counted in the wide shape
         ("bf16", "8q1kv64", [30000], None), ("fp8", "16q8kv64", [700], None),
         ("bf16", "16q8kv128", [40000], None), ("fp8", "16q8kv128", [40000], None),  # one request, polled
         ("bf16", "16q8kv128", BS16, None), ("fp8", "16q8kv128", BS16, None), ("fp8", "14q2kv64", [2000, 37, 9, 900], None),
         ("bf16", "16q8kv64", [900] * 100, None)]


@pytest.mark.parametrize("kind,geom,lens,width", CALLS)
def test_what_other_calls_left_does_not_matter(cuda_device, kind, geom, lens, width):
    """The counted records' bytes filled with the worst that they may hold, words that look like tagged ones: the same
    outputs twice, and all other bytes left zero."""
    c = _make(kind, geom, lens, cuda_device, width)
    want = _bits(c.step())
    counted = _counted(c.ws)
    assert torch.count_nonzero(c.ws.tensor[~counted]).item() == 0
    c.ws.tensor[counted] = 0xA5
    for _ in range(2):
        c.out.fill_(float("nan"))
        assert torch.equal(_bits(c.step()), want)
    assert torch.count_nonzero(c.ws.tensor[~counted]).item() == 0 and c.ws.status() == 0


def test_calls_of_different_sizes_alternate_on_one_workspace(cuda_device):
    """One-request steps of large groups between batches of small ones: the outputs of calls with a workspace each, bit
    for bit."""
    calls = [_make(*a[:3], cuda_device, a[3]) for a in CALLS if a[2] != [40000]]
    want = [_bits(c.step()) for c in calls]
    torch.cuda.synchronize()
    shared = pkv.Workspace(max(c.ws.nbytes for c in calls), cuda_device)
    for c in calls:
        c.ws = shared
    for i in np.random.default_rng(62).integers(0, len(calls), size=150):
        calls[i].out.fill_(float("nan"))
        assert torch.equal(_bits(calls[i].step()), want[i]), i
    assert torch.count_nonzero(shared.tensor[~_counted(shared)]).item() == 0 and shared.status() == 0


class _Prefill:
    """A prefill call, or (with decode requests) a mixed step."""

    def __init__(self, geom, prefix, qlens, dec, dev):
        ensure_built()
        g = W.Geometry(*GEOMS[geom])
        c = W.prefill_case(63, prefix, qlens, dec_seq_lens=dec or (), geom=g)
        self.geom, self.max_q, self.scale = g, int(c.q_lens.max()), g.scale
        kp, vp = c.k_pages[0].to(dev), c.v_pages[0].to(dev)
        pkv.append(c.k_new[0].to(dev), c.v_new[0].to(dev), i32(c.slot_mapping, dev), kp, vp)
        self.args = [c.q[0].to(dev), kp, vp, i32(c.block_table, dev), i32(c.prefix_lens, dev), i32(c.cu_q_lens, dev)]
        self.out = torch.full_like(self.args[0], float("nan"))
        self.dec = None
        if dec is None:
            nbytes = pkv.prefill_workspace_bytes(len(qlens), self.max_q, 1, g.n_q_heads, g.n_kv_heads, g.head_dim)
        else:
            pkv.append(c.dec_k_new[0].to(dev), c.dec_v_new[0].to(dev), i32(c.dec_slot_mapping, dev), kp, vp)
            self.dec = [c.dec_q[0].to(dev), i32(c.dec_block_table, dev), i32(c.dec_seq_lens, dev)]
            self.dout = torch.full_like(self.dec[0], float("nan"))
            nbytes = pkv.mixed_workspace_bytes(len(qlens), self.max_q, len(dec), c.dec_block_table.shape[1])
        self.ws = pkv.Workspace(nbytes, dev)

    def step(self):
        self.out.fill_(float("nan"))
        if self.dec is None:
            pkv.prefill_chunk_attn(*self.args, self.out, self.scale, self.max_q, self.ws)
            return _bits(self.out)
        self.dout.fill_(float("nan"))
        pkv.mixed_step_attn(*self.args, self.out, self.max_q, *self.dec, self.dout, self.scale, self.ws)
        return torch.cat([_bits(self.out), _bits(self.dout)])


PREFILLS = [("16q8kv128", [9000], [100], None), ("16q8kv128", [6000], [4096], None),
            ("16q8kv128", [0, 500, 3000, 40], [900, 300, 1500, 1], None), ("16q8kv64", [9000], [700], None),
            ("28q4kv128", [5000, 17], [1000, 3000], None), ("32q32kv64", [3000], [2048], None)]
MIXED = [("16q8kv128", [9000], [100], [5000, 30, 2000]), ("16q8kv128", [6000], [4096], [1500] * 15),
         ("16q8kv128", [0, 2000], [500, 900], [9000, 17000]), ("16q8kv128", [100], [1024], [300] * 60)]


def _prefill_records(ws):
    """Mask of the workspace's bytes that may hold records of cut query tiles: two of 67,584 bytes per SM."""
    at = torch.arange(ws.nbytes, device=ws.tensor.device) - pkv.PKV_STATUS_BYTES
    sms = torch.cuda.get_device_properties(ws.tensor.device).multi_processor_count
    return (at >= 0) & (at < 2 * sms * 67584)


@pytest.mark.parametrize("call", PREFILLS + MIXED, ids=str)
def test_prefill_clears_what_the_next_call_counts_in(cuda_device, call):
    c = _Prefill(*call, cuda_device)
    want = c.step()
    records = _prefill_records(c.ws)
    assert torch.isfinite(want.view(torch.bfloat16).float()).all()
    assert torch.count_nonzero(c.ws.tensor[~records]).item() == 0
    c.ws.tensor[records] = 0xA5
    for _ in range(2):
        assert torch.equal(c.step(), want)
    assert torch.count_nonzero(c.ws.tensor[~records]).item() == 0 and c.ws.status() == 0


@pytest.mark.parametrize("calls", [PREFILLS, MIXED], ids=["prefill", "mixed"])
def test_prefill_calls_of_different_sizes_alternate_on_one_workspace(cuda_device, calls):
    calls = [_Prefill(*c, cuda_device) for c in calls]
    want = [c.step() for c in calls]
    torch.cuda.synchronize()
    shared = pkv.Workspace(max(c.ws.nbytes for c in calls), cuda_device)
    for c in calls:
        c.ws = shared
    for i in np.random.default_rng(64).integers(0, len(calls), size=60):
        assert torch.equal(calls[i].step(), want[i]), i
    assert torch.count_nonzero(shared.tensor[~_prefill_records(shared)]).item() == 0 and shared.status() == 0
