"""One decode workspace shared by calls of different geometries, batches and merges, bf16 and 8-bit. Where a call's split
records lie depends on its sizes, so nothing that a call leaves uncleared may lie where another looks for zeros. Only
counted records stay behind; they have every other 512 bytes of a workspace, behind the status header and the counters."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gb300 as pkv
from gpu_util import DecodeOnDevice
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
