"""Tree attention where values or scores leave the ordinary range: value rows that are no numbers because of their scale byte,
and scales of zero and next to it with scores of any size."""
import numpy as np
import pytest
import torch

import paged_kv_decode_gb300 as pkv
from gpu_util import i32
from parity import bf16_to_f64
from test_tree_attn import GEOMS, Tree


def _bits(t):
    return t.clone().view(torch.int16)


def _expanded(c):
    """The tree's call over bf16 pages that expand_fp8 makes of its 8-bit ones, and the value pages."""
    k, v = (torch.zeros(c.pools[0].shape, dtype=torch.bfloat16, device=c.dev) for _ in range(2))
    pkv.expand_fp8(*c.pools, c.bt, i32([p + t for p, t in c.reqs], c.dev), k, v, c.bt)
    out = torch.empty_like(c.out)
    pkv.tree_attn(c.q, k, v, c.bt, c.prefix, c.cu, c.mask, out, c.scale, c.most, c.ws)
    return out, v


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [255, 254, 250], ids=str)
@pytest.mark.parametrize("geom,reqs", [("16q8kv128", [(300, 24), (120, 40), (0, 64)]), ("14q2kv64", [(9000, 33), (125, 7)])],
                         ids=str)
def test_scale_bytes_that_make_no_numbers_of_a_value_row(cuda_device, geom, reqs, byte):
    """A node's value row whose scale byte is the NaN of e8m0 (255: every product is infinite or NaN) or so large that 2^e v
    overflows: what expand_fp8 and tree_attn give, bit for bit, no number in those columns where a node sees the row, and the
    old bits where it does not."""
    c = Tree(41, GEOMS[geom], reqs, cuda_device, fp8=True)
    clean = _bits(c.step())
    sick = [(b, t // 3) for b, (_, t) in enumerate(reqs)]
    scales = c.pools[2].view(torch.uint8)
    for b, j in sick:
        at = reqs[b][0] + j
        scales[int(c.table[b, at // 16]), :, 1, at % 16] = byte
    got = c.step().clone()
    want, v = _expanded(c)
    assert torch.equal(_bits(got), _bits(want))
    got64 = bf16_to_f64(got)
    for b, j in sick:
        at = reqs[b][0] + j
        row = bf16_to_f64(v[int(c.table[b, at // 16]), :, at % 16])  # [hkv, d]
        none = np.repeat(~np.isfinite(row), c.hq // c.hkv, axis=0)
        assert none.any()
        for i in range(reqs[b][1]):
            n = int(c.cu_np[b]) + i
            if c.mask_np[n] >> j & 1:
                assert not np.isfinite(got64[n][none]).any()
            else:
                assert torch.equal(_bits(got)[n], clean[n])
    assert c.ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-42, 1e-45])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_scales_of_nothing_with_large_scores(cuda_device, scale, fp8):
    """Scores up to 2^126 and a scale that takes them to zero: every visible key has the same weight (the bound of the scores'
    own rounding, in proportion to the scale, is below 2^-30 here)."""
    c = Tree(42, GEOMS["12q4kv128"], [(130, 20), (0, 3), (700, 9)], cuda_device, fp8=fp8, q_size=2.0 ** 120)
    assert 2.0 ** 122 < float(c.q.abs().max()) < 2.0 ** 123.5
    c.scale = scale
    c.step()
    c.check()
