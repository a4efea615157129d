"""The status word of the calls that use nothing else of a workspace is an int that kernels update by atomics: a workspace that
does not start on 4 bytes is refused on the host by each of them."""
import ctypes

import pytest

from paged_kv_decode_gb300 import _lib
from paged_kv_decode_gb300.build import build_library


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _lib.load()


def _calls(lib, p, ws):
    """Each call with good arguments (addresses that the host never reads, save the arrays of pools) and this workspace."""
    d = ctypes.byref(_lib.CacheDesc(num_q_heads=8, num_kv_heads=8, head_dim=128, page_size=16, num_pages=4))
    pools, n = (ctypes.c_void_p * 2)(p, p + 1024), 4096
    row = (p, 1024, p, 1024, p, 1024, p, p, 2, p, 8, p, p, 1e-6, p, p, p)
    return {
        "append": lambda: lib.pkv_append(p, p, p, 2, p, p, d, None, ws, n),
        "append_rope": lambda: lib.pkv_append_rope(*row, d, None, ws, n),
        "append_rope_fp8": lambda: lib.pkv_append_rope_fp8(*row, p, d, None, ws, n),
        "expand_fp8": lambda: lib.pkv_expand_fp8(p, p, p, p, p, 2, 4, p, p, p, 4, d, None, ws, n),
        "keep_nodes": lambda: lib.pkv_keep_nodes(p, p, p, p, 2, 4, 4, pools, pools, None, 2, d, None, ws, n),
        "copy_pages": lambda: lib.pkv_copy_pages(p, p, 2, pools, pools, None, 2, d, None, ws, n),
    }


@pytest.mark.parametrize("off", [1, 2, 3, 7])
@pytest.mark.parametrize("name", ["append", "append_rope", "append_rope_fp8", "expand_fp8", "keep_nodes", "copy_pages"])
def test_a_workspace_off_its_status_words_alignment_is_refused(lib, name, off):
    buf = ctypes.create_string_buffer(8192)
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    assert _calls(lib, p, p + off)[name]() == -8
