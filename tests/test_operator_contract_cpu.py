"""What the serving operators accept and refuse before anything is enqueued, through the C ABI (no GPU is needed)."""
import ctypes as C

import pytest

from dynamic_depth_b200 import _lib

A = 0x100000  # an aligned address that nothing reads


def pool(**kw):
    f = dict(dev_pool=A, n_pages=4, dtype=_lib.TL_F16, n_kv_heads=2, head_dim=64, page_tokens=16)
    f.update(kw)
    return C.byref(_lib.TlKvPool(**f))


@pytest.mark.parametrize("R,rows", [(2, 0), (0, 0)])
def test_tree_attention_of_no_rows_needs_no_masks(R, rows):
    """The masks of an empty batch are an empty tensor, which has no address."""
    st = _lib.lib().tl_tree_attention(None, 128, pool(), A, 4, A, A, R, rows, 2, 8, None, 1, 0.0, None, _lib.TL_F16, 128,
                                      None, A, 1 << 30, None, None)
    assert st == _lib.TL_OK


def test_masks_are_still_wanted_where_there_are_rows():
    assert _lib.lib().tl_tree_attention(A, 128, pool(), A, 4, A, A, 2, 3, 2, 8, None, 1, 0.0, A, _lib.TL_F16, 128, None,
                                        A, 1 << 30, None, None) == _lib.TL_EINVAL
