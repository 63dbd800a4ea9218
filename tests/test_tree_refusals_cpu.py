"""Arguments of the drafted-token and cache-budget calls that the library and its binding
refuse before any launch."""
import ctypes

import pytest

import sparse_kv_b200 as skv
from test_tree_abi_cpu import FAKE, tree_args


@pytest.mark.parametrize("kw", [dict(scale=3e38), dict(scale=-2.5e38), dict(softcap=2.5e38), dict(softcap=3e38, scale=1e30)])
def test_factors_past_fp32_in_base_2(kw):
    # scores are taken in base 2: a factor that is finite only before it is multiplied by log2 e
    a = tree_args(**kw)
    L = skv.lib()
    assert L.attn_tree_decode(ctypes.byref(a), None) == skv.SKV_EINVAL
    assert L.skv_tree_workspace_size(ctypes.byref(a)) == 0
    assert L.attn_key_mass(ctypes.byref(a), None, None, 1.0, 1 << 21, FAKE, None) == skv.SKV_EINVAL
    for ok in (dict(scale=2.3e38), dict(softcap=2.3e38)):
        assert L.skv_tree_workspace_size(ctypes.byref(tree_args(**ok))) > 0
