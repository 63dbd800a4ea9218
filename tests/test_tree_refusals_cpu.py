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


def tree_tensors():
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    return dict(q=torch.zeros(2, 3, 8, 128, dtype=bf16), k_pool=torch.zeros(5, 2, 64, 128, dtype=bf16),
                v_pool=torch.zeros(5, 2, 64, 128, dtype=bf16), block_table=torch.zeros(2, 4, dtype=i32),
                seq_lens=torch.zeros(2, dtype=i32), out=torch.zeros(2, 3, 8, 128), lse=torch.zeros(2, 3, 8),
                tree_mask=torch.zeros(2, 3, dtype=torch.int64), tree_lens=torch.zeros(2, dtype=i32),
                slopes=torch.zeros(8))


def sized(**kw):
    t = dict(tree_tensors(), **kw)
    pos = [t.pop(n) for n in ("q", "k_pool", "v_pool", "block_table", "seq_lens", "out", "lse")]
    return skv.tree_workspace_size(*pos, max_seq_len=256, **t)


@pytest.mark.parametrize("name,order", [("v_pool", (1, 0, 2, 3)), ("v_pool", (0, 1, 3, 2)), ("block_table", (1, 0)),
                                        ("out", (0, 2, 1, 3)), ("lse", (0, 2, 1)), ("tree_mask", (1, 0))])
def test_dimensions_in_another_order_are_refused(name, order):
    """As many elements, but not the tensor that the call reads."""
    assert sized() > 0
    with pytest.raises(skv.SkvError) as e:
        sized(**{name: tree_tensors()[name].permute(order).contiguous()})
    assert e.value.status == skv.SKV_EINVAL and name in str(e.value)


def test_one_word_of_status_may_have_any_shape():
    import torch
    for shape in ((), (1,), (1, 1)):
        assert sized(status=torch.zeros(shape, dtype=torch.int32)) > 0
    with pytest.raises(skv.SkvError):
        sized(status=torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("kw", [dict(max_seq_len=1 << 32), dict(max_seq_len=-(1 << 31) - 1), dict(window=(1 << 32, 0)),
                                dict(window=(0, (1 << 40) + 5))])
def test_numbers_past_32_bits(kw):
    t = tree_tensors()
    pos = [t.pop(n) for n in ("q", "k_pool", "v_pool", "block_table", "seq_lens", "out", "lse")]
    with pytest.raises(skv.SkvError) as e:
        skv.tree_workspace_size(*pos, **dict(dict(max_seq_len=256), **kw))
    assert e.value.status == skv.SKV_EINVAL


@pytest.mark.parametrize("kw", [dict(max_seq_len=(1 << 32) + 4), dict(sink=1 << 32), dict(recent=-(1 << 32)),
                                dict(sink=1 << 33, recent=1)])
def test_eviction_numbers_past_32_bits(kw, monkeypatch):
    """A C int would keep their low 32 bits: a sink of 2^32 would be none."""
    import torch
    launched = []
    monkeypatch.setattr(skv, "_launch", lambda *a: launched.append(a))
    call = [torch.zeros(1, 1, 4), torch.zeros(1, dtype=torch.int32), 2, torch.zeros(1, 1, 2, dtype=torch.int32),
            torch.zeros(1, dtype=torch.int32)]
    skv.attn_evict_select(*call, max_seq_len=4)
    assert len(launched) == 1
    with pytest.raises(skv.SkvError) as e:
        skv.attn_evict_select(*call, **dict(dict(max_seq_len=4), **kw))
    assert e.value.status == skv.SKV_EINVAL and len(launched) == 1


def test_compaction_numbers_past_32_bits(monkeypatch):
    import torch
    monkeypatch.setattr(skv, "_launch", lambda *a: None)
    pool, one = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    ids, table = torch.zeros(1, 1, 2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(skv.SkvError) as e:
        skv.attn_compact_cache(pool, pool, table, one, ids, one, one, max_seq_len=1 << 32)
    assert e.value.status == skv.SKV_EINVAL


@pytest.mark.parametrize("off", [0, 1, -3])
def test_lengths_written_over_lengths_that_are_read(off):
    """Every CTA of a sequence reads its lengths, one writes the new one: the arrays may not
    share a word."""
    L = skv.lib()
    assert L.attn_evict_select(FAKE, FAKE + 256, 4, 8, 4096, 4096, 1024, 64, 256, FAKE, FAKE + 256 + 4 * off, None,
                               None) == skv.SKV_EINVAL
    for name in ("seq_lens", "keep_lens", "first"):
        a = skv.CompactArgs()
        a.k_pool = a.v_pool = a.block_table = a.keep_ids = FAKE
        a.seq_lens, a.keep_lens, a.first = FAKE + 256, FAKE + 512, FAKE + 768
        a.batch, a.kv_heads, a.head_dim, a.block_size = 4, 8, 128, 64
        a.max_blocks, a.num_pages, a.max_seq_len, a.ids_heads, a.max_keep = 64, 256, 4096, 8, 100
        a.new_lens = getattr(a, name) + 4 * off
        assert L.attn_compact_cache(ctypes.byref(a), None) == skv.SKV_EINVAL, name
