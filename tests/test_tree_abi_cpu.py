"""The draft-tree, key-mass and eviction entry points without a GPU: struct layouts
and the refusal of bad arguments on the host, before any launch."""
import ctypes
import os
import shutil
import subprocess

import pytest

import sparse_kv_b200 as skv
from sparse_kv_b200 import CompactArgs, TreeArgs, _Window

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000001000  # aligned, never dereferenced: every case fails validation first


@pytest.mark.parametrize("struct,name", [(TreeArgs, "skv_tree_args"), (CompactArgs, "skv_compact_args")])
def test_binding_struct_matches_the_header(struct, name, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    fields = [f[0] for f in struct._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sparsekv.h"\nint main(void) {\n'
                   f'  printf("size %zu\\n", sizeof({name}));\n' +
                   "".join(f'  printf("{n} %zu\\n", offsetof({name}, {n}));\n' for n in fields) + "  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(struct)
    for n in fields:
        assert int(got[n]) == getattr(struct, n).offset, n


def test_packed_arguments_match_the_structs():
    # the binding fills the structs from packed bytes: same size, and the fields land in place
    assert skv._TREE.size == ctypes.sizeof(TreeArgs) and skv._COMPACT.size == ctypes.sizeof(CompactArgs)
    for struct, packer in ((TreeArgs, skv._TREE), (CompactArgs, skv._COMPACT)):
        n = len(packer.unpack(bytes(packer.size)))
        a = struct.from_buffer_copy(packer.pack(*range(1, n + 1)))
        got = []
        for f, t in struct._fields_:
            v = getattr(a, f)
            got += [v.sink_tokens, v.recent_tokens] if f == "window" else [v]
        assert [int(x) for x in got] == list(range(1, n + 1))


def tree_args(**kw):
    a = TreeArgs()
    a.q = a.k_pool = a.v_pool = a.block_table = a.seq_lens = a.out = a.lse = FAKE
    a.batch, a.q_tokens, a.q_heads, a.kv_heads, a.head_dim, a.block_size = 16, 16, 32, 8, 128, 64
    a.max_blocks, a.num_pages, a.max_seq_len, a.scale = 512, 8192, 32768, 0.088
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_TREE = [
    (dict(q=None), skv.SKV_EINVAL), (dict(k_pool=None), skv.SKV_EINVAL), (dict(lse=None), skv.SKV_EINVAL),
    (dict(seq_lens=None), skv.SKV_EINVAL), (dict(block_table=None), skv.SKV_EINVAL),
    (dict(batch=0), skv.SKV_EINVAL), (dict(q_tokens=0), skv.SKV_EINVAL), (dict(q_heads=30), skv.SKV_EINVAL),
    (dict(q_heads=24), skv.SKV_EUNSUPPORTED), (dict(q_tokens=65), skv.SKV_EUNSUPPORTED),
    (dict(head_dim=64), skv.SKV_EUNSUPPORTED), (dict(block_size=32), skv.SKV_EUNSUPPORTED),
    (dict(q=FAKE + 8), skv.SKV_EINVAL), (dict(k_pool=FAKE + 4), skv.SKV_EINVAL),
    (dict(max_blocks=100), skv.SKV_EINVAL), (dict(num_pages=0), skv.SKV_EINVAL), (dict(max_seq_len=-1), skv.SKV_EINVAL),
    (dict(scale=float("nan")), skv.SKV_EINVAL), (dict(softcap=-1.0), skv.SKV_EINVAL),
    (dict(softcap=float("inf")), skv.SKV_EINVAL), (dict(window=_Window(-1, 4)), skv.SKV_EINVAL),
    (dict(window=_Window(4, -1)), skv.SKV_EINVAL),
    (dict(softcap=1e-38, scale=1e3), skv.SKV_EINVAL),
    (dict(batch=1, kv_heads=1, q_heads=1, max_seq_len=(1 << 30) + 1, max_blocks=(1 << 24) + 1), skv.SKV_EUNSUPPORTED),
    (dict(batch=1 << 20, max_seq_len=1 << 21, max_blocks=1 << 15), skv.SKV_EUNSUPPORTED),  # tiles past 32 bits
]


@pytest.mark.parametrize("kw,want", BAD_TREE)
def test_tree_and_mass_reject_on_host(kw, want):
    L = skv.lib()
    a = tree_args(**kw)
    assert L.attn_tree_decode(ctypes.byref(a), None) == want
    assert L.skv_tree_workspace_size(ctypes.byref(a)) == 0
    assert L.attn_key_mass(ctypes.byref(a), None, None, 1.0, 1 << 21, FAKE, None) == want


def test_tree_only_and_mass_only_fields():
    L = skv.lib()
    for kw in (dict(v_pool=None), dict(out=None), dict(v_pool=FAKE + 2), dict(out=FAKE + 4)):
        assert L.attn_tree_decode(ctypes.byref(tree_args(**kw)), None) == skv.SKV_EINVAL
    a = tree_args()
    assert L.attn_key_mass(ctypes.byref(a), None, None, 1.0, 32768, None, None) == skv.SKV_EINVAL
    assert L.attn_key_mass(ctypes.byref(a), None, None, 1.0, 32767, FAKE, None) == skv.SKV_EINVAL
    assert L.attn_key_mass(ctypes.byref(a), None, None, float("nan"), 32768, FAKE, None) == skv.SKV_EINVAL
    assert L.attn_tree_decode(None, None) == skv.SKV_EINVAL


@pytest.mark.parametrize("kw,want", [
    (dict(mass=None), skv.SKV_EINVAL), (dict(ids=None), skv.SKV_EINVAL), (dict(lens=None), skv.SKV_EINVAL),
    (dict(out_lens=None), skv.SKV_EINVAL), (dict(B=0), skv.SKV_EINVAL), (dict(keep=0), skv.SKV_EINVAL),
    (dict(sink=-1), skv.SKV_EINVAL), (dict(sink=900, recent=200), skv.SKV_EINVAL),
    (dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1), skv.SKV_EINVAL), (dict(stride=4095), skv.SKV_EINVAL),
    (dict(B=1 << 23), skv.SKV_EUNSUPPORTED), (dict(maxlen=(1 << 22) + 1, stride=1 << 23), skv.SKV_EUNSUPPORTED),
    (dict(keep=(1 << 30) + 1), skv.SKV_EUNSUPPORTED),
])
def test_evict_select_rejects_on_host(kw, want):
    names = ["mass", "lens", "B", "H", "maxlen", "stride", "keep", "sink", "recent", "ids", "out_lens", "status", "s"]
    a = dict(zip(names, [FAKE, FAKE, 4, 8, 4096, 4096, 1024, 64, 256, FAKE, FAKE, None, None]), **kw)
    assert skv.lib().attn_evict_select(*[a[n] for n in names]) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k_pool=None), skv.SKV_EINVAL), (dict(keep_ids=None), skv.SKV_EINVAL), (dict(new_lens=None), skv.SKV_EINVAL),
    (dict(new_lens=FAKE + 64), skv.SKV_EINVAL), (dict(batch=0), skv.SKV_EINVAL), (dict(max_keep=0), skv.SKV_EINVAL),
    (dict(ids_heads=3), skv.SKV_EINVAL), (dict(head_dim=64), skv.SKV_EUNSUPPORTED),
    (dict(block_size=16), skv.SKV_EUNSUPPORTED), (dict(v_pool=FAKE + 8), skv.SKV_EINVAL),
    (dict(dst_k_pool=FAKE, dst_v_pool=FAKE), skv.SKV_EINVAL),                     # pools without a table
    (dict(dst_block_table=FAKE, dst_k_pool=FAKE, dst_num_pages=9), skv.SKV_EINVAL),  # one pool of two
    (dict(dst_block_table=FAKE, dst_num_pages=0), skv.SKV_EINVAL),
    (dict(mass=FAKE, mass_stride=100), skv.SKV_EINVAL), (dict(max_blocks=10), skv.SKV_EINVAL),
])
def test_compact_rejects_on_host(kw, want):
    a = CompactArgs()
    a.k_pool = a.v_pool = a.block_table = a.keep_ids = a.keep_lens = a.new_lens = FAKE
    a.seq_lens = FAKE + 64
    a.batch, a.kv_heads, a.head_dim, a.block_size = 4, 8, 128, 64
    a.max_blocks, a.num_pages, a.max_seq_len, a.ids_heads, a.max_keep = 64, 256, 4096, 8, 100
    a.keep_lens = FAKE + 128
    for k, v in kw.items():
        setattr(a, k, v)
    assert skv.lib().attn_compact_cache(ctypes.byref(a), None) == want
    assert skv.lib().attn_compact_cache(None, None) == skv.SKV_EINVAL


def test_cpu_tensors_are_refused():
    import torch
    ids = torch.zeros(1, 1, 2, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    pool = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16)
    table = torch.zeros(1, 1, dtype=torch.int32)
    calls = [
        lambda: skv.attn_evict_select(torch.zeros(1, 1, 4), one, 2, ids, one.clone(), max_seq_len=4),
        lambda: skv.attn_compact_cache(pool, pool.clone(), table, one, ids, one.clone(), one.clone(), max_seq_len=4),
        lambda: skv.attn_tree_decode(torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16), pool, pool, table, one,
                                     torch.zeros(1, 1, 1, 128), torch.zeros(1, 1, 1), max_seq_len=4),
    ]
    for call in calls:
        with pytest.raises(skv.SkvError) as e:
            call()
        assert e.value.status == skv.SKV_EINVAL
