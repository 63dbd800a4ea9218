"""Tensors of the cache-budget calls whose elements are as many as wanted, in another shape:
refused before any launch."""
import pytest
import torch

import sparse_kv_b200 as skv

pytestmark = pytest.mark.gpu

B, H, S, N, P = 2, 3, 6, 4, 5
BF16, I32 = torch.bfloat16, torch.int32


def zeros(*shape, dtype=I32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def evict(**kw):
    a = dict(mass=zeros(B, H, S, dtype=torch.float32), seq_lens=zeros(B), keep=N, keep_ids=zeros(B, H, N), keep_lens=zeros(B))
    a.update(kw)
    skv.attn_evict_select(*a.values(), max_seq_len=S)


def compact(**kw):
    a = dict(k_pool=zeros(P, H, 64, 128, dtype=BF16), v_pool=zeros(P, H, 64, 128, dtype=BF16), block_table=zeros(B, 1),
             seq_lens=zeros(B), keep_ids=zeros(B, H, N), keep_lens=zeros(B), new_lens=zeros(B))
    opts = dict(first=zeros(B), mass=zeros(B, H, S, dtype=torch.float32),
                dst=(zeros(P, H, 64, 128, dtype=BF16), zeros(P, H, 64, 128, dtype=BF16), zeros(B, 2)))
    for k, v in kw.items():
        (a if k in a else opts)[k] = v
    skv.attn_compact_cache(*a.values(), max_seq_len=S, **opts)


def mass(**kw):
    a = dict(q=zeros(B, 2, 2 * H, 128, dtype=BF16), k_pool=zeros(P, H, 64, 128, dtype=BF16), block_table=zeros(B, 1),
             seq_lens=zeros(B), lse=zeros(B, 2, 2 * H, dtype=torch.float32), mass=zeros(B, H, S, dtype=torch.float32))
    opts = dict(row_weight=zeros(B, 2, dtype=torch.float32), prev=zeros(B, H, S, dtype=torch.float32))
    for k, v in kw.items():
        (a if k in a else opts)[k] = v
    skv.attn_key_mass(*a.values(), max_seq_len=S, **opts)


def f32(*shape):
    return zeros(*shape, dtype=torch.float32)


@pytest.mark.parametrize("call,kw", [
    (evict, lambda: dict(seq_lens=zeros(1, B))), (evict, lambda: dict(keep_ids=zeros(B, N, H))),
    (evict, lambda: dict(keep_ids=zeros(H, B, N))), (evict, lambda: dict(keep_lens=zeros(B, 1))),
    (compact, lambda: dict(v_pool=zeros(H, P, 64, 128, dtype=BF16))), (compact, lambda: dict(block_table=zeros(1, B, 1))),
    (compact, lambda: dict(dst=(zeros(P, H, 128, 64, dtype=BF16), zeros(P, H, 64, 128, dtype=BF16), zeros(B, 2)))),
    (compact, lambda: dict(dst=(zeros(P, H, 64, 128, dtype=BF16), zeros(P, 64, H, 128, dtype=BF16), zeros(B, 2)))),
    (compact, lambda: dict(dst=(None, None, zeros(1, B, 2)))), (compact, lambda: dict(mass=f32(H, B, S))),
    (compact, lambda: dict(first=zeros(1, B))), (compact, lambda: dict(new_lens=zeros(B, 1))),
    (mass, lambda: dict(prev=f32(H, B, S))), (mass, lambda: dict(mass=f32(H, B, S))),
    (mass, lambda: dict(lse=f32(B, 2 * H, 2))),
    (mass, lambda: dict(row_weight=f32(1, B, 2))),
])
def test_other_shapes_are_refused(call, kw):
    call()
    with pytest.raises(skv.SkvError) as e:
        call(**kw())
    assert e.value.status == skv.SKV_EINVAL
    torch.cuda.synchronize()


def test_lengths_may_lie_side_by_side():
    """Rows of one tensor: no word is shared."""
    lens = torch.tensor([[6, 5], [0, 0], [0, 0]], dtype=torch.int32, device="cuda")
    evict(seq_lens=lens[0], keep_lens=lens[1])
    compact(seq_lens=lens[0], keep_lens=lens[1], new_lens=lens[2], first=None, dst=None)
    torch.cuda.synchronize()
    assert lens.tolist() == [[6, 5], [4, 4], [4, 4]]
    with pytest.raises(skv.SkvError) as e:
        evict(seq_lens=lens[0], keep_lens=lens[0])
    assert e.value.status == skv.SKV_EINVAL
