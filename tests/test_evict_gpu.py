"""Eviction on the GPU: the kept positions and the compacted cache equal the
oracle's exactly (both only choose and move values)."""
import numpy as np
import pytest
import torch

import oracle
import sparse_kv_b200 as skv
from test_tree_gpu import Problem, bits

pytestmark = pytest.mark.gpu

NAN = float("nan")


def select(mass, lens, keep, sink=0, recent=0, max_len=None, status=None):
    B, H, S = mass.shape
    ids = torch.full((B, H, keep), 12345, dtype=torch.int32, device="cuda")
    kl = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    skv.attn_evict_select(mass, sl, keep, ids, kl, max_seq_len=max_len or S, sink=sink, recent=recent, status=status)
    torch.cuda.synchronize()
    return ids, kl


def check_select(mass, lens, keep, sink=0, recent=0):
    ids, kl = select(mass, lens, keep, sink, recent)
    m = mass.cpu().numpy()
    for b, n in enumerate(lens):
        assert int(kl[b]) == min(n, keep)
        for h in range(mass.shape[1]):
            want = oracle.evict_keep(m[b, h, :n], keep, sink, recent)
            got = ids[b, h].cpu().numpy()
            assert np.array_equal(got[:len(want)], want), (b, h, got[:8], want[:8])
            assert (got[len(want):] == -1).all()


@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 1, 0), (7, 2, 3), (64, 0, 64), (64, 32, 32), (100, 4, 16),
                                              (1000, 64, 256), (5000, 0, 0)])
def test_select_lengths(keep, sink, recent):
    lens = [0, 1, 2, 63, 64, 65, 100, 101, 999, 1000, 1001, 4096, 4999]
    g = torch.Generator(device="cuda").manual_seed(keep)
    mass = torch.exp2(torch.randn(len(lens), 2, 4999, generator=g, device="cuda") * 4)
    check_select(mass, lens, keep, sink, recent)


@pytest.mark.parametrize("L,keep", [(2000, 500), (20000, 6001), (131071, 4096)])
def test_select_ties_and_special_values(L, keep):
    g = torch.Generator(device="cuda").manual_seed(L)
    x = torch.randn(6, 1, L, generator=g, device="cuda")
    x[0] = (x[0] * 2).round()                       # many equal values, zeros of both signs
    x[1] = 0.25                                     # all equal: the lowest positions
    x[2] = torch.where(x[2] > 1, x[2], torch.zeros_like(x[2]))
    x[3, 0, ::3] = NAN
    x[3, 0, 1::7] = float("inf")
    x[3, 0, 2::5] = float("-inf")
    x[4] = x[4].abs() * 1e-42                       # denormals
    x[5] = 1 + torch.arange(L, device="cuda") % 3 * 2.0 ** -23  # neighbours in the last bit
    check_select(x, [L, L, L, L, L, L - 17], keep, 16, 33)


@pytest.mark.parametrize("L,keep", [(4000, 3900), (17000, 16384), (40000, 36000)])
def test_select_many_equal_weights_again_and_again(L, keep):
    """The last kept weight is one of thousands of zeros: the digits are taken one after
    the other, call after call with the same result."""
    g = torch.Generator(device="cuda").manual_seed(L)
    x = torch.exp2(torch.randn(16, 4, L, generator=g, device="cuda") * 3 - 8)
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.2] = 0
    check_select(x[:1, :1].contiguous(), [L], keep, 64, 128)
    ids, kl = select(x, [L] * 16, keep, 64, 128)
    again = torch.empty_like(ids)
    sl = torch.full((16,), L, dtype=torch.int32, device="cuda")
    for _ in range(200):
        skv.attn_evict_select(x, sl, keep, again, kl, max_seq_len=L, sink=64, recent=128)
    torch.cuda.synchronize()
    assert torch.equal(ids, again)


@pytest.mark.parametrize("groups,L,keep", [(8, 131073, 16384), (2, 262149, 32768), (3, 524288, 65536), (1, 1048653, 300),
                                           (40, 200000, 25000), (1, 4194304, 500000)])
def test_select_of_long_caches(groups, L, keep):
    """Open tokens that fit in the lists of a cluster, that only fit where a CTA has an SM
    to itself, and that do not fit."""
    g = torch.Generator(device="cuda").manual_seed(L)
    x = torch.exp2(torch.randn(1, groups, L, generator=g, device="cuda") * 3 - 8)
    check_select(x, [L], keep, 64, 100)


def test_select_bad_length_is_reported():
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, kl = select(torch.rand(2, 1, 50, device="cuda"), [51, 50], 10, max_len=50, status=st)
    assert int(st.item()) == skv.DEV_BITS["bad_seqlen"]
    assert int(kl[0]) == 0 and (ids[0] == -1).all() and int(kl[1]) == 10


def rows_of(pool, table, b, h, n):
    pages = table[b, :(n + 63) // 64].long().cpu()
    return pool.cpu()[pages, h].reshape(-1, 128)[:n]


def subset(B, H, lens, first, count, width, seed):
    r = np.random.default_rng(seed)
    ids = np.full((B, H, width), -1, dtype=np.int32)
    for b in range(B):
        for h in range(H):
            span = np.arange(first[b], lens[b])
            ids[b, h, :count[b]] = np.sort(r.choice(span, count[b], replace=False))
    return torch.tensor(ids, device="cuda")


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("first,count", [
    ([0, 0, 0, 0, 0], [3000, 700, 0, 1, 129]),          # eviction; nothing kept; all kept
    ([0, 0, 0, 0, 0], [4000, 1, 5, 64, 60]),
    ([3990, 690, 0, 1, 200], [5, 0, 5, 64, 1]),         # commit at the end; first at a page's border and inside one
    ([64, 640, 3, 63, 128], [1000, 60, 2, 66, 72]),
])
def test_compact(shared, copy, first, count):
    lens = [4000, 700, 5, 129, 200]
    count = [min(c, n - f) for c, n, f in zip(count, lens, first)]
    p = Problem(5, 6, 3, 1, lens, seed=91).to_gpu()
    mass = torch.rand(5, 3, 4003, device="cuda")
    m0, k0, v0 = mass.clone(), p.k.clone(), p.v.clone()
    ids = subset(5, 1 if shared else 3, lens, first, count, max(max(count), 1) + 3, 7)
    kl = torch.tensor(count, dtype=torch.int32, device="cuda")
    f = torch.tensor(first, dtype=torch.int32, device="cuda")
    nl = torch.full((5,), -9, dtype=torch.int32, device="cuda")
    dst, to_k, to_v, table = None, p.k, p.v, p.bt
    if copy:
        need = [(x + c + 63) // 64 for x, c in zip(first, count)]
        table = torch.full((5, max(max(need), 1)), -1, dtype=torch.int32)
        perm, at = torch.randperm(sum(need) + 2), 0
        for b in range(5):
            table[b, :need[b]] = perm[at:at + need[b]].int()
            at += need[b]
        table = table.cuda()
        to_k = torch.full((sum(need) + 2, 3, 64, 128), NAN, dtype=torch.bfloat16, device="cuda")
        to_v = torch.full_like(to_k, NAN)
        dst = (to_k, to_v, table)
    b_k, b_v = to_k.clone(), to_v.clone()
    skv.attn_compact_cache(p.k, p.v, p.bt, p.sl, ids, kl, nl, first=f, dst=dst, mass=mass, max_seq_len=4000,
                           status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    assert nl.tolist() == [x + c for x, c in zip(first, count)]
    for b in range(5):
        a, e = first[b], first[b] + count[b]
        for h in range(3):
            i = ids[b, 0 if shared else h, :count[b]].long().cpu()
            for now, was, src, base in ((to_k, k0, p.bt, b_k), (to_v, v0, p.bt, b_v)):
                got = rows_of(now, table, b, h, e)
                assert same(got[a:e], rows_of(was, src, b, h, lens[b])[i])
                assert same(got[:a], rows_of(base, table, b, h, e)[:a])
            if not copy:  # what lies behind is left as it was
                assert same(rows_of(p.k, p.bt, b, h, lens[b])[e:], rows_of(k0, p.bt, b, h, lens[b])[e:])
            assert torch.equal(mass[b, h, a:e].cpu(), m0[b, h].cpu()[i])
            assert torch.equal(mass[b, h, e:], m0[b, h, e:]) and torch.equal(mass[b, h, :a], m0[b, h, :a])


def test_compact_copies_in_any_order():
    p = Problem(1, 1, 1, 1, [300], seed=95).to_gpu()
    ids = torch.tensor([[[299, 0, 7, 7, 64, 63]]], dtype=torch.int32, device="cuda")
    to = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device="cuda")
    to2, nl = torch.zeros_like(to), torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.attn_compact_cache(p.k, p.v, p.bt, p.sl, ids, torch.tensor([6], dtype=torch.int32, device="cuda"), nl,
                           dst=(to, to2, torch.zeros(1, 1, dtype=torch.int32, device="cuda")), max_seq_len=300,
                           status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0 and int(nl) == 6
    assert same(to[0, 0, :6].cpu(), rows_of(p.k, p.bt, 0, 0, 300)[ids[0, 0].long().cpu()])
    assert same(to2[0, 0, :6].cpu(), rows_of(p.v, p.bt, 0, 0, 300)[ids[0, 0].long().cpu()])
    assert (to[0, 0, 6:] == 0).all()


def test_compact_reports_bad_entries():
    """Bad ids and pages: that row does not move, the others do.  Bad lengths: the
    sequence is left as it was."""
    p = Problem(3, 1, 1, 1, [300, 300, 300], seed=97).to_gpu()
    k0, v0 = p.k.clone(), p.v.clone()
    ids = torch.tensor([[[0, 5, 300, 2, -1, 200, 290]], [[0, 1, 2, 3, 4, 5, 6]], [[9, 9, 9, 9, 9, 9, 9]]],
                       dtype=torch.int32, device="cuda")
    kl = torch.tensor([7, 7, 8], dtype=torch.int32, device="cuda")
    nl = torch.zeros(3, dtype=torch.int32, device="cuda")
    f = torch.tensor([0, 301, 0], dtype=torch.int32, device="cuda")
    skv.attn_compact_cache(p.k, p.v, p.bt, p.sl, ids, kl, nl, first=f, max_seq_len=300, status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == skv.DEV_BITS["bad_order"] | skv.DEV_BITS["bad_seqlen"]
    assert nl.tolist() == [7, 300, 300]
    want = rows_of(k0, p.bt, 0, 0, 300).clone()
    want[1], want[5], want[6] = want[5].clone(), want[200].clone(), want[290].clone()
    assert same(rows_of(p.k, p.bt, 0, 0, 300), want)
    for b in (1, 2):
        assert same(rows_of(p.k, p.bt, b, 0, 300), rows_of(k0, p.bt, b, 0, 300))
    ids[0, 0] = torch.tensor([190, 191, 200, 256, 257, 258, 259])
    one = Problem(1, 1, 1, 1, [300], seed=98).to_gpu()
    was = rows_of(one.k, one.bt, 0, 0, 300).clone()
    one.bt[0, 3] = -1  # tokens 192 .. 255
    skv.attn_compact_cache(one.k, one.v, one.bt, one.sl, ids[:1].contiguous(), kl[:1].contiguous(), nl[:1].contiguous(),
                           max_seq_len=300, status=one.status)
    torch.cuda.synchronize()
    assert int(one.status.item()) == skv.DEV_BITS["bad_page"]
    got = one.k.cpu()[one.table[0, 0].long(), 0]
    assert same(got[[0, 1, 3, 4, 5, 6]], was[[190, 191, 256, 257, 258, 259]]) and same(got[2], was[2])


def test_refused_arguments():
    p = Problem(2, 2, 2, 1, [100, 50], seed=99).to_gpu()
    ids = torch.zeros(2, 2, 8, dtype=torch.int32, device="cuda")
    kl = torch.ones(2, dtype=torch.int32, device="cuda")
    nl = torch.zeros(2, dtype=torch.int32, device="cuda")

    def refused(**kw):
        a = dict(k_pool=p.k, v_pool=p.v, block_table=p.bt, seq_lens=p.sl, keep_ids=ids, keep_lens=kl, new_lens=nl)
        opts = dict(max_seq_len=100)
        for k, v in kw.items():
            (a if k in a else opts)[k] = v
        with pytest.raises(skv.SkvError) as e:
            skv.attn_compact_cache(*a.values(), **opts)
        assert e.value.status == skv.SKV_EINVAL

    refused(new_lens=p.sl)
    refused(new_lens=kl)
    refused(keep_ids=torch.zeros(2, 3, 8, dtype=torch.int32, device="cuda"))
    refused(keep_ids=ids.long())
    refused(k_pool=p.k.float())
    refused(v_pool=p.v[..., ::2])
    refused(mass=torch.zeros(2, 2, 99, device="cuda"))
    refused(dst=(p.k, None, p.bt))
    refused(max_seq_len=1000)
    m = torch.rand(2, 2, 100, device="cuda")
    for kw in (dict(keep=0, ids=ids[..., :0]), dict(sink=5, recent=4), dict(sink=-1), dict(recent=-1),
               dict(max_seq_len=101), dict(ids=ids.long()), dict(mass=m.double())):
        with pytest.raises(skv.SkvError) as e:
            skv.attn_evict_select(kw.get("mass", m), p.sl, kw.get("keep", 8), kw.get("ids", ids), kl,
                                  sink=kw.get("sink", 0), recent=kw.get("recent", 0),
                                  max_seq_len=kw.get("max_seq_len", 100))
        assert e.value.status == skv.SKV_EINVAL


def test_draft_commit_evict_decode():
    """One round of serving: verify a tree, commit its accepted path, count the
    weight, shrink the cache to a budget, decode over what is left."""
    B, Hq, Hkv, T, lens = 2, 8, 2, 8, [900, 330]
    p = Problem(B, Hq, Hkv, T, lens, seed=101).to_gpu()
    p.words = [[0b1, 0b11, 0b101, 0b1011, 0b10101, 0b110101, 0b1000001, 0b10001011]] * 2
    p.mask = torch.tensor(p.words, dtype=torch.int64)
    p.opts["tree_mask"] = p.mask.cuda()
    o, l = p.decode()
    p.check(o, l)
    path = [[0, 2, 4, 5], [0, 1]]
    w = torch.zeros(B, T, device="cuda")
    for b in range(B):
        w[b, path[b]] = 1
    mass = torch.zeros(B, Hkv, p.Lmax, device="cuda")
    p.mass(l, weight=w, prev=mass, into=mass)
    ctx = [n - T for n in lens]
    ids = torch.full((B, 1, T), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        ids[b, 0, :len(path[b])] = torch.tensor([ctx[b] + j for j in path[b]])
    lens2 = torch.zeros(B, dtype=torch.int32, device="cuda")
    skv.attn_compact_cache(p.k, p.v, p.bt, p.sl, ids, torch.tensor([4, 2], dtype=torch.int32, device="cuda"), lens2,
                           first=torch.tensor(ctx, dtype=torch.int32, device="cuda"), mass=mass, max_seq_len=p.Lmax,
                           status=p.status)
    keep = 256
    kept = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")
    kl, lens3 = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    skv.attn_evict_select(mass, lens2, keep, kept, kl, sink=4, recent=32, max_seq_len=p.Lmax, status=p.status)
    before = mass.clone()
    skv.attn_compact_cache(p.k, p.v, p.bt, lens2, kept, kl, lens3, mass=mass, max_seq_len=p.Lmax, status=p.status)
    q = torch.randn(B, 1, Hq, 128, device="cuda").bfloat16()
    out, lse = torch.empty(B, 1, Hq, 128, device="cuda"), torch.empty(B, 1, Hq, device="cuda")
    skv.attn_decode(q, p.k, p.v, p.bt, lens3, out, lse, max_seq_len=keep, scale=p.scale, status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0 and lens3.tolist() == [256, 256]
    for b in range(B):
        tokens = list(range(ctx[b])) + [ctx[b] + j for j in path[b]]
        assert int(lens2[b]) == len(tokens)
        for h in range(Hkv):
            m = before[b, h, :len(tokens)].cpu().numpy()
            sel = oracle.evict_keep(m, keep, 4, 32)
            assert np.array_equal(kept[b, h].cpu().numpy(), sel)
            at = [tokens[i] for i in sel]
            O, le = oracle.attend(bits(q[b, 0, h * 4:h * 4 + 4])[None], bits(p.K[b][h][at])[None],
                                  bits(p.V[b][h][at])[None], [[np.arange(keep)] * 4], p.scale)
            assert np.abs(out[b, 0, h * 4:h * 4 + 4].cpu().numpy() - O[0]).max() <= 2e-3
            assert np.abs(lse[b, 0, h * 4:h * 4 + 4].cpu().numpy() - le[0]).max() <= 1e-4 * max(1, np.abs(le).max())
