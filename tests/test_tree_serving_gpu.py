"""The drafted-token and cache-budget calls as a server makes them: one token a sequence
with each option, batches of which few sequences have drafts, smooth weights, long
compactions, captured steps.  Tolerances as in test_tree_gpu."""
import numpy as np
import pytest
import torch

import oracle
import sparse_kv_b200 as skv
from test_evict_gpu import check_select, rows_of, same
from test_tree_gpu import Problem, bits

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("opt", [dict(softcap=8.0), dict(slopes=True), dict(window=(4, 96)), dict(window=(0, 1)),
                                 dict(window=(7, 0)), dict(softcap=30.0, slopes=True), dict(slopes=True, window=(64, 700)),
                                 dict(softcap=2.0, slopes=True, window=(1, 300)), dict(scale=-0.1, softcap=8.0)])
def test_one_token_with_options(G, opt):
    lens = [1, 2, 64, 65, 128, 129, 640, 3001]
    p = Problem(len(lens), 2 * G, 2, 1, lens, seed=G, gain=2.0, tree="chain", **opt).to_gpu()
    o, l = p.decode()
    p.check(o, l)
    prev = torch.rand(len(lens), 2, p.Lmax, device="cuda")
    p.check_mass(p.mass(l, prev=prev, decay=0.9), l, None, prev, 0.9)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("L,opt", [(30000, dict(softcap=20.0, slopes=True)), (30000, dict(window=(64, 9000))),
                                   (30000, dict(slopes=True, window=(100, 20000)))])
def test_one_token_over_a_long_cache(L, opt):
    p = Problem(2, 8, 1, 1, [L, L - 4321], seed=L, tree="chain", **opt).to_gpu()
    o, l = p.decode()
    p.check(o, l)
    p.check_mass(p.mass(l), l)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_slopes_of_either_sign(sign):
    """Weights that fall, or grow, with the distance."""
    p = Problem(2, 8, 2, 5, [3000, 77], seed=11, slopes=True)
    p.slopes = sign * torch.linspace(0.001, 0.02, 8)
    p.to_gpu()
    o, l = p.decode()
    torch.cuda.synchronize()
    for b in range(2):
        for h in range(2):
            hs = slice(4 * h, 4 * h + 4)
            z = p.scores(b, h)
            O, lse = oracle.softmax_rows(z, bits(p.V[b][h]))
            # a bias is off by two roundings of itself: 2^-23 of the largest
            ez = p.score_error(b, h) + 2.0 ** -23 * 0.02 * 3000
            assert np.abs(o[b, :, hs].cpu().numpy() - O).max() <= 2 * float(p.V[b][h].float().abs().max()) * (ez + 2.0 ** -17)
            assert (np.abs(l[b, :, hs].cpu().numpy() - lse) <= ez + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)).all()


@pytest.mark.parametrize("where", ["first", "last", "spread"])
@pytest.mark.parametrize("window", [None, (10, 50)])
def test_few_of_many_sequences_have_drafts(where, window):
    B, T = 700, 4
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(T, 400, B)]
    some = {"first": range(3), "last": range(B - 3, B), "spread": range(17, B, 97)}[where]
    p = Problem(B, 8, 2, T, lens, [T if b in some else 0 for b in range(B)], seed=6, window=window).to_gpu()
    o, l = p.decode()
    p.check(o, l)
    assert int(p.status.item()) == 0


def test_no_sequence_has_drafts():
    p = Problem(40, 8, 2, 3, [100 + i for i in range(40)], [0] * 40, seed=7).to_gpu()
    o, l = p.decode()
    torch.cuda.synchronize()
    assert torch.isnan(o).all() and torch.isnan(l).all() and int(p.status.item()) == 0


@pytest.mark.parametrize("L,keep", [(131072, 16384), (131072, 65536), (40000, 20000), (300000, 150000)])
@pytest.mark.parametrize("spread", ["uniform", "third of an octave", "rising", "two values"])
def test_eviction_of_smooth_weights(L, keep, spread):
    g = torch.Generator(device="cuda").manual_seed(keep)
    x = torch.rand(1, 3, L, generator=g, device="cuda")
    if spread == "third of an octave":
        x = torch.exp2(torch.randn(1, 3, L, generator=g, device="cuda") * 0.3 - 8)
    elif spread == "rising":
        x = (torch.arange(L, device="cuda") * 1e-4).expand(1, 3, L).contiguous()
    elif spread == "two values":
        x = torch.where(x < 0.5, 0.5, 0.25)
    check_select(x, [L], keep, 64, 1000)


@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("B,Hkv,L,keep", [(1, 8, 32768, 30000), (1, 1, 50000, 49000), (40, 8, 700, 650)])
def test_long_compactions(B, Hkv, L, keep, copy):
    g = torch.Generator(device="cuda").manual_seed(L)
    blocks = (L + 63) // 64
    k = torch.randn(B * blocks, Hkv, 64, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(k.shape, generator=g, device="cuda", dtype=torch.bfloat16)
    table = torch.randperm(B * blocks, generator=g, device="cuda").int().view(B, blocks)
    ids = torch.rand(B, Hkv, L, generator=g, device="cuda").argsort(-1)[..., :keep].sort(-1).values.int()
    mass = torch.rand(B, Hkv, L, generator=g, device="cuda")
    k0, v0, m0 = k.clone(), v.clone(), mass.clone()
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    kl, nl = torch.full_like(lens, keep), torch.zeros_like(lens)
    dst, to_k, to_v, to_table = None, k, v, table
    if copy:
        n = (keep + 63) // 64
        to_table = torch.randperm(B * n, generator=g, device="cuda").int().view(B, n)
        to_k = torch.zeros(B * n, Hkv, 64, 128, dtype=torch.bfloat16, device="cuda")
        to_v = torch.zeros_like(to_k)
        dst = (to_k, to_v, to_table)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    skv.attn_compact_cache(k, v, table, lens, ids, kl, nl, dst=dst, mass=mass, max_seq_len=L, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and (nl == keep).all()
    for b in {0, B - 1}:
        for h in {0, Hkv - 1}:
            at = ids[b, h].long().cpu()
            assert same(rows_of(to_k, to_table, b, h, keep), rows_of(k0, table, b, h, L)[at])
            assert same(rows_of(to_v, to_table, b, h, keep), rows_of(v0, table, b, h, L)[at])
    assert torch.equal(mass[..., :keep], m0.gather(2, ids.long())) and torch.equal(mass[..., keep:], m0[..., keep:])
    if copy:
        assert same(k, k0) and same(v, v0)


def test_captured_serving_step():
    """Copies, verification, mass, eviction and compaction in one graph: replayed on new
    inputs it does what the calls do one by one."""
    B, Hq, Hkv, T, keep = 3, 16, 4, 5, 200
    lens = [700, 300, 555]
    p = Problem(B, Hq, Hkv, T, lens, seed=13).to_gpu()
    q_in, k_in, v_in = p.qd.clone(), p.k.clone(), p.v.clone()
    ws = p.workspace()
    out, lse = p.buffers()
    prev = torch.rand(B, Hkv, p.Lmax, device="cuda")
    mass = torch.zeros_like(prev)
    ids = torch.zeros(B, Hkv, keep, dtype=torch.int32, device="cuda")
    kl, nl = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        p.k.copy_(k_in)
        p.v.copy_(v_in)
        p.qd.copy_(q_in)
        skv.attn_tree_decode(p.qd, p.k, p.v, p.bt, p.sl, out, lse, workspace=ws, **p.opts)
        skv.attn_key_mass(p.qd, p.k, p.bt, p.sl, lse, mass, prev=prev, decay=0.5, **p.opts)
        skv.attn_evict_select(mass, p.sl, keep, ids, kl, sink=4, recent=16, max_seq_len=p.Lmax, status=p.status)
        skv.attn_compact_cache(p.k, p.v, p.bt, p.sl, ids, kl, nl, mass=mass, max_seq_len=p.Lmax, status=p.status)

    def state():
        torch.cuda.synchronize()
        return [x.clone() for x in (out, lse, mass, ids, kl, nl, p.k.view(torch.int16), p.v.view(torch.int16))]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q_in.copy_(torch.randn(q_in.shape, generator=g, device="cuda"))
        prev.copy_(torch.rand(prev.shape, generator=g, device="cuda"))
        step()
        one = state()
        mass.zero_()
        out.fill_(NAN)
        graph.replay()
        graph.replay()
        for x, y in zip(one, state()):
            assert torch.equal(x.nan_to_num() if x.is_floating_point() else x, y.nan_to_num() if y.is_floating_point() else y)
        p.q = q_in.cpu()
        p.check(out, lse)
    assert int(p.status.item()) == 0
