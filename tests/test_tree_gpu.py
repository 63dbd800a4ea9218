"""Draft-tree attention and key mass on the GPU against the fp64 oracle.

Tolerances.  A score is a sum of 128 exact products in fp32: its error is at most
128 * 2^-24 * scale * sum |q_i k_i| (twice that where the tensor core drops bits
instead of rounding), plus 8 roundings of 2^-24 on numbers as large as the
largest score, bias or cap.  Call the sum of these ez.  A weight e^(z - m) then
has a relative error of ez + 2^-21 (exponential) and enters the product with V
as two bf16 terms that keep it to 2^-18, so an output
sum p v / sum p is off by at most 2 max|v| (ez + 2^-17); the log-sum-exp by
ez + 2^-20 + 2^-22 |lse|; a key's mass by its relative error times the mass, and by
2^-126 for each of its rows: a weight below the smallest normal number counts as 0.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import sparse_kv_b200 as skv

pytestmark = pytest.mark.gpu

NAN = float("nan")


def bits(x):
    return x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


class Problem:
    """A paged cache whose unused rows hold NaN, its queries and its trees."""

    def __init__(self, B, Hq, Hkv, T, lens, drafts=None, tree="random", seed=0, gain=1.0, scale=None,
                 softcap=0.0, slopes=False, window=None):
        g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.T, self.G = B, Hq, Hkv, T, Hq // Hkv
        self.lens, self.drafts = lens, drafts or [T] * B
        self.scale, self.softcap, self.window = 1 / math.sqrt(128) if scale is None else scale, softcap, window
        self.Lmax = max(max(lens), 1)
        mb = (self.Lmax + 63) // 64
        nb = [(n + 63) // 64 for n in lens]
        pages = max(sum(nb), 1)
        perm = torch.randperm(pages, generator=g)
        self.table = torch.full((B, mb), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :nb[b]] = perm[at:at + nb[b]].int()
            at += nb[b]
        self.q = (torch.randn(B, T, Hq, 128, generator=g) * gain).bfloat16()
        self.K = [torch.randn(Hkv, n, 128, generator=g).bfloat16() for n in lens]
        self.V = [torch.randn(Hkv, n, 128, generator=g).bfloat16() for n in lens]
        self.words = []
        for b in range(B):
            n = self.drafts[b]
            w = oracle.tree_chain(n)
            if tree == "random":     # each token below an earlier one
                w = []
                for t in range(n):
                    above = w[int(torch.randint(t, (1,), generator=g))] if t and torch.rand(1, generator=g) < 0.8 else 0
                    w.append(above | (1 << t))
            elif tree == "any":      # any bits at all, rows without their own bit and without any
                w = [int(torch.randint(1 << 30, (1,), generator=g)) * int(torch.randint(1 << 30, (1,), generator=g))
                     & ((1 << n) - 1) for _ in range(n)]
                w = [0] + w[1:] if n else w
            self.words.append(w)
        self.chain = tree == "chain"
        self.mask = torch.zeros(B, T, dtype=torch.int64)
        for b in range(B):
            for t in range(T):
                w = self.words[b][t] if t < self.drafts[b] else 0
                w |= ~((1 << self.drafts[b]) - 1) & ((1 << 64) - 1)  # bits past the drafts are ignored
                self.mask[b, t] = w - (1 << 64) if w >> 63 else w
        self.slopes = 2.0 ** (-8 * torch.arange(1, Hq + 1) / Hq) if slopes else None
        self.pages = pages
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def to_gpu(self):
        k = torch.full((self.pages, self.Hkv, 64, 128), NAN, dtype=torch.bfloat16)
        v = torch.full_like(k, NAN)
        for b, n in enumerate(self.lens):
            for j in range((n + 63) // 64):
                a, e = j * 64, min(n, j * 64 + 64)
                k[self.table[b, j], :, :e - a] = self.K[b][:, a:e]
                v[self.table[b, j], :, :e - a] = self.V[b][:, a:e]
        self.k, self.v, self.bt = k.cuda(), v.cuda(), self.table.cuda()
        self.sl = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.tl = torch.tensor(self.drafts, dtype=torch.int32, device="cuda")
        self.qd = self.q.cuda()
        self.opts = dict(max_seq_len=self.Lmax, scale=self.scale, softcap=self.softcap, window=self.window,
                         tree_lens=self.tl, tree_mask=None if self.chain else self.mask.cuda(),
                         slopes=None if self.slopes is None else self.slopes.cuda(), status=self.status)
        return self

    def buffers(self):
        out = torch.full((self.B, self.T, self.Hq, 128), NAN, device="cuda")
        return out, torch.full((self.B, self.T, self.Hq), NAN, device="cuda")

    def workspace(self):
        o, l = self.buffers()
        n = skv.tree_workspace_size(self.qd, self.k, self.v, self.bt, self.sl, o, l, **self.opts)
        return torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")  # NaN bytes

    def decode(self, stream=None, workspace=None):
        o, l = self.buffers()
        ws = self.workspace() if workspace is None else workspace
        skv.attn_tree_decode(self.qd, self.k, self.v, self.bt, self.sl, o, l, workspace=ws, stream=stream, **self.opts)
        return o, l

    def scores(self, b, h):
        n, G = self.drafts[b], self.G
        sl = None if self.slopes is None else self.slopes.double().numpy()[h * G:(h + 1) * G]
        return oracle.tree_scores(bits(self.q[b, :n, h * G:(h + 1) * G]), bits(self.K[b][h]), self.words[b],
                                  self.scale, self.softcap, sl, self.window)

    def score_error(self, b, h):
        n, G = self.drafts[b], self.G
        if n == 0:
            return 0.0
        q, k = self.q[b, :n, h * G:(h + 1) * G].float().abs().reshape(-1, 128), self.K[b][h].float().abs()
        dot = float((q @ k.T).max()) * abs(self.scale) if k.shape[0] else 0.0
        big = max(dot, self.softcap) + (float(self.slopes.max()) * (self.lens[b] + 64) if self.slopes is not None else 0)
        if self.slopes is not None:  # weights of tokens e^-40 below the best do not show
            big = max(dot, self.softcap) + 40 + 2 * dot
        return 2 * 128 * 2.0 ** -24 * dot + 8 * 2.0 ** -24 * big

    def check(self, o, l, groups=None):
        torch.cuda.synchronize()
        o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
        for b in range(self.B):
            n = self.drafts[b]
            assert np.isnan(o[b, n:]).all() and np.isnan(l[b, n:]).all(), "rows past the drafts were written"
            for h in range(self.Hkv) if groups is None else [h for (x, h) in groups if x == b]:
                if n == 0:
                    continue
                hs = slice(h * self.G, (h + 1) * self.G)
                O, lse = oracle.softmax_rows(self.scores(b, h), bits(self.V[b][h]))
                ez = self.score_error(b, h)
                vmax = float(self.V[b][h].float().abs().max()) if self.lens[b] else 0.0
                assert np.isfinite(o[b, :n, hs]).all()
                err = np.abs(o[b, :n, hs] - O).max()
                assert err <= 2 * vmax * (ez + 2.0 ** -17), (b, h, err, ez)
                empty = np.isneginf(lse)
                assert np.array_equal(empty, np.isneginf(l[b, :n, hs]))
                d = np.abs(l[b, :n, hs][~empty] - lse[~empty])
                assert (d <= ez + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse[~empty])).all(), (b, h, d.max(), ez)

    def mass(self, lse, weight=None, prev=None, decay=1.0, stride=None, into=None, stream=None):
        m = into if into is not None else torch.full((self.B, self.Hkv, stride or self.Lmax), NAN, device="cuda")
        skv.attn_key_mass(self.qd, self.k, self.bt, self.sl, lse, m, row_weight=weight, prev=prev, decay=decay,
                          stream=stream, **self.opts)
        return m

    def check_mass(self, m, lse, weight=None, prev=None, decay=1.0, groups=None):
        torch.cuda.synchronize()
        m, lse = m.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(self.B):
            n, L = self.drafts[b], self.lens[b]
            assert np.isnan(m[b, :, L:]).all(), "entries past the sequence were written"
            for h in range(self.Hkv) if groups is None else [h for (x, h) in groups if x == b]:
                hs = slice(h * self.G, (h + 1) * self.G)
                w = np.ones(n) if weight is None else weight[b, :n].double().cpu().numpy()
                want = oracle.key_mass(self.scores(b, h), lse[b, :n, hs], w)
                near = max([abs(x) for x in lse[b, :n, hs].ravel() if np.isfinite(x)], default=0.0)
                rel = self.score_error(b, h) + 2.0 ** -21 + 2.0 ** -22 * near + n * self.G * 2.0 ** -24
                old = 0.0 if prev is None else decay * prev[b, h, :L].double().cpu().numpy()
                tol = n * self.G * 2.0 ** -126 * np.abs(w).max(initial=0) + rel * oracle.key_mass(self.scores(b, h), lse[b, :n, hs], np.abs(w)) + 2.0 ** -22 * np.abs(old)
                bad = np.abs(m[b, h, :L] - (old + want)) > tol
                assert not bad.any(), (b, h, np.nonzero(bad)[0][:4], m[b, h, :L][bad][:4], (old + want)[bad][:4])


EDGES = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 300]


@pytest.mark.parametrize("G,T", [(1, 1), (4, 1), (8, 1), (4, 2), (1, 5), (2, 8), (4, 8), (8, 7), (4, 16), (4, 20),
                                 (8, 13), (4, 32), (8, 16), (2, 64), (4, 40), (8, 40), (4, 64), (8, 64)])
def test_tree_lengths_and_groups(G, T):
    lens = [max(e, T) for e in EDGES] + [1000]
    p = Problem(len(lens), 2 * G, 2, T, lens, seed=G * 100 + T).to_gpu()
    o, l = p.decode()
    p.check(o, l)
    p.check_mass(p.mass(l), l)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("tree", ["chain", "random", "any"])
@pytest.mark.parametrize("opt", [dict(), dict(softcap=5.0), dict(slopes=True), dict(window=(3, 50)),
                                 dict(softcap=20.0, slopes=True, window=(64, 130)), dict(window=(0, 2)),
                                 dict(window=(70, 0))])
def test_tree_masks_and_options(tree, opt):
    # ragged drafts, among them none at all and a sequence that is nothing but drafts
    lens, drafts = [500, 37, 6, 129, 0, 12], [11, 0, 6, 12, 0, 12]
    p = Problem(6, 8, 2, 12, lens, drafts, tree=tree, seed=7, gain=3.0, **opt).to_gpu()
    o, l = p.decode()
    p.check(o, l)
    w = torch.rand(6, 12, device="cuda") - 0.3
    w[:, 1] = 0
    prev = torch.rand(6, 2, p.Lmax + 5, device="cuda")
    m = p.mass(l, weight=w, prev=prev, decay=0.5, stride=p.Lmax + 5)
    p.check_mass(m, l, w, prev, 0.5)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("order", ["rising", "falling", "spikes"])
@pytest.mark.parametrize("G,T", [(4, 4), (4, 30), (8, 32)])
def test_tree_peaky_scores(order, G, T):
    """Scores over a range of about 200: the running maximum moves in every tile, or
    only at a few, and by more than the weights' range."""
    L = 1500
    p = Problem(2, 2 * G, 2, T, [L, L - 77], seed=21, tree="random")
    u = torch.nn.functional.normalize(torch.randn(128, generator=torch.Generator().manual_seed(5)), dim=0)
    p.q = (p.q.float() * 0.3 + 40 * u).bfloat16()
    for b in range(2):
        n = p.lens[b]
        a = torch.linspace(-28, 28, n)
        if order == "falling":
            a = a.flip(0)
        if order == "spikes":
            a = torch.where(torch.arange(n) % 211 == 100, torch.arange(n) * 0.03, torch.tensor(-20.0))
        p.K[b] = (p.K[b].float() * 0.1 + a[None, :, None] * u).bfloat16()
    o, l = p.to_gpu().decode()
    p.check(o, l)
    p.check_mass(p.mass(l), l)


@pytest.mark.parametrize("kw", [dict(scale=-0.2), dict(scale=-0.2, softcap=3.0), dict(scale=1e-9), dict(scale=0.4, softcap=0.05),
                                dict(scale=0.3, softcap=1e4, slopes=True)])
def test_tree_scales(kw):
    """Negative and vanishing scales; caps that every score passes, or none comes near."""
    p = Problem(2, 8, 2, 9, [400, 131], seed=23, **kw).to_gpu()
    o, l = p.decode()
    p.check(o, l)
    p.check_mass(p.mass(l), l)


def test_rows_past_the_drafts_may_hold_anything():
    p = Problem(4, 16, 2, 40, [300, 200, 150, 90], [40, 1, 17, 0], seed=25)
    for b in range(4):
        p.q[b, p.drafts[b]:] = NAN
    o, l = p.to_gpu().decode()
    p.check(o, l)
    w = torch.rand(4, 40, device="cuda")
    w[:, ::3] = 0
    p.qd[:, ::3] = NAN  # rows of weight 0 do not count, whatever they hold
    p.check_mass(p.mass(torch.where(torch.isnan(l), torch.zeros_like(l), l), weight=w), l.nan_to_num(), w)


def test_wide_trees_with_few_drafts():
    """512 rows at most, four row tiles: some have no row at all."""
    p = Problem(5, 8, 1, 64, [900, 500, 64, 257, 70], [64, 3, 17, 0, 33], seed=27).to_gpu()
    o, l = p.decode()
    p.check(o, l)
    p.check_mass(p.mass(l), l)


@pytest.mark.parametrize("G,T", [(4, 2), (8, 7), (8, 13)])
@pytest.mark.parametrize("order", ["any", "older is larger"])
def test_long_walks(G, T, order):
    """Over 32 tiles in a CTA's walk: 24 sequences over the same pages, one KV head.  In
    the second form the maxima grow all the way along the walk, newest to oldest."""
    L = 26500
    p = Problem(1, G, 1, T, [L], seed=29 + G, tree="random")
    if order != "any":
        u = torch.nn.functional.normalize(torch.randn(128, generator=torch.Generator().manual_seed(6)), dim=0)
        p.q = (p.q.float() * 0.3 + 20 * u).bfloat16()
        p.K[0] = (p.K[0].float() * 0.3 + torch.linspace(30, -30, L)[None, :, None] * u).bfloat16()
    p.to_gpu()
    n = 24
    assert n * (L + 127) // 128 // 148 > 32
    g = torch.Generator().manual_seed(1)
    more = (torch.randn(n - 1, T, G, 128, generator=g) * p.q.float().abs().mean()).bfloat16()
    p.q = torch.cat([p.q, more if order == "any" else p.q.expand(n - 1, -1, -1, -1) + 0.1 * more])
    p.B, p.lens, p.drafts, p.words = n, [L] * n, [T] * n, p.words * n
    p.K, p.V = p.K * n, p.V * n
    p.qd, p.bt = p.q.cuda(), p.bt.expand(n, -1).contiguous()
    p.sl, p.tl = p.sl.expand(n).contiguous(), p.tl.expand(n).contiguous()
    p.opts.update(tree_lens=p.tl, tree_mask=p.mask.expand(n, -1).contiguous().cuda())
    o, l = p.decode()
    p.check(o, l, [(0, 0), (11, 0), (23, 0)])
    p.check_mass(p.mass(l), l, groups=[(0, 0), (12, 0), (23, 0)])


def test_one_token_equals_attn_decode():
    p = Problem(3, 8, 2, 1, [700, 64, 1], tree="chain", seed=31).to_gpu()
    o, l = p.decode()
    o2, l2 = p.buffers()
    n = skv.decode_workspace_size(p.qd, p.k, p.v, p.bt, p.sl, o2, l2, max_seq_len=700)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    skv.attn_decode(p.qd, p.k, p.v, p.bt, p.sl, o2, l2, max_seq_len=700, workspace=ws)
    torch.cuda.synchronize()
    p.check(o2, l2)
    p.check(o, l)


@pytest.mark.parametrize("B,Hkv,G,T,L", [(1, 1, 4, 8, 40000), (1, 2, 8, 40, 9000), (20, 8, 4, 4, 1500),
                                         (40, 1, 1, 3, 700), (3, 4, 2, 64, 5000)])
def test_tree_shared_out_over_the_gpu(B, Hkv, G, T, L):
    """Few long sequences (many pieces of one KV group) and many short ones."""
    lens = [L - (i * 997) % (L // 2) for i in range(B)]
    p = Problem(B, Hkv * G, Hkv, T, lens, seed=B + L).to_gpu()
    o, l = p.decode()
    groups = [(0, 0), (B - 1, Hkv - 1), (B // 2, Hkv // 2)]
    p.check(o, l, groups)
    p.check_mass(p.mass(l), l, groups=groups)
    o2, l2 = p.decode()  # equal inputs, equal bits
    assert torch.equal(o.nan_to_num(), o2.nan_to_num()) and torch.equal(l.nan_to_num(), l2.nan_to_num())


def test_window_pages_need_not_be_mapped():
    """Outside the window nothing is read: pages are unmapped and rows hold NaN."""
    p = Problem(2, 8, 2, 5, [1000, 777], seed=41, window=(64, 200))
    p.to_gpu()
    for b in range(2):
        lo = (p.lens[b] - 5 + 1 - 200) // 64
        p.bt[b, 1:lo] = -1
    o, l = p.decode()
    p.check(o, l)
    assert int(p.status.item()) == 0
    p.check_mass(p.mass(l), l)
    assert int(p.status.item()) == 0


def test_infinities_where_no_row_looks():
    p = Problem(1, 4, 1, 4, [200], tree="any", seed=43)
    p.words[0] = [0b0001, 0b0011, 0b0001, 0b0011]   # tokens 2 and 3 are seen by no row
    p.mask[0, :4] = torch.tensor(p.words[0])
    p.K[0][:, 198:] = float("inf")
    p.V[0][:, 198:] = float("-inf")
    o, l = p.to_gpu().decode()
    p.check(o, l)


def test_bad_pages_and_lengths_are_reported():
    """A page outside the pool: its tokens are absent.  Bad lengths: the sequence
    attends nothing, and the others are computed."""
    p = Problem(4, 8, 2, 6, [700, 300, 400, 129], seed=51).to_gpu()
    good = p.decode()
    torch.cuda.synchronize()
    p.bt[0, 3] = p.pages
    p.bt[0, 10] = -7   # holds the drafted tokens' last rows
    o, l = p.decode()
    torch.cuda.synchronize()
    assert int(p.status.item()) == skv.DEV_BITS["bad_page"]
    m = p.mass(l)
    torch.cuda.synchronize()
    assert (m[0, :, 192:256] == 0).all() and (m[0, :, 640:700] == 0).all()
    assert torch.isfinite(o).all()
    z = p.scores(0, 1)
    z[..., 192:256] = -np.inf
    z[..., 640:] = -np.inf
    O, lse = oracle.softmax_rows(z, bits(p.V[0][1]))
    assert np.abs(o[0, :, 4:].cpu().numpy() - O).max() <= 2 * 6 * (p.score_error(0, 1) + 2.0 ** -17)
    assert torch.equal(o[1:], good[0][1:]) and torch.equal(l[1:], good[1][1:])
    p.status.zero_()
    p.sl[1], p.tl[2], p.tl[3] = 701, 7, -1
    o, l = p.decode()
    keep = torch.full((4, 2, 700), 5.0, device="cuda")
    p.mass(l, into=keep)
    torch.cuda.synchronize()
    assert int(p.status.item()) & skv.DEV_BITS["bad_seqlen"]
    assert (o[1:] == 0).all() and torch.isneginf(l[1:]).all() and (keep[1:] == 5).all()


def test_mass_in_place_and_decode_rows():
    """prev may be mass itself; lse of attn_decode serves for one token."""
    p = Problem(2, 8, 2, 1, [500, 130], tree="chain", seed=61).to_gpu()
    _, l = p.decode()
    m0 = torch.rand(2, 2, 500, device="cuda")
    m = m0.clone()
    for b in range(2):
        m[b, :, p.lens[b]:] = NAN
    p.mass(l, prev=m, decay=0.75, into=m)
    p.check_mass(m, l, None, m0, 0.75)


def test_streams_and_graphs():
    """Two calls at once on two streams, each with a workspace of its own; and calls
    captured into a graph, replayed on new inputs."""
    p = Problem(2, 16, 4, 9, [5000, 2500], seed=71).to_gpu()
    r = Problem(3, 16, 4, 21, [4000, 50, 333], seed=72).to_gpu()
    wp, wr = p.workspace(), r.workspace()
    for x, w in ((p, wp), (r, wr)):
        o, l = x.decode(workspace=w)
        x.mass(l)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    res = []
    for _ in range(4):
        res += [(p, p.decode(stream=s1, workspace=wp)), (r, r.decode(stream=s2, workspace=wr))]
    torch.cuda.synchronize()
    for x, (o, l) in res[-4:]:
        x.check(o, l)
    out, lse = p.buffers()
    m = torch.full((2, 4, 5000), NAN, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        skv.attn_tree_decode(p.qd, p.k, p.v, p.bt, p.sl, out, lse, workspace=wp, **p.opts)
        skv.attn_key_mass(p.qd, p.k, p.bt, p.sl, lse, m, **p.opts)
    p.q = torch.randn(p.q.shape).bfloat16()
    p.qd.copy_(p.q)
    p.lens, p.drafts = [4321, 2499], [9, 3]
    p.words[1] = [w & 0b111 for w in p.words[1][:3]]
    p.K, p.V = [k[:, :n] for k, n in zip(p.K, p.lens)], [v[:, :n] for v, n in zip(p.V, p.lens)]
    # drafted tokens are the last ones of a sequence: the words stay, the lengths move
    p.sl.copy_(torch.tensor(p.lens))
    p.tl.copy_(torch.tensor(p.drafts))
    for _ in range(3):
        g.replay()
    p.check(out, lse)
    p.check_mass(m, lse)


def test_refused_tensors():
    """What a raw pointer cannot stand for is refused before any launch."""
    p = Problem(2, 8, 2, 4, [100, 50], seed=81).to_gpu()
    o, l = p.buffers()
    good = dict(q=p.qd, k_pool=p.k, v_pool=p.v, block_table=p.bt, seq_lens=p.sl, out=o, lse=l)

    def refused(**kw):
        a = dict(good, **{k: v for k, v in kw.items() if k in good})
        opts = dict(p.opts, **{k: v for k, v in kw.items() if k not in good})
        with pytest.raises(skv.SkvError) as e:
            skv.attn_tree_decode(*a.values(), workspace=p.workspace(), **opts)
        assert e.value.status in (skv.SKV_EINVAL, skv.SKV_EUNSUPPORTED)

    refused(q=p.qd.float())
    refused(q=p.qd.transpose(1, 2).contiguous().transpose(1, 2))
    refused(out=o[..., ::2])
    refused(out=o.bfloat16())
    refused(lse=l.cpu())
    refused(seq_lens=p.sl.long())
    refused(block_table=p.bt.cpu())
    refused(tree_mask=p.mask.cuda().int())
    refused(tree_mask=p.mask.cuda()[:, :3])
    refused(tree_lens=p.tl[:1])
    refused(slopes=torch.ones(4, device="cuda"))
    refused(softcap=-1.0)
    refused(softcap=NAN)
    refused(scale=float("inf"))
    refused(window=(-1, 5))
    refused(max_seq_len=64 * p.bt.shape[1] + 1)
    with pytest.raises(skv.SkvError):
        skv.attn_key_mass(p.qd, p.k, p.bt, p.sl, l, torch.empty(2, 2, p.Lmax - 1, device="cuda"), **p.opts)
    with pytest.raises(skv.SkvError):
        skv.attn_key_mass(p.qd, p.k, p.bt, p.sl, l, torch.empty(2, 4, p.Lmax, device="cuda"), **p.opts)
    big = torch.zeros(2, 65, 8, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(skv.SkvError):
        skv.attn_tree_decode(big, p.k, p.v, p.bt, p.sl, torch.empty(2, 65, 8, 128, device="cuda"),
                             torch.empty(2, 65, 8, device="cuda"), max_seq_len=100)


@pytest.mark.parametrize("G,T,lens,window", [(8, 64, [50000], None), (4, 40, [20000, 45, 30000], (300, 29000)),
                                             (8, 40, [48000, 40], (100, 20000)), (1, 2, [1, 52000], (5000, 17000)),
                                             (4, 5, [0, 50000, 5], None)])
def test_mass_of_long_lists(G, T, lens, window):
    """A CTA's share spans more tiles than a batch of page numbers, several passes of rows,
    several sequences, and tiles between them that a window hides."""
    drafts = [min(T, n) for n in lens]
    x = Problem(len(lens), 8 * G, 8, T, lens, drafts, window=window, seed=T).to_gpu()
    o, l = x.decode()
    prev = torch.rand(len(lens), 8, x.Lmax, device="cuda")
    m = x.mass(l, prev=prev, decay=0.5)
    groups = [(b, h) for b in range(len(lens)) for h in (0, 5)]
    x.check(o, l, groups)
    x.check_mass(m, l, prev=prev, decay=0.5, groups=groups)
    assert int(x.status) == 0
