"""Drafted-token attention and key mass where values leave the ordinary range: NaN and
infinite scores, sequences without drafts, score caps far above or below the scores."""
import numpy as np
import pytest
import torch

import oracle
from test_tree_gpu import Problem, bits

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# One long sequence (every group is cut into many pieces), sequences cut here and there,
# and one tile each (no group is cut); 32, 64, 128 and more rows a group.
SHAPES = [(1, 2, 4, 2, 20000), (1, 2, 8, 7, 9000), (2, 1, 8, 13, 6000), (1, 1, 8, 40, 5000), (20, 8, 4, 4, 1500),
          (40, 4, 4, 3, 100), (40, 4, 8, 12, 128)]


def check_rows(p, o, l, errors):
    """Rows with a NaN or +inf score are NaN throughout, all others as ever."""
    torch.cuda.synchronize()
    o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
    seen = [0, 0]
    for b, h in errors:
        n, hs = p.drafts[b], slice(h * p.G, (h + 1) * p.G)
        with np.errstate(invalid="ignore"):
            z = p.scores(b, h)
        bad = (np.isnan(z) | (z == INF)).any(-1)
        seen[0] += int(bad.sum())
        seen[1] += int((~bad).sum())
        got_o, got_l = o[b, :n, hs], l[b, :n, hs]
        assert np.isnan(got_o[bad]).all() and np.isnan(got_l[bad]).all(), (b, h)
        O, lse = oracle.softmax_rows(z[~bad], bits(p.V[b][h]))
        ez, vmax = errors[b, h], float(p.V[b][h].float().abs().max())
        assert (np.abs(got_o[~bad] - O) <= 2 * vmax * (ez + 2.0 ** -17)).all(), (b, h)
        assert (np.abs(got_l[~bad] - lse) <= ez + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)).all(), (b, h)
    return seen


@pytest.mark.parametrize("B,Hkv,G,T,L", SHAPES)
@pytest.mark.parametrize("what", ["nan key", "inf key", "nan drafted key", "nan query"])
@pytest.mark.parametrize("opt", [dict(), dict(slopes=True), dict(softcap=10.0), dict(window=(64, 3000))])
def test_scores_that_are_no_numbers(B, Hkv, G, T, L, what, opt):
    lens = [L - (i * 37) % (L // 3) for i in range(B)]
    p = Problem(B, Hkv * G, Hkv, T, lens, seed=L + T, **opt)
    groups = {(b, h) for b in (0, B // 2, B - 1) for h in (0, Hkv - 1)}
    errors = {x: p.score_error(*x) for x in groups}
    b = B // 2
    if what == "nan query":
        p.q[b, T - 1, Hkv * G - 1, 5] = NAN
        p.q[0, 0, 0] = NAN
    elif what == "nan drafted key":
        p.K[b][0][lens[b] - T + T // 2, 7] = NAN
    else:  # inside the window
        p.K[b][0][lens[b] - T - 20, 100] = NAN if what == "nan key" else INF
    o, l = p.to_gpu().decode()
    bad, good = check_rows(p, o, l, errors)
    assert (good > 0 or len(groups) == 1) and (bad > 0 or (what == "inf key" and "softcap" in opt))


@pytest.mark.parametrize("drafted", [0, 7, 61])  # no sequence, every seventh, every 61st
@pytest.mark.parametrize("B,Hkv,longest,window", [(1500, 2, 130, None), (1500, 2, 130, (3, 20)), (300, 8, 900, None),
                                                  (37, 4, 20000, (100, 500))])
def test_mass_of_many_sequences_without_drafts(B, Hkv, longest, window, drafted):
    """Sequences without drafts are only decayed; a CTA passes over dozens of them between
    two that have scores."""
    G, T = 2, 3
    r = np.random.default_rng(B + longest)
    lens = [int(x) for x in np.exp(r.uniform(np.log(4), np.log(longest), B))]
    has = [drafted and b % drafted == drafted // 2 for b in range(B)]
    drafts = [int(r.integers(1, T + 1)) if x else 0 for x in has]
    p = Problem(B, Hkv * G, Hkv, T, lens, drafts, seed=B, window=window).to_gpu()
    _, l = p.decode()
    prev = torch.rand(B, Hkv, p.Lmax, device="cuda")
    at = [b for b in range(B) if has[b]][:40]
    for decay, old in ((0.5, prev), (1.0, None)):
        m = p.mass(l, prev=old, decay=decay)
        for b in at:
            for h in range(Hkv):  # the oracle of the rows with drafts; the rest below
                z, n = p.scores(b, h), lens[b]
                hs = slice(h * G, (h + 1) * G)
                lse = l[b, :drafts[b], hs].double().cpu().numpy()
                want = oracle.key_mass(z, lse, np.ones(drafts[b]))
                rel = p.score_error(b, h) + 2.0 ** -21 + 2.0 ** -22 * np.abs(lse).max() + T * G * 2.0 ** -24
                was = 0.0 if old is None else decay * old[b, h, :n].double().cpu().numpy()
                assert (np.abs(m[b, h, :n].double().cpu().numpy() - was - want) <= rel * want + 2.0 ** -22 * was + 1e-30).all(), (b, h)
        inside = torch.arange(p.Lmax, device="cuda") < p.sl[:, None, None]
        rest = inside & (p.tl == 0)[:, None, None]
        want = decay * old if old is not None else torch.zeros_like(m)
        assert torch.equal(m[rest.expand_as(m)], want[rest.expand_as(m)])
        assert torch.isnan(m[~inside.expand_as(m)]).all()
        assert torch.isfinite(m[inside.expand_as(m)]).all()
    assert int(p.status.item()) == 0


def mass_rows(p, m, base, marked, value):
    """Tokens that a marked row (b, t, head) attends hold `value` (None: not a number); the
    others what they hold without it."""
    torch.cuda.synchronize()
    m, base = m.cpu().numpy(), base.cpu().numpy()
    for b in range(p.B):
        for h in range(p.Hkv):
            n = p.lens[b]
            hit = np.zeros(n, dtype=bool)
            for (x, t, head) in marked:
                if x == b and head // p.G == h:
                    hit |= np.isfinite(p.clean[b, h][t, head % p.G])
            got = m[b, h, :n]
            assert (np.isnan(got[hit]) if value is None else got[hit] == value).all(), (b, h, got[hit][:8])
            assert np.isfinite(got[~hit]).all() and (np.abs(got - base[b, h, :n])[~hit] <= 1e-5).all(), (b, h)


@pytest.mark.parametrize("G,T,lens", [(8, 1, [300, 64]), (8, 4, [200, 129]), (4, 40, [700, 41]), (1, 33, [128, 40])])
@pytest.mark.parametrize("opt", [dict(), dict(softcap=4.0, slopes=True), dict(window=(5, 40))])
def test_mass_of_rows_that_are_no_numbers(G, T, lens, opt):
    """A row that counts and whose lse or query is NaN: NaN at the tokens it attends, in
    every column that a row may take, and nowhere else; an lse of +inf gives it no weight,
    and one far below the scores an infinite one."""
    p = Problem(2, 2 * G, 2, T, lens, seed=G + T, **opt)
    p.clean = {(b, h): p.scores(b, h) for b in range(2) for h in range(2)}
    _, l = p.to_gpu().decode()
    prev = torch.rand(2, 2, p.Lmax, device="cuda")
    base = p.mass(l, prev=prev)
    rows = [(t, i) for t in sorted({0, 1, 2, T // 2, T - 1} & set(range(T))) for i in range(G)]
    for j, (t, i) in enumerate(rows):
        marked = [(j % 2, t, G + i)]
        bad = l.clone()
        bad[j % 2, t, G + i] = NAN
        mass_rows(p, p.mass(bad, prev=prev), base, marked, None)
        q = p.qd
        p.qd = q.clone()
        p.qd[j % 2, t, G + i, 3] = NAN
        mass_rows(p, p.mass(l, prev=prev), base, marked, None)
        p.qd = q
        bad[j % 2, t, G + i] = INF
        bad_mass = p.mass(bad, prev=prev)
        torch.cuda.synchronize()
        assert all(torch.isfinite(bad_mass[b, :, :lens[b]]).all() for b in range(2))
        bad[j % 2, t, G + i] = -2000.0  # e^2000 and more: above every finite number
        mass_rows(p, p.mass(bad, prev=prev), base, marked, INF)


def single_scores(cap, T, widest, seed):
    """Three sequences that are all drafts, each of which sees itself alone: lse is the score.
    One product per dot, exact in fp32.  Scores over five decades of the cap, up to `widest`
    times it."""
    g = torch.Generator().manual_seed(seed)
    p = Problem(3, 8, 1, T, [T] * 3, seed=3, scale=0.125, softcap=float(np.float32(cap)))
    p.words = [[1 << t for t in range(T)]] * 3
    p.mask = torch.tensor([[(1 << t) - (1 << 64 if t == 63 else 0) for t in range(T)]] * 3)
    u = widest * 10 ** (-5 * torch.rand(3, T, 8, generator=g, dtype=torch.float64))
    u *= 1 - 2 * (torch.rand(u.shape, generator=g) < 0.5)
    p.q = torch.zeros(3, T, 8, 128, dtype=torch.bfloat16)
    p.q[..., 17] = (u * cap * 8).bfloat16()
    for b in range(3):
        p.K[b] = torch.zeros(1, T, 128).bfloat16()
        p.K[b][..., 17] = 1
    z = p.q[..., 17].double().numpy() * 0.125
    return p.to_gpu(), p.softcap * np.tanh(z / p.softcap)


CAPS = [0.05, 5.0, 50.0, 1e3, 1e5, 1e6, 1e30, 2.3e38]


# widest: inside the fit's range, on both sides of its end, far past the cap (of 2.3e38 no bf16 is)
@pytest.mark.parametrize("T", [1, 4, 8, 16, 60])
@pytest.mark.parametrize("cap,widest", [(c, w) for c in CAPS for w in (0.45, 0.69, 1.0, 30.0) if c * w < 1e39])
def test_cap_keeps_the_scores_bits(cap, T, widest):
    """cap tanh(z / cap) to 24 half steps of fp32, relative to itself, however large the cap.
    Base 2 and back: four roundings of constants and products.  Inside: three of z / cap,
    which the quotient tanh(u) / u passes on less than once, four of its polynomial.
    Outside, from |u| = 1/2 on: 2 / (1 + e^2u) with four roundings of the argument and four
    half steps of the exponential (7 of the tanh in all), the reciprocal's two (3 of the
    tanh), and three to put it together."""
    p, want = single_scores(cap, T, widest, seed=T)
    _, l = p.decode()
    torch.cuda.synchronize()
    got = l.double().cpu().numpy()
    off = np.abs(got / want - 1) * 2.0 ** 24
    assert (off <= 24).all(), off.max()
    if cap <= 50:  # e^(z - lse) with an lse of half the score: the score shows in the mass
        for i in range(8):
            lse = torch.full((3, T, 8), -INF, device="cuda")
            lse[..., i] = torch.tensor(want[..., i] / 2, device="cuda").float()
            m = p.mass(lse)
            torch.cuda.synchronize()
            true = np.exp(want[..., i] - lse[..., i].double().cpu().numpy())
            err = np.abs(m[:, 0].double().cpu().numpy() / true - 1)
            assert (err <= 32 * 2.0 ** -24 * np.abs(want[..., i]) + 2.0 ** -21).all(), (i, err.max())


@pytest.mark.parametrize("G,T", [(4, 4), (8, 8), (8, 16)])
def test_rescaled_walks_repeat_bit_for_bit(G, T):
    """Maxima that grow in every tile of a walk of more than 32: sums that are rescaled, and
    moved to the record, between the products that add to them.  Right, and the same over
    and over."""
    L, n = 26500, 24
    p = Problem(1, G, 1, T, [L], seed=5 + G + T)
    u = torch.nn.functional.normalize(torch.randn(128, generator=torch.Generator().manual_seed(8)), dim=0)
    p.q = (p.q.float() * 0.3 + 20 * u).bfloat16()
    p.K[0] = (p.K[0].float() * 0.3 + torch.linspace(30, -30, L)[None, :, None] * u).bfloat16()
    p.to_gpu()
    p.B, p.lens, p.drafts, p.words, p.K, p.V = n, [L] * n, [T] * n, p.words * n, p.K * n, p.V * n
    p.q = p.q.expand(n, -1, -1, -1).contiguous()
    p.qd, p.bt = p.q.cuda(), p.bt.expand(n, -1).contiguous()
    p.sl, p.tl = p.sl.expand(n).contiguous(), p.tl.expand(n).contiguous()
    p.opts.update(tree_lens=p.tl, tree_mask=p.mask.expand(n, -1).contiguous().cuda())
    o, l = p.decode()
    p.check(o, l, [(0, 0), (13, 0)])
    for _ in range(30):
        o2, l2 = p.decode()
        assert torch.equal(o, o2) and torch.equal(l, l2)
