"""Filtered sampling and the kept-set logprob against plain forms in 64 bits.

Tokens, kept counts and kept sets must be equal.  Tolerance of a log
probability, counted in fp32 roundings (2^-24 each): (z - max)/tau is rounded
twice; the sum of exponentials carries at most 64 + 13 + 32 additions and an
exponent's own error of 4 roundings; its logarithm 4 more: below 1e-5 of
1 + |log p|.  A gradient entry carries the rounding to its type (eps/2) and
p's: the exponent z/tau - lse of size x is off by 2^-22 (1 + |z/tau| + |lse|)
at most, plus lse's own error."""

import numpy as np
import pytest
import torch

from rollout_ref import filter_row, keep_logprob, pack

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _t(x, dtype=torch.float32):
    return torch.tensor(np.asarray(x), dtype=dtype, device=DEV)


def _logits(kind, T, V, g):
    z = torch.randn(T, V, generator=g, device=DEV)
    if kind == "peaked":
        z = z * 2
        z[:, V // 3] += 9
    elif kind == "flat":
        z = z * 0.05
    elif kind == "wide":
        z = z * 40
    elif kind == "constant":
        z = torch.full_like(z, -3.25)
    elif kind == "ties":
        z = (z * 1.5).round() / 2
        z[z == 0] *= -1  # zeros of both signs
    elif kind == "banned":
        z[:, : V - max(1, V // 7)] = -torch.inf
    elif kind == "huge":
        z = z * 1e4
    return z


FILTERS = [(0, 1.0, 0.0), (1, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.9, 0.0), (0, 0.05, 0.0),
           (0, 0.9999, 0.0), (0, 1.0, 0.1), (50, 0.8, 0.0), (50, 0.8, 0.02), (0, 0.0, 0.0),
           (3, 1.0, 1.0), (10**9, 1.0, -1.0), (-4, 2.0, 0.0)]
TEMPS = [1.0, 0.7, 1.7, 0.0]


def _run(rz, z, temp, k, p, mp, u, **kw):
    return rz.rz_filter_sample(z, u, temperature=temp, top_k=k, top_p=p, min_p=mp, want_keep=True,
                               **kw)


@pytest.mark.parametrize("kind", ["normal", "peaked", "flat", "wide", "constant", "ties", "banned",
                                  "huge"])
@pytest.mark.parametrize("dtype,V", [("f32", 1000), ("bf16", 2049), ("f16", 333), ("f32", 1),
                                     ("bf16", 31), ("f32", 40003), ("f16", 20000)])
def test_matches_exact_arithmetic(rz, kind, dtype, V):
    g = torch.Generator(device=DEV)
    g.manual_seed(V)
    T = len(FILTERS) * len(TEMPS)
    z = _logits(kind, T, V, g).to(DT[dtype])
    rows = [(t, *f) for f in FILTERS for t in TEMPS]
    u = torch.rand(T, generator=g, device=DEV)
    u[:2] = torch.tensor([0.0, 1 - 2.0 ** -24])
    temp, k, p, mp = (_t([r[i] for r in rows], d) for i, d in
                      enumerate([torch.float32, torch.int32, torch.float32, torch.float32]))
    err = rz.new_err_flag(DEV)
    tok, lp, n, keep = _run(rz, z, temp, k, p, mp, u, err_flag=err)
    assert err.item() == 0
    zd, keeps = z.double().cpu().numpy(), []
    got = [x.cpu().numpy() for x in (tok, lp, n, keep)]
    f = lambda x: float(np.float32(x))  # noqa: E731
    for r, (t, kk, pp, mm) in enumerate(rows):
        a, want, kept = filter_row(zd[r], f(t), kk, f(pp), f(mm), float(u[r]))
        assert (got[0][r], got[2][r]) == (a, len(kept)), (r, rows[r])
        assert abs(got[1][r] - want) <= 1e-5 * (1 + abs(want)), (r, rows[r], got[1][r], want)
        keeps.append(kept)
    assert np.array_equal(got[3], pack(keeps, V))
    # the learner's log probability of these tokens is the same float
    temp1 = torch.where(temp == 0, 1.0, temp)
    for tt in (temp, temp1):
        lp2, _ = rz.rz_keep_logprob(z, tok, keep=keep, temperature=tt)
        assert torch.equal(lp, lp2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_full_vocabulary(rz, dtype):
    V, T = 151936, 24
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    z = torch.randn(T, V, generator=g, device=DEV) * torch.linspace(0.3, 4, T, device=DEV)[:, None]
    z[::3, 5000:5020] += 12
    z = z.to(DT[dtype])
    p = _t([[0.95, 1.0, 0.5][r % 3] for r in range(T)])
    k = _t([[0, 0, 1000, 30][r % 4] for r in range(T)], torch.int32)
    mp = _t([[0.0, 0.0, 0.0, 0.0, 0.01][r % 5] for r in range(T)])
    temp = _t([[1.0, 0.8][r % 2] for r in range(T)])
    u = torch.rand(T, generator=g, device=DEV)
    tok, lp, n, keep = _run(rz, z, temp, k, p, mp, u)
    zd = z.double().cpu().numpy()
    keeps = []
    for r in range(T):
        a, want, kept = filter_row(zd[r], float(temp[r]), int(k[r]), float(p[r]), float(mp[r]),
                                   float(u[r]))
        assert (int(tok[r]), int(n[r])) == (a, len(kept)), r
        assert abs(float(lp[r]) - want) <= 1e-5 * (1 + abs(want))
        keeps.append(kept)
    assert np.array_equal(keep.cpu().numpy(), pack(keeps, V))
    assert torch.equal(rz.rz_keep_logprob(z, tok, keep=keep, temperature=temp)[0], lp)
    # a row's result is its own: alone, and in a batch that fills the GPU
    one = _run(rz, z[5:6], temp[5:6], k[5:6], p[5:6], mp[5:6], u[5:6])
    many = _run(rz, z.repeat(40, 1), temp.repeat(40), k.repeat(40), p.repeat(40), mp.repeat(40),
                u.repeat(40))
    for x, a, b in zip((tok, lp, n, keep), one, many):
        assert torch.equal(x[5:6], a)
        assert torch.equal(x.repeat(40, *[1] * (x.dim() - 1)), b)


@pytest.mark.parametrize("V,dtype", [(3_000_001, "f32"), (1_000_000, "bf16"), (1 << 24, "f16")])
def test_wide_vocabulary(rz, V, dtype):
    """Rows past what a cluster's shared memory holds, up to the largest."""
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    z = torch.randn(2, V, generator=g, device=DEV).to(DT[dtype])
    u = torch.rand(2, generator=g, device=DEV)
    p = _t([0.7, 1.0])
    tok, lp, n, keep = rz.rz_filter_sample(z, u, top_p=p, want_keep=True)
    for r in range(2):
        a, want, kept = filter_row(z[r].double().cpu().numpy(), 1.0, 0, float(p[r]), 0.0,
                                   float(u[r]))
        assert (int(tok[r]), int(n[r])) == (a, len(kept))
        assert abs(float(lp[r]) - want) <= 1e-5 * (1 + abs(want))
    lp2, lse = rz.rz_keep_logprob(z, tok, keep=keep)
    assert torch.equal(lp2, lp)
    d = rz.rz_keep_logprob_bwd(z, tok, lse, torch.ones(2, device=DEV), keep=keep)
    p_tok = torch.exp(lp.double())
    got = d.double().gather(1, tok.long()[:, None])[:, 0]
    eps = torch.finfo(d.dtype).eps
    assert ((got - (1 - p_tok)).abs() <= eps).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [8193, 9217, 16385, 40003, 151936, 700001])
def test_few_rows_as_in_a_large_batch(rz, V, dtype):
    """One to four rows, which more CTAs share, give what they give among sixty-four."""
    g = torch.Generator(device=DEV)
    g.manual_seed(14)
    T = 64
    z = (2 * torch.randn(T, V, generator=g, device=DEV)).to(DT[dtype])
    f = [FILTERS[r % len(FILTERS)] for r in range(T)]
    temp = _t([[1.0, 0.7, 0.0][r % 3] for r in range(T)])
    k, p, mp = (_t([x[i] for x in f], d) for i, d in
                enumerate([torch.int32, torch.float32, torch.float32]))
    u = torch.rand(T, generator=g, device=DEV)
    all_ = _run(rz, z, temp, k, p, mp, u)
    for lo, n in [(0, 1), (1, 1), (2, 2), (4, 3), (7, 4), (11, 4), (15, 6)]:
        at = slice(lo, lo + n)
        few = _run(rz, z[at], temp[at], k[at], p[at], mp[at], u[at])
        for x, y in zip(few, all_):
            assert torch.equal(x, y[at])


@pytest.mark.parametrize("dtype,V,T", [("f32", 151936, 310), ("bf16", 1 << 21, 310),
                                       ("f16", 32003, 3000), ("f32", 4097, 150)])
def test_many_rows_as_alone(rz, dtype, V, T):
    """Rows of a batch of several waves give what they give alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(15)
    z = (2 * torch.randn(T, V, generator=g, device=DEV, dtype=torch.float32).to(DT[dtype]))
    f = [FILTERS[r % len(FILTERS)] for r in range(T)]
    temp = _t([[1.0, 0.7, 0.0][r % 3] for r in range(T)])
    k, p, mp = (_t([x[i] for x in f], d) for i, d in
                enumerate([torch.int32, torch.float32, torch.float32]))
    u = torch.rand(T, generator=g, device=DEV)
    all_ = _run(rz, z, temp, k, p, mp, u)
    for lo, n in [(0, 3), (57, 16), (T - 40, 40)]:
        at = slice(lo, lo + n)
        few = _run(rz, z[at], temp[at], k[at], p[at], mp[at], u[at])
        for x, y in zip(few, all_):
            assert torch.equal(x, y[at])


def test_no_filters_at_all_and_row_strides(rz):
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    for dtype in DT.values():
        wide = torch.randn(9, 1013, generator=g, device=DEV).to(dtype)
        u = torch.rand(9, generator=g, device=DEV)
        for z in (wide[:, :1000], wide[:, 3:1003], wide[::2, 1:]):
            tok, lp, n, keep = rz.rz_filter_sample(z, u[: len(z)])
            assert keep is None and (n == z.shape[1]).all()
            for r in range(len(z)):
                a, want, _ = filter_row(z[r].double().cpu().numpy(), 1.0, 0, 1.0, 0.0, float(u[r]))
                assert int(tok[r]) == a and abs(float(lp[r]) - want) <= 1e-5 * (1 + abs(want))
            assert torch.equal(rz.rz_keep_logprob(z, tok)[0], lp)


def test_rows_and_parameters_that_cannot_be(rz):
    V, T = 500, 12
    z = torch.zeros(T, V, device=DEV)
    z[1, 17] = float("nan")
    z[2, 499] = float("inf")
    z[3] = -torch.inf
    temp = torch.ones(T, device=DEV)
    p, mp, u = torch.ones(T, device=DEV), torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)
    temp[4], temp[5], temp[6] = -1.0, float("nan"), 1e30
    p[7] = float("nan")
    mp[8] = 1.5
    u[9], u[10] = 1.0, float("nan")
    err = rz.new_err_flag(DEV)
    tok, lp, n, keep = rz.rz_filter_sample(z, u, temperature=temp, top_p=p, min_p=mp,
                                           want_keep=True, err_flag=err)
    assert err.item() == rz.RZ_DEVERR_LOGITS | rz.RZ_DEVERR_PARAM
    good = [0, 11]
    assert tok.tolist() == [0 if r in good else -1 for r in range(T)]
    assert n.tolist() == [V if r in good else 0 for r in range(T)]
    assert [bool(x) for x in lp.isnan().tolist()] == [r not in good for r in range(T)]
    assert not keep[1:11].any()
    err.zero_()
    rz.rz_filter_sample(z[:1], u[:1], err_flag=err)
    assert err.item() == 0


# ------------------------------------------------------------------ kept-set logprob
def _keep_case(T, V, dtype, seed, share, std=2.0, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = (torch.randn(T, V + pad, generator=g, device=DEV) * std).to(DT[dtype])[:, :V]
    kept = torch.rand(T, V, generator=g, device=DEV) < share
    tok = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    kept[torch.arange(T), tok.long()] = True
    temp = 0.5 + torch.rand(T, generator=g, device=DEV)
    coef = torch.randn(T, generator=g, device=DEV)
    words = _t(pack([np.flatnonzero(x) for x in kept.cpu().numpy()], V), torch.int32)
    return z, kept, words, tok, temp, coef


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V,share,pad", [(1, 1, 1.0, 0), (5, 31, 0.5, 0), (3, 2048, 0.01, 8),
                                           (7, 2049, 0.3, 3), (2, 32003, 0.001, 5),
                                           (400, 5000, 0.02, 0), (3, 151936, 0.5, 0)])
@pytest.mark.parametrize("masked", [True, False])
def test_keep_logprob_and_gradient(rz, dtype, T, V, share, pad, masked):
    z, kept, words, tok, temp, coef = _keep_case(T, V, dtype, T + V, share, pad=pad)
    if masked:
        z[~kept] = float("nan")  # what is not kept is not looked at
    else:
        kept, words = torch.ones_like(kept), None
    lp, lse = rz.rz_keep_logprob(z, tok, keep=words, temperature=temp)
    d = rz.rz_keep_logprob_bwd(z, tok, lse, coef, keep=words, temperature=temp)
    eps = torch.finfo(DT[dtype]).eps / 2
    for r in range(0, T, max(1, T // 20)):
        zr = torch.where(kept[r], z[r].double(), 0.0)
        want, wlse, wd = keep_logprob(zr, float(temp[r]), int(tok[r]), kept[r], float(coef[r]))
        tol = 1e-5 * (1 + abs(want) + abs(wlse))
        assert abs(float(lp[r]) - want) <= tol and abs(float(lse[r]) - wlse) <= tol
        x = zr / float(temp[r])
        p = torch.where(kept[r], torch.exp(x - wlse), 0.0)
        slack = abs(float(coef[r])) / float(temp[r]) * p * (2.0 ** -21 * (1 + x.abs() + abs(wlse)) + tol)
        tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -126  # half the smallest step
        assert ((d[r].double() - wd).abs() <= (eps + 2.0 ** -22) * wd.abs() + slack + tiny).all()
    assert not d[~kept].any()
    # in place, and into rows of another stride
    ldd = torch.full((T, V + 5), 7.0, dtype=DT[dtype], device=DEV)
    rz.rz_keep_logprob_bwd(z, tok, lse, coef, keep=words, temperature=temp, dlogits_out=ldd[:, :V])
    assert torch.equal(ldd[:, :V], d) and (ldd[:, V:] == 7).all()
    same = rz.rz_keep_logprob_bwd(z, tok, lse, coef, keep=words, temperature=temp, dlogits_out=z)
    assert same is z and torch.equal(z, d)


def test_gradient_against_differences(rz):
    """Central differences of the kernel's own forward pass: at a step of 0.05
    the third-order term is below 0.05^2 / 6 of the entry's scale, and the
    forward pass's error of 2e-5 enters as 2e-5 / 0.1."""
    z, kept, words, tok, temp, _ = _keep_case(4, 67, "f32", 9, 0.4)
    temp.fill_(1.0)
    lp, lse = rz.rz_keep_logprob(z, tok, keep=words, temperature=temp)
    d = rz.rz_keep_logprob_bwd(z, tok, lse, torch.ones(4, device=DEV), keep=words, temperature=temp)
    h = 0.05
    for v in range(67):
        up, dn = z.clone(), z.clone()
        up[:, v] += h
        dn[:, v] -= h
        diff = (rz.rz_keep_logprob(up, tok, keep=words, temperature=temp)[0] -
                rz.rz_keep_logprob(dn, tok, keep=words, temperature=temp)[0]) / (2 * h)
        assert ((diff - d[:, v]).abs() <= h * h / 6 + 2e-4).all()


def test_rows_with_nothing_to_say(rz):
    V, T = 3000, 7
    g = torch.Generator(device=DEV)
    g.manual_seed(10)
    z = torch.randn(T, V, generator=g, device=DEV)
    kept = torch.zeros(T, V, dtype=torch.bool)
    kept[1:, :50] = True
    tok = torch.zeros(T, dtype=torch.int32, device=DEV)
    tok[2], tok[3], tok[4] = 60, V, -1  # not kept, past the vocabulary, negative
    z[5, :50] = -torch.inf
    temp = torch.ones(T, device=DEV)
    temp[6] = -2.0
    words = _t(pack([np.flatnonzero(x) for x in kept.numpy()], V), torch.int32)
    err = rz.new_err_flag(DEV)
    lp, lse = rz.rz_keep_logprob(z, tok, keep=words, temperature=temp, err_flag=err)
    assert err.item() == rz.RZ_DEVERR_TOKEN_RANGE | rz.RZ_DEVERR_PARAM
    inf = float("inf")
    assert lp[0] == -inf and lse[0] == -inf  # nothing kept
    assert lp[2] == -inf and torch.isfinite(lse[2])
    assert lp[3].isnan() and lp[4].isnan() and torch.isfinite(lse[3:5]).all()
    assert lp[5] == -inf and lse[5] == -inf
    assert lp[6].isnan() and lse[6].isnan()
    coef = torch.ones(T, device=DEV)
    d = rz.rz_keep_logprob_bwd(z, tok, lse, coef, keep=words, temperature=temp)
    assert d[1].any() and not d[[0, 2, 3, 4, 5, 6]].any()
    coef.zero_()
    z[1, :50] = float("nan")
    assert not rz.rz_keep_logprob_bwd(z, tok, lse, coef, keep=words, temperature=temp).any()


def test_a_likely_token_keeps_its_small_gradient(rz):
    """log p near 0: the token's entry g expm1(log p) keeps its relative size."""
    V = 1000
    z = torch.zeros(1, V, device=DEV)
    z[0, 7] = 22.0
    tok = torch.tensor([7], dtype=torch.int32, device=DEV)
    lp, lse = rz.rz_keep_logprob(z, tok)
    want = -np.log1p(999 * np.exp(-22.0))
    assert abs(float(lp) - want) <= 2.0 ** -20 * abs(want)
    d = rz.rz_keep_logprob_bwd(z, tok, lse, torch.ones(1, device=DEV))
    # lse itself is rounded at 22: half a step there is 2^-20
    assert abs(float(d[0, 7]) - (-np.expm1(want))) <= 2.0 ** -20


def test_sample_and_score_in_a_graph(rz):
    """Sampling, its score and the gradient captured once and replayed on new logits."""
    T, V = 40, 5003
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    z = torch.randn(T, V, generator=g, device=DEV)
    u = torch.rand(T, generator=g, device=DEV)
    p = torch.full((T,), 0.9, device=DEV)
    coef = torch.randn(T, generator=g, device=DEV)
    bufs = dict(tokens_out=torch.empty(T, dtype=torch.int32, device=DEV),
                logprob_out=torch.empty(T, device=DEV),
                kept_out=torch.empty(T, dtype=torch.int32, device=DEV),
                keep_out=torch.empty(T, (V + 31) // 32, dtype=torch.int32, device=DEV))
    lp, lse, d = torch.empty(T, device=DEV), torch.empty(T, device=DEV), torch.empty_like(z)

    def work():
        rz.rz_filter_sample(z, u, top_p=p, **bufs)
        rz.rz_keep_logprob(z, bufs["tokens_out"], keep=bufs["keep_out"], logprob_out=lp,
                           lse_out=lse)
        rz.rz_keep_logprob_bwd(z, bufs["tokens_out"], lse, coef, keep=bufs["keep_out"],
                               dlogits_out=d)

    work()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    z.copy_(torch.randn(T, V, generator=g, device=DEV))
    u.copy_(torch.rand(T, generator=g, device=DEV))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (*bufs.values(), lp, lse, d)]
    work()
    for a, b in zip(got, (*bufs.values(), lp, lse, d)):
        assert torch.equal(a, b)
    assert torch.equal(bufs["logprob_out"], lp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tok, lp2, _, _ = rz.rz_filter_sample(z, u, top_p=p, stream=s)
    s.synchronize()
    assert torch.equal(tok, bufs["tokens_out"]) and torch.equal(lp2, lp)
