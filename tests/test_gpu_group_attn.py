"""Decode attention of response groups against the formula in 64 bits.

Tolerance, counted in roundings: the output is rounded once to its type
(eps/2 of it) and each softmax term once as the second product's operand
(eps/2 of sum p |v|); a score carries at most delta = (D + 4) 2^-24
max_j sum_i |q_i k_ji| scale, which moves every p by a factor e^(2 delta) at
most; the fp32 sums and exponentials add 2^-18 of sum p |v|.  lse carries
delta, 2^-18 from its sum and the rounding of its own size."""

import math

import numpy as np
import pytest
import torch

from rollout_ref import attention

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _build(dtype, Hq, Hkv, D, page, sizes, pre, lens, seed=0, layout="plain", fill=None, std=1.0):
    """Caches in one of three layouts; every page no token lives in, and every
    place past a length, holds `fill`."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n_pre, n_own = [-(-a // page) for a in pre], [-(-a // page) for a in lens]
    n_pages = sum(n_pre) + sum(n_own) + 4
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).cpu().numpy()
    shape = (n_pages, page, Hkv, D)
    if layout == "plain":
        k, v = (torch.empty(shape, dtype=dtype, device=DEV) for _ in range(2))
    elif layout == "heads_first":  # [page, head, token, D] in memory
        k, v = (torch.empty(n_pages, Hkv, page, D, dtype=dtype, device=DEV).transpose(1, 2)
                for _ in range(2))
    else:  # K and V side by side, rows wider than D
        kv = torch.empty(n_pages, page, 2, Hkv, D + 8, dtype=dtype, device=DEV)
        k, v = kv[:, :, 0, :, :D], kv[:, :, 1, :, :D]
    for t in (k, v):
        t.copy_(torch.randn(shape, generator=g, device=DEV) * std)
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    at = 0

    def rows(counts, lengths):
        nonlocal at
        tab = np.full((len(counts), max(1, max(counts, default=1))), -1, np.int32)
        for i, c in enumerate(counts):
            tab[i, :c] = perm[at:at + c]
            at += c
            for t in range(lengths[i]):
                used[tab[i, t // page], t % page] = True
        return torch.tensor(tab, device=DEV)

    ptab, tab = rows(n_pre, pre), rows(n_own, lens)
    if fill is not None:
        hole = ~used.to(DEV)
        k[hole], v[hole] = fill, fill
    B = len(lens)
    q = (torch.randn(B, Hq, D, generator=g, device=DEV) * 2 * std).to(dtype)
    cu = np.concatenate([[0], np.cumsum(sizes)]) if len(sizes) else np.zeros(1)
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device=DEV)  # noqa: E731
    return dict(q=q, k_cache=k, v_cache=v, table=tab, lens=i32(lens), prefix_table=ptab,
                prefix_lens=i32(pre), cu_group=i32(cu))


def _tokens(cache, pages, n):
    page = cache.shape[1]
    rows = cache[pages[: -(-n // page)].long()].flatten(0, 1)
    return rows[:n].double()


def _check(a, out, lse, scale=None):
    q, k, v = a["q"], a["k_cache"], a["v_cache"]
    B, Hq, D = q.shape
    rep = Hq // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    eps = torch.finfo(q.dtype).eps / 2
    cu, pre, lens = a["cu_group"].tolist(), a["prefix_lens"].tolist(), a["lens"].tolist()
    worst = 0.0
    for b in range(B):
        g = next((i for i in range(len(pre)) if cu[i] <= b < cu[i + 1]), None)
        ks, vs = _tokens(k, a["table"][b], lens[b]), _tokens(v, a["table"][b], lens[b])
        if g is not None:
            ks = torch.cat([_tokens(k, a["prefix_table"][g], pre[g]), ks])
            vs = torch.cat([_tokens(v, a["prefix_table"][g], pre[g]), vs])
        for h in range(Hq):
            o, s, size, delta = attention(q[b, h].double(), ks[:, h // rep], vs[:, h // rep], scale)
            tol = eps * (o.abs() + 1.01 * size) + (2 * delta + 2.0 ** -18) * size
            off = (out[b, h].double() - o).abs()
            assert (off <= tol).all(), (b, h, float((off - tol).max()), float((off / size).max()))
            if len(ks):
                assert abs(float(lse[b, h]) - s) <= delta + 2.0 ** -18 + 2.0 ** -23 * abs(s), (b, h)
                worst = max(worst, float((off / (size * eps + 1e-30)).max()))
            else:
                assert float(lse[b, h]) == -math.inf and not out[b, h].any()
    return worst


BF, HF = torch.bfloat16, torch.float16

CASES = [
    # dtype, Hq, Hkv, D, page, group sizes, prefix lengths, own lengths
    (BF, 4, 2, 128, 16, [3], [1], [0, 1, 2]),
    (BF, 8, 1, 64, 16, [2, 0, 1], [130, 55, 0], [17, 0, 0]),
    (HF, 6, 6, 80, 24, [1, 4], [127, 129], [1, 200, 0, 33, 128]),
    (HF, 12, 2, 128, 1, [5], [40], [3, 1, 7, 64, 65]),
    (BF, 12, 2, 96, 100, [4, 3], [257, 1000], [100, 99, 101, 0, 1, 300, 5]),
    (BF, 32, 8, 128, 16, [8, 8], [512, 700], list(range(0, 160, 10))),
    (HF, 8, 2, 8, 8, [2], [64], [9, 70]),
    (BF, 64, 1, 128, 64, [3], [300], [1, 2, 3]),
    (BF, 128, 1, 64, 64, [2], [300], [70, 2]),
    (HF, 8, 8, 72, 16, [40], [385], [3] * 40),
    (BF, 8, 1, 128, 16, [37], [500], [(7 * i) % 90 for i in range(37)]),
    (BF, 2, 1, 128, 128, [1], [5000], [1]),
    (HF, 4, 4, 64, 16, [], [], [5, 0, 300]),
    (BF, 4, 1, 104, 32, [1, 1], [0, 0], [0, 0]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_the_formula(rz, case):
    dtype, Hq, Hkv, D, page, sizes, pre, lens = CASES[case]
    a = _build(dtype, Hq, Hkv, D, page, sizes, pre, lens, seed=case)
    err = rz.new_err_flag(DEV)
    out, lse = rz.rz_group_decode_attn(**a, err_flag=err)
    assert err.item() == 0
    _check(a, out, lse)


@pytest.mark.parametrize("layout", ["plain", "heads_first", "side_by_side"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 256), (96, 32), (128, 40),
                                    (128, 20), (64, 48)])
def test_strides_and_what_lies_past_the_lengths(rz, layout, fill, D, page):
    """Other cache layouts; NaN or inf in every place that holds no token."""
    a = _build(BF, 8, 2, D, page, [2, 3], [77, 300], [1, 40, 0, 129, 16], seed=5, layout=layout,
               fill=fill)
    # queries inside a fused projection's rows
    wide = torch.empty(5, 12, D, dtype=BF, device=DEV)
    wide[:, 2:10] = a["q"]
    a["q"] = wide[:, 2:10]
    out, lse = rz.rz_group_decode_attn(**a)
    _check(a, out, lse)


@pytest.mark.parametrize("std,scale", [(0.0, None), (3.0, None), (1.0, 0.0), (1.0, -0.5), (0.3, 4.0)])
def test_flat_and_peaked_rows(rz, std, scale):
    a = _build(HF, 8, 2, 128, 16, [4], [1500], [300, 0, 128, 1], seed=6, std=std)
    out, lse = rz.rz_group_decode_attn(**a, scale=scale)
    _check(a, out, lse, scale)


def test_rising_scores(rz):
    """Scores that grow along the tokens: the running maximum moves in every tile."""
    a = _build(BF, 4, 1, 64, 16, [2], [2000], [500, 700], seed=7)
    up = torch.linspace(0, 8, 2000, device=DEV)
    a["q"].fill_(1.0)
    k, page = a["k_cache"], 16
    for t in range(2000):
        k[a["prefix_table"][0, t // page].long(), t % page] = float(up[t])
    out, lse = rz.rz_group_decode_attn(**a)
    _check(a, out, lse)


def test_requests_outside_every_group(rz):
    a = _build(BF, 4, 2, 64, 16, [1, 2], [50, 60], [5, 6, 7, 8, 9], seed=8)
    out, lse = rz.rz_group_decode_attn(**a)  # requests 3 and 4 have no prompt
    _check(a, out, lse)
    b = {**a, "cu_group": a["cu_group"] + 1}  # nor has request 0
    err = rz.new_err_flag(DEV)
    out, lse = rz.rz_group_decode_attn(**b, err_flag=err)
    assert err.item() == 0
    _check(b, out, lse)


def test_no_pages_at_all(rz):
    """Tables without a column and a pool without a page."""
    a = _build(HF, 4, 2, 64, 16, [2], [50], [0, 0], seed=12)
    own = {**a, "table": a["table"][:, :0].contiguous()}
    _check(own, *rz.rz_group_decode_attn(**own))
    none = {**own, "prefix_table": a["prefix_table"][:, :0].contiguous(),
            "prefix_lens": torch.zeros_like(a["prefix_lens"]), "k_cache": a["k_cache"][:0],
            "v_cache": a["v_cache"][:0]}
    err = rz.new_err_flag(DEV)
    out, lse = rz.rz_group_decode_attn(**none, err_flag=err)
    assert not out.any() and (lse == -math.inf).all() and err.item() == 0


def test_bad_tables_are_flagged_and_skipped(rz):
    a = _build(BF, 4, 2, 64, 16, [2, 1], [40, 33], [20, 21, 22], seed=9)
    want, _ = rz.rz_group_decode_attn(**a)
    for what in ("page", "negative page", "long", "negative length", "groups"):
        b = {k: v.clone() for k, v in a.items()}
        code = rz.RZ_DEVERR_PAGES
        if what == "page":
            b["prefix_table"][0, 1] = b["k_cache"].shape[0]
        elif what == "negative page":
            b["table"][1, 0] = -3
        elif what == "long":
            b["lens"][2] = 1000
        elif what == "negative length":
            b["prefix_lens"][1] = -1
        else:
            b["cu_group"][1], b["cu_group"][2] = 9, -4
            code = rz.RZ_DEVERR_CU_SEQLENS
        err = rz.new_err_flag(DEV)
        out, lse = rz.rz_group_decode_attn(**b, err_flag=err)
        assert err.item() & code, what
        if what == "negative page":
            assert torch.equal(out[[0, 2]], want[[0, 2]])
            c = {**a, "lens": torch.tensor([20, 5, 22], dtype=torch.int32, device=DEV),
                 "table": a["table"].clone()}
            c["table"][1, 0] = a["table"][1, 1]  # tokens 16 .. 20 alone are left
            _check({**c}, out, lse)
        if what == "long":
            assert torch.equal(out[:2], want[:2])


def test_cache_offsets_past_32_bits(rz):
    """Pages more than 2^31 elements apart in one buffer."""
    n, page, Hkv, D = 40, 16, 2, 64
    stride = (1 << 31) // 16 + 64  # elements from page to page: 40 of them pass 2^32
    big = torch.empty(stride * n, dtype=BF, device=DEV)
    view = big.as_strided((n, page, Hkv, D), (stride, Hkv * D, D, 1))
    a = _build(BF, 4, Hkv, D, page, [2], [200], [100, 60], seed=10)
    perm = torch.arange(n, device=DEV, dtype=torch.int32).flip(0)
    m = a["k_cache"].shape[0]
    assert m <= n
    view[perm[:m].long()] = a["k_cache"]
    move = lambda t: torch.where(t >= 0, perm[t.clamp(min=0).long()], t)  # noqa: E731
    want, want_lse = rz.rz_group_decode_attn(**a)
    out, lse = rz.rz_group_decode_attn(**{**a, "k_cache": view, "table": move(a["table"]),
                                          "prefix_table": move(a["prefix_table"]),
                                          "v_cache": _moved(a["v_cache"], perm, n)})
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def _moved(cache, perm, n):
    out = torch.zeros((n,) + tuple(cache.shape[1:]), dtype=cache.dtype, device=DEV)
    out[perm[: cache.shape[0]].long()] = cache
    return out


def test_repeats_streams_and_graphs(rz):
    """Same bits again, on another stream and from a graph that owns its buffers."""
    # (built one token longer: the last replay's extra token has its page)
    a = _build(BF, 16, 4, 128, 16, [6, 5], [900, 3000], [50 * i + 1 for i in range(11)], seed=11)
    a["lens"].sub_(1)
    want, want_lse = rz.rz_group_decode_attn(**a)
    for _ in range(3):
        out, lse = rz.rz_group_decode_attn(**a)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = rz.rz_group_decode_attn(**a, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    ws = rz.alloc_workspace(rz.RZ_OP_GROUP_DECODE_ATTN, 11, 128, 16, 2, DEV)
    bufs = dict(out=torch.empty_like(want), lse_out=torch.empty_like(want_lse), ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rz.rz_group_decode_attn(**a, **bufs)
        rz.rz_group_decode_attn(**a, **bufs)
    a["lens"].add_(1)
    a["lens"][0] = 0
    graph.replay()
    torch.cuda.synchronize()
    _check(a, bufs["out"], bufs["lse_out"])
