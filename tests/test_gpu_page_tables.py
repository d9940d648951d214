"""Block tables and slot maps against a plain loop, whole numbers exactly."""

import numpy as np
import pytest
import torch

from rollout_ref import page_tables

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(B, page, len_hi, new_hi, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, len_hi + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    width = max([1] + [-(-int(a + b) // page) for a, b in zip(lens, new)])
    table = np.full((B, width), -7, np.int32)
    ids = rng.permutation(1 << 21)[: B * width + 8].astype(np.int32)
    at = 0
    for i, n in enumerate(lens):
        c = -(-int(n) // page)
        table[i, :c] = ids[at:at + c]
        at += c
    return lens.astype(np.int32), new.astype(np.int32), ids[at:], table


def _run(rz, lens, new, free, page, table, n_slots, err=None):
    t = torch.tensor(table, device=DEV)
    c = lambda x: torch.tensor(np.asarray(x, np.int32), device=DEV)  # noqa: E731
    slots, cu, used = rz.rz_page_tables(c(lens), c(new), c(free), page, t, n_slots, err_flag=err)
    return t.cpu().numpy(), slots.cpu().numpy(), cu.cpu().numpy(), int(used.item())


@pytest.mark.parametrize("B,page,len_hi,new_hi", [
    (1, 16, 0, 1), (1, 1, 5, 7), (7, 16, 100, 1), (64, 16, 5000, 1), (33, 24, 300, 40),
    (1024, 16, 2000, 1), (1025, 16, 2000, 1), (1024, 16, 100, 32), (900, 100, 0, 700),
    (5000, 8, 40, 3), (3, 64, 0, 60000), (12000, 16, 64, 2)])
@pytest.mark.parametrize("extra", [0, 37])
def test_matches_the_loop(rz, B, page, len_hi, new_hi, extra):
    lens, new, free, table = _case(B, page, len_hi, new_hi, seed=B + page)
    n_slots = int(new.sum()) + extra
    want = page_tables(lens, new, free, page, table, n_slots)
    err = rz.new_err_flag(DEV)
    for _ in range(2):  # the second call finds its own pages and takes the same ones
        got = _run(rz, lens, new, free, page, table, n_slots, err)
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
        table = got[0]
    assert err.item() == 0


def test_no_requests(rz):
    got = _run(rz, [], [], [], 16, np.zeros((0, 3), np.int32), 5)
    assert got[1].tolist() == [-1] * 5 and got[2].tolist() == [0] and got[3] == 0


@pytest.mark.parametrize("big", [False, True])
def test_trouble_is_flagged_and_stays_inside(rz, big):
    """Too few free pages, a row too narrow, a negative length, too few slots."""
    page, B = 4, 3000 if big else 3
    lens = np.zeros(B, np.int32)
    new = np.full(B, 6, np.int32)
    table = np.full((B, 2), -9, np.int32)
    free = np.arange(100, 100 + 2 * B - 1, dtype=np.int32)  # one page short
    for what in ("free", "row", "negative", "slots", "held"):
        ln, nw, fr, n_slots = lens.copy(), new.copy(), free.copy(), 6 * B
        if what != "free":
            fr = np.arange(100, 100 + 2 * B + 9, dtype=np.int32)
        if what == "row":
            nw[1] = 11  # three pages in a row of two
            n_slots += 5
        if what == "negative":
            ln[1], nw[2] = -5, -1
            n_slots -= 6
        if what == "slots":
            n_slots -= 7
        if what == "held":
            ln[0] = 2  # a token in a page that the row does not have
        err = rz.new_err_flag(DEV)
        got = _run(rz, ln, nw, fr, page, table, n_slots, err)
        want = page_tables(np.maximum(ln, 0), np.maximum(nw, 0), fr, page, table, n_slots)
        for g, w in zip(got, want):
            assert np.array_equal(g, w), what
        assert err.item() == rz.RZ_DEVERR_PAGES, what


def test_slots_past_32_bits(rz):
    """Page id times page size leaves 32 bits."""
    got = _run(rz, [5], [3], [2_000_000_000], 1000, np.full((1, 1), 2_100_000_000, np.int32), 3)
    assert got[1].tolist() == [2_100_000_000_005, 2_100_000_000_006, 2_100_000_000_007]
