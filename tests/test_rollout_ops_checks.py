"""CPU checks of the group-rollout operators' boundary: the binding refuses
bad tensors before the library is called, the library answers bad sizes with
its codes, and a valid call reaches the library (which refuses it without an
sm_103 device)."""

import ctypes

import pytest
import torch

import invariant_logprobs_gb300 as rz
from test_binding_checks import CUDA1, S, _Stream, _unsupported, dev, workspace, zeros

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device tensors are kept off machines with a GPU")

B, T, V = 3, 4, 100
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    from invariant_logprobs_gb300 import build
    return rz.load(build.build())


@pytest.fixture(autouse=True)
def current_device_0(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def _pages(**k):
    a = dict(lens=zeros(B, dtype=I32), new_lens=zeros(B, dtype=I32),
             free_pages=zeros(9, dtype=I32), page_size=16, table=zeros(B, 5, dtype=I32), n_slots=7,
             slots_out=zeros(7, dtype=torch.int64), cu_out=zeros(B + 1, dtype=torch.int64),
             used_out=zeros(1, dtype=I32), err_flag=zeros(1, dtype=I32), stream=S)
    return rz.rz_page_tables(**{**a, **k})


def _attn(**k):
    Hq, Hkv, D, bf = 4, 2, 64, torch.bfloat16
    a = dict(q=zeros(B, Hq, D, dtype=bf), k_cache=zeros(6, 16, Hkv, D, dtype=bf),
             v_cache=zeros(6, 16, Hkv, D, dtype=bf), table=zeros(B, 2, dtype=I32),
             lens=zeros(B, dtype=I32), prefix_table=zeros(2, 3, dtype=I32),
             prefix_lens=zeros(2, dtype=I32), cu_group=zeros(3, dtype=I32),
             out=zeros(B, Hq, D, dtype=bf), lse_out=zeros(B, Hq),
             ws=workspace(rz.workspace_size(rz.RZ_OP_GROUP_DECODE_ATTN, B, D, Hq, 2)),
             err_flag=zeros(1, dtype=I32), stream=S)
    return rz.rz_group_decode_attn(**{**a, **k})


def _sample(**k):
    a = dict(logits=zeros(T, V), uniform=zeros(T), temperature=zeros(T), top_k=zeros(T, dtype=I32),
             top_p=zeros(T), min_p=zeros(T), tokens_out=zeros(T, dtype=I32), logprob_out=zeros(T),
             kept_out=zeros(T, dtype=I32), keep_out=zeros(T, 4, dtype=I32),
             err_flag=zeros(1, dtype=I32), stream=S)
    return rz.rz_filter_sample(**{**a, **k})


def _keep(**k):
    a = dict(logits=zeros(T, V), tokens=zeros(T, dtype=I32), keep=zeros(T, 4, dtype=I32),
             temperature=zeros(T), logprob_out=zeros(T), lse_out=zeros(T),
             err_flag=zeros(1, dtype=I32), stream=S)
    return rz.rz_keep_logprob(**{**a, **k})


def _bwd(**k):
    a = dict(logits=zeros(T, V), tokens=zeros(T, dtype=I32), lse=zeros(T), dlogprob=zeros(T),
             keep=zeros(T, 4, dtype=I32), temperature=zeros(T), dlogits_out=zeros(T, V),
             err_flag=zeros(1, dtype=I32), stream=S)
    return rz.rz_keep_logprob_bwd(**{**a, **k})


@pytest.mark.parametrize("call", [_pages, _attn, _sample, _keep, _bwd])
def test_valid_calls_reach_the_library(lib, call):
    _unsupported(call)
    _unsupported(call, err_flag=None)


@pytest.mark.parametrize("call,bad,error", [
    (_pages, dict(lens=zeros(B)), TypeError),
    (_pages, dict(new_lens=zeros(B + 1, dtype=I32)), ValueError),
    (_pages, dict(table=zeros(B, dtype=I32)), ValueError),
    (_pages, dict(slots_out=zeros(6, dtype=torch.int64)), ValueError),
    (_pages, dict(slots_out=zeros(7, dtype=I32)), TypeError),
    (_pages, dict(cu_out=zeros(B, dtype=torch.int64)), ValueError),
    (_pages, dict(n_slots=-1, slots_out=None), ValueError),
    (_pages, dict(stream=_Stream(1)), ValueError),
    (_attn, dict(q=zeros(B, 4, 64)), TypeError),
    (_attn, dict(v_cache=zeros(6, 16, 2, 64, dtype=torch.float16)), TypeError),
    (_attn, dict(v_cache=zeros(6, 8, 2, 64, dtype=torch.bfloat16)), ValueError),
    (_attn, dict(k_cache=zeros(6, 16, 128, dtype=torch.bfloat16)), ValueError),
    (_attn, dict(k_cache=zeros(6, 16, 64, 2, dtype=torch.bfloat16).transpose(2, 3)), ValueError),
    (_attn, dict(prefix_lens=None), TypeError),
    (_attn, dict(cu_group=zeros(2, dtype=I32)), ValueError),
    (_attn, dict(lens=zeros(B + 1, dtype=I32)), ValueError),
    (_attn, dict(out=zeros(B, 4, 64)), TypeError),
    (_attn, dict(lse_out=zeros(B, 3)), ValueError),
    (_attn, dict(ws=zeros(64)), TypeError),
    (_attn, dict(table=zeros(B, 2, dtype=I32, cls=CUDA1)), ValueError),
    (_sample, dict(logits=zeros(T, V, dtype=torch.float64)), TypeError),
    (_sample, dict(logits=zeros(V, T).t()), ValueError),
    (_sample, dict(logits=dev(torch.zeros(1, V).expand(T, V))), ValueError),
    (_sample, dict(logits=zeros(T, 0)), ValueError),
    (_sample, dict(uniform=None), TypeError),
    (_sample, dict(uniform=zeros(T + 1)), ValueError),
    (_sample, dict(top_k=zeros(T)), TypeError),
    (_sample, dict(keep_out=zeros(T, 3, dtype=I32)), ValueError),
    (_sample, dict(tokens_out=zeros(T, dtype=torch.int64)), TypeError),
    (_keep, dict(keep=zeros(T, 3, dtype=I32)), ValueError),
    (_keep, dict(tokens=zeros(T, dtype=torch.int64)), TypeError),
    (_keep, dict(temperature=zeros(1)), ValueError),
    (_keep, dict(lse_out=zeros(T - 1)), ValueError),
    (_bwd, dict(dlogits_out=zeros(T, V, dtype=torch.bfloat16)), TypeError),
    (_bwd, dict(dlogits_out=zeros(T, V + 1)), ValueError),
    (_bwd, dict(lse=zeros(T, dtype=torch.float64)), TypeError),
    (_bwd, dict(dlogprob=zeros(T, cls=CUDA1)), ValueError),
])
def test_bad_tensors_are_refused(lib, call, bad, error):
    with pytest.raises(error):
        call(**bad)


def _status(fn, *a, **k):
    with pytest.raises(rz.RzError) as e:
        fn(*a, **k)
    return e.value.status


def test_sizes_and_alignment(lib):
    assert _status(_pages, page_size=0) == rz.RZ_ERR_INVALID_ARG
    bf = torch.bfloat16
    # query heads that do not share KV heads evenly, a head size of 12 or 136
    assert _status(_attn, q=zeros(B, 5, 64, dtype=bf), out=zeros(B, 5, 64, dtype=bf),
                   lse_out=zeros(B, 5)) == rz.RZ_ERR_INVALID_ARG
    for D in (12, 136):
        assert _status(_attn, q=zeros(B, 4, D, dtype=bf), k_cache=zeros(6, 16, 2, D, dtype=bf),
                       v_cache=zeros(6, 16, 2, D, dtype=bf), out=zeros(B, 4, D, dtype=bf),
                       ws=workspace(1 << 20)) == rz.RZ_ERR_UNSUPPORTED
    # a cache whose rows are not 16-byte aligned
    odd = zeros(6, 16, 2, 68, dtype=bf)
    assert _status(_attn, k_cache=odd[..., :64]) == rz.RZ_ERR_UNSUPPORTED
    assert _status(_attn, scale=float("nan")) == rz.RZ_ERR_INVALID_ARG


def test_library_answers(lib):
    P, null = ctypes.c_void_p, None
    f = P(1 << 20)  # never dereferenced: every call fails validation or finds no device
    # page tables: no outputs, a table too large, slots without a buffer
    assert lib.rz_page_tables(f, f, 2, f, 9, 16, f, 5, f, 7, null, f, null, null) == 1
    assert lib.rz_page_tables(f, f, 1 << 20, f, 9, 16, f, 1 << 12, f, 7, f, f, null, null) == 1
    assert lib.rz_page_tables(f, f, 2, f, 9, 16, f, 5, null, 7, f, f, null, null) == 1
    assert lib.rz_page_tables(f, f, -1, f, 9, 16, f, 5, f, 7, f, f, null, null) == 1
    # sampler: dtype, row stride, V, misaligned rows; no row is nothing to do
    smp = lib.rz_filter_sample
    assert smp(f, 100, 3, 5, 100, null, null, null, null, f, f, f, null, null, null, null) == 1
    assert smp(f, 99, 0, 5, 100, null, null, null, null, f, f, f, null, null, null, null) == 1
    assert smp(f, 1 << 25, 0, 5, 1 << 25, null, null, null, null, f, f, f, null, null, null,
               null) == 1
    assert smp(f, 100, 0, 5, 100, null, null, null, null, null, f, f, null, null, null, null) == 1
    assert smp(P((1 << 20) + 2), 100, 0, 5, 100, null, null, null, null, f, f, f, null, null, null,
               null) == 2
    assert smp(null, 100, 0, 0, 100, null, null, null, null, null, null, null, null, null, null,
               null) == 0
    # kept-set logprob: no tokens; backward: in place with another row stride
    assert lib.rz_keep_logprob(f, 100, 1, 5, 100, null, null, null, f, null, null, null) == 1
    assert lib.rz_keep_logprob(null, 100, 1, 0, 100, null, null, null, null, null, null, null) == 0
    bwd = lib.rz_keep_logprob_bwd
    assert bwd(f, 100, 1, 5, 100, null, null, f, f, f, f, 104, null, null) == 1
    assert bwd(f, 100, 1, 5, 100, null, null, f, f, null, f, 100, null, null) == 1
    assert bwd(f, 100, 1, 5, 100, null, null, f, f, f, P((1 << 20) + 1), 100, null, null) == 2
    # attention: dtype fp32, a missing cache, a missing group table
    st2, st6 = (ctypes.c_int64 * 2)(256, 64), (ctypes.c_int64 * 6)(*[64] * 6)
    attn = lib.rz_group_decode_attn
    ok = [f, st2, f, f, st6, 6, 16, f, 3, f, f, 2, f, 2, f, 3, 4, 2, 64, 1, 0.1, f, f, f, 1 << 30,
          null, null]

    def call(**k):
        a = list(ok)
        for i, v in k.items():
            a[int(i[1:])] = v
        return attn(*a)

    assert call() == 2  # valid; no device
    assert call(_19=0) == 1
    assert call(_2=null) == 1
    assert call(_9=null) == 1
    assert call(_15=-1) == 1
    assert call(_6=0) == 1
    assert call(_0=P((1 << 20) + 8)) == 2
    assert call(_15=0, _0=null, _21=null) == 0
