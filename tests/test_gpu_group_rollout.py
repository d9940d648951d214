"""The group-rollout example end to end: the operators as a program uses them."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "group_rollout", os.path.join(ROOT, "examples", "group_rollout.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("prompts,group,steps,V", [(4, 8, 20, 5003), (1, 1, 3, 33), (3, 5, 40, 1024)])
def test_rollout_and_learner_agree_bit_for_bit(rz, prompts, group, steps, V):
    out = _example().run(prompts, group, steps, V)
    assert len(out["logpi"]) == prompts * group * steps
    assert torch.isfinite(out["logpi"]).all() and (out["logpi"] <= 0).all()
    # at equal weights: the same floats, so every weight is 1 and D3 is 0
    assert torch.equal(out["logpi"], out["logmu"])
    assert float(out["d3"]) == 0.0
    assert torch.isfinite(out["dH"]).all() and torch.isfinite(out["dW"]).all()
    # a probability's shift moves no logit: columns of dz sum to 0 in every row,
    # so the LM head's gradient sums to 0 over the vocabulary (fp32 sums of
    # V terms a row and as many rows as tokens)
    size = out["dW"].abs().sum(0)
    assert (out["dW"].sum(0).abs() <= 1e-4 * size + 1e-7).all()


def test_attention_matches_a_prefix_in_own_pages(rz):
    """The prompt's tokens as a shared prefix, or copied into every response's
    own pages: the same attention, up to the order of its sums (two roundings
    of a term to bf16, and the output's)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    P, G, page, Hkv, D = 2, 3, 16, 2, 64
    pre, own = 4 * page, 2 * page
    n = P * 4 + P * G * 2
    k, v = (torch.randn(n, page, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    q = torch.randn(P * G, 4, D, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    prefix = torch.arange(P * 4, device="cuda").view(P, 4)
    table = P * 4 + torch.arange(P * G * 2, device="cuda").view(P * G, 2)
    out, lse = rz.rz_group_decode_attn(
        q, k, v, i32(table), i32([own] * P * G), prefix_table=i32(prefix),
        prefix_lens=i32([pre] * P), cu_group=i32([0, G, 2 * G]))
    both = torch.cat([prefix.repeat_interleave(G, 0), table], 1)
    out2, lse2 = rz.rz_group_decode_attn(q, k, v, i32(both), i32([pre + own] * P * G))
    assert (lse - lse2).abs().max() <= 1e-5
    assert (out.float() - out2.float()).abs().max() <= 3 * 2.0 ** -9 * v.float().abs().max()
