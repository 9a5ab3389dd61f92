"""Full attention where masks, groups and values that are not finite meet:
corners beside those of test_gpu_attn.py, with its reference and tolerances.
"""
import pytest
import torch

from linear_attention_serving_delta_gb300 import kda
from test_gpu_attn import Pool, check, cu_of, gen, rand, reference

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ one token to a row tile
@pytest.mark.parametrize("D,dtype", [(256, "bf16"), (128, "bf16"), (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("G", [64, 65, 100, 128])
@pytest.mark.parametrize("at", [5, 100])
def test_later_tokens_never_reach_wide_groups(D, dtype, G, at):
    """Groups of more than 64 query heads: a row tile holds one token, its last key tile those behind it too."""
    g = gen(G + at)
    T = 150
    q, k, v = rand(g, T, 2 * G, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
    clean = kda.attn_prefill(q, k, v, cu_of([T]).cuda())
    v[at] = float("inf")
    v[at + 1:] = float("nan")
    o = kda.attn_prefill(q, k, v, cu_of([T]).cuda())
    check(o[:at], *reference(q[:at], k[:at], v[:at], 0, D ** -0.5, dtype))
    assert torch.equal(o[:at], clean[:at])
    assert torch.isposinf(o[at].float()).all() and torch.isnan(o[at + 1:].float()).all()


@pytest.mark.parametrize("D,dtype", [(256, "bf16"), (128, "bf16"), (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("G", [65, 128])
def test_later_tokens_of_a_chunk_never_reach_wide_groups(D, dtype, G):
    ctx, new, at = 70, 60, 20
    p = Pool([ctx], [new], 1, D, 16, dtype, 7)
    q = rand(gen(G), new, G, D, dtype=dtype)
    cu = cu_of([new]).cuda()
    clean = kda.attn_paged(q, p.k, p.v, p.table, p.lens, cu)
    x = torch.arange(ctx + at, ctx + new)
    slot = (p.table[0].cpu().long()[x // 16] * 16 + x % 16).cuda()
    p.v.view(-1, 1, D)[slot] = float("nan")
    o = kda.attn_paged(q, p.k, p.v, p.table, p.lens, cu)
    check(o[:at], *reference(q[:at], p.K[0][:ctx + at], p.V[0][:ctx + at], ctx, D ** -0.5, dtype))
    assert torch.equal(o[:at], clean[:at]) and torch.isnan(o[at:].float()).all()
