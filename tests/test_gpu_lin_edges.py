"""Linear attention with a decay for each head where values that are not finite meet
the borders of chunks, segments and chains, and where products are far from 1: corners
beside those of test_gpu_lin.py, with its inputs and bounds.
"""
import math

import pytest
import torch

from linear_attention_serving_delta_gb300 import kda
from test_gpu_lin import check_prefill, inputs, offsets

pytestmark = pytest.mark.gpu

# every shape of the tensor-core prompts
SHAPES = [(64, 64), (128, 128), (256, 128), (64, 128), (128, 64)]


def poison(d, lens, at):
    """Infinities and NaN into v at (sequence, token, head, channel); which elements of o and of the states
    may keep their bits."""
    T, H, dv = d["v"].shape
    o, s = torch.ones(T, H, dv, dtype=torch.bool), torch.ones(len(lens), H, d["k"].shape[2], dv, dtype=torch.bool)
    cu = offsets(lens).tolist()
    v = d["v"].cpu()
    for i, (seq, t, h, c) in enumerate(at):
        v[cu[seq] + t, h, c] = (float("inf"), float("nan"), float("-inf"))[i % 3]
        o[cu[seq] + t:cu[seq + 1], h, c] = False
        s[seq, h, :, c] = False
    return dict(d, v=v.cuda()), o.cuda(), s.cuda()


def check_poisoned(got, clean, same_o, same_s):
    assert torch.equal(got[0][same_o], clean[0][same_o])
    assert not torch.isfinite(got[0][~same_o].float()).any()
    assert torch.equal(got[1][same_s], clean[1][same_s])
    assert not torch.isfinite(got[1][~same_s]).any()


def prompts(d, lens):
    call = kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], initial_state=d["state"]).run()
    assert call.device_status() == 0
    return call.o, call.final_state


# ------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("at", [0, 60, 127])
def test_first_chunk_behind_a_state(dk, dv, at):
    """Nothing of a chain precedes its first chunk, so the state that it starts from stays as it is."""
    lens, H = [200, 150], 2
    d = inputs(dk + dv + at, 350, H, H, dk, dv, "bf16", "g", n=2)
    clean = prompts(d, lens)
    bad, same_o, same_s = poison(d, lens, [(0, at, 0, 5), (1, at, 1, dv - 1), (1, at, 1, 8)])
    check_poisoned(prompts(bad, lens), clean, same_o, same_s)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 64)])
def test_first_chunk_of_a_later_segment(dk, dv):
    """A long prompt is cut into segments: a value in each of its chunks in turn."""
    lens, H = [2600], 2
    d = inputs(dk + dv, 2600, H, H, dk, dv, "bf16", "g")
    clean = prompts(d, lens)
    for t in range(5, 2600, 128):
        bad, same_o, same_s = poison(d, lens, [(0, t, 1, 9)])
        check_poisoned(prompts(bad, lens), clean, same_o, same_s)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("most", [120, 390])
def test_chains_of_a_cta_one_after_the_other(dk, dv, most):
    """Many more chains than CTAs, and in each channels whose values are not finite in its first and its last
    chunk: what one chain notes must not hide what the chain before it is still asked for."""
    n, H = 240, 4
    g = torch.Generator().manual_seed(dk + dv + most)
    lens = torch.randint(1, most + 1, (n,), generator=g).tolist()
    d = inputs(dk + 2 * dv + most, sum(lens), H, 2, dk, dv, "bf16", "g", n=n)
    clean = prompts(d, lens)
    at = []
    for s in range(n):
        for h in range(H):
            if (s + h) % 5 == 4:  # (and some chains without any)
                continue
            at += [(s, lens[s] - 1, h, dv - 1), (s, 0, h, dv - 1), (s, lens[s] - 1, h, dv - 2),
                   (s, max(0, lens[s] - 9), h, dv // 2), (s, int(lens[s] * 0.7), h, 0)]
    bad, same_o, same_s = poison(d, lens, at)
    call = kda.LinPrefill(bad["q"], bad["k"], bad["v"], offsets(lens), g=bad["g"], initial_state=bad["state"])
    for _ in range(5):
        call.run()
        check_poisoned((call.o, call.final_state), clean, same_o, same_s)
    assert call.device_status() == 0


# ------------------------------------------------------------------ range
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_large_products_in_decaying_chunks(dk, dv):
    """Chunks that decay by nearly 2^64 and products q.k of some 2^70: o of 2^70 is well within bf16 and fp32."""
    lens, H = [300, 128, 40], 2
    d = inputs(3 * dk + dv, sum(lens), H, H, dk, dv, "bf16", None, n=3)
    d["q"], d["k"], d["state"] = d["q"] * 2.0 ** 33, d["k"] * 2.0 ** 33, d["state"] * 2.0 ** 33
    d["slope"] = torch.tensor([63.0, 40.0], device="cuda") / 128 * math.log(2.0)
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), slope=d["slope"], initial_state=d["state"])
    check_prefill(d, lens, H, dk, "bf16", o, final, 1.0)


@pytest.mark.parametrize("dk,dv", SHAPES)
def test_small_products_in_decaying_chunks(dk, dv):
    """And products of some 2^-60, which the factors of such a chunk must not push out of bf16."""
    lens, H = [300, 128, 40], 2
    d = inputs(5 * dk + dv, sum(lens), H, H, dk, dv, "bf16", None, n=3)
    d["q"], d["k"], d["state"] = d["q"] * 2.0 ** -32, d["k"] * 2.0 ** -32, d["state"] * 2.0 ** -32
    d["slope"] = torch.tensor([63.0, 40.0], device="cuda") / 128 * math.log(2.0)
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), slope=d["slope"], initial_state=d["state"])
    check_prefill(d, lens, H, dk, "bf16", o, final, 1.0)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 64)])
def test_gates_that_are_not_numbers_in_decaying_chunks(dk, dv):
    """Tokens before one whose gate is NaN keep their bits, whatever their chunk decays by."""
    lens, H, t = [300], 2, 240
    d = inputs(dk, 300, H, H, dk, dv, "bf16", "g", n=1)
    d["g"] = torch.full_like(d["g"], -1.1)  # log2 alpha -0.41: 53 in a chunk
    clean = prompts(d, lens)
    d["g"][t, 1] = float("nan")
    o, final = prompts(d, lens)
    same = torch.ones(300, H, dtype=torch.bool, device="cuda")
    same[t:, 1] = False
    assert torch.equal(o[same], clean[0][same]) and torch.equal(final[:, 0], clean[1][:, 0])
    assert not torch.isfinite(o[t:, 1].float()).any() and not torch.isfinite(final[:, 1]).any()
