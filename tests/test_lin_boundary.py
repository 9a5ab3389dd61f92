"""Host-side checks of the linear-attention entry points (no GPU): structure
layouts against a C program, refusals before any launch, workspace sizes, and
the Python binding's checks of shapes, types and numbers.
"""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
PTR = 0x1000  # never dereferenced: every call below is refused before a launch


@pytest.fixture(scope="module")
def kda():
    from linear_attention_serving_delta_gb300 import build, kda as binding
    build.build()
    binding.lib()
    return binding


def test_struct_layouts_match_c(kda, tmp_path):
    structs = {"kda_lin_prefill_args": kda.LinPrefillArgs, "kda_lin_decode_args": kda.LinDecodeArgs,
               "kda_lin_draft_args": kda.LinDraftArgs, "kda_lin_commit_args": kda.LinCommitArgs}
    body = ['printf("draft %d\\n", KDA_LIN_MAX_DRAFT);']
    for name, cls in structs.items():
        body.append(f'printf("{name} %zu\\n", sizeof({name}));')
        body += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    c = tmp_path / "layout.c"
    c.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kda.h"\nint main(void) {\n'
                 + "\n".join(body) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {k: int(v) for k, v in (line.rsplit(" ", 1) for line in out.splitlines())}
    want = {"draft": kda.LIN_MAX_DRAFT}
    for name, cls in structs.items():
        want[name] = ctypes.sizeof(cls)
        want.update({f"{name}.{f}": getattr(cls, f).offset for f, _ in cls._fields_})
    assert got == want


def block(cls, kda, **over):
    a = cls()
    for n in ("num_seqs", "batch"):
        if hasattr(a, n):
            setattr(a, n, 2)
    a.num_heads, a.num_key_heads, a.dk, a.dv, a.in_dtype, a.num_states = 8, 2, 64, 128, kda.KDA_BF16, 2
    if hasattr(a, "total_tokens"):
        a.total_tokens = 100
    for n in ("cu_seqlens", "q", "k", "v", "g", "o", "state", "state_out", "initial_state", "final_state", "last"):
        if hasattr(a, n):
            setattr(a, n, PTR)
    for k, v in over.items():
        assert hasattr(a, k)
        setattr(a, k, v)
    return a


HEADS = [(dict(num_heads=0), INVALID), (dict(num_key_heads=0), INVALID), (dict(num_key_heads=3), INVALID),
         (dict(num_heads=65536, num_key_heads=1), UNSUPPORTED), (dict(dk=96), UNSUPPORTED), (dict(dv=0), UNSUPPORTED),
         (dict(in_dtype=2), INVALID), (dict(g=None), INVALID), (dict(num_states=-1), INVALID),
         (dict(num_states=1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID)]
TOKENS = [(dict(num_seqs=0), INVALID), (dict(total_tokens=-1), INVALID), (dict(total_tokens=1 << 30), UNSUPPORTED),
          (dict(cu_seqlens=None), INVALID)]
TREES = [(dict(max_seqlen=-1), INVALID), (dict(max_seqlen=65), UNSUPPORTED), (dict(state=None), INVALID),
         (dict(state=PTR + 4), INVALID)]


@pytest.mark.parametrize("over,status", HEADS + TOKENS + [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(initial_state=PTR + 8), INVALID),
    (dict(final_state=PTR + 4), INVALID)])
def test_lin_prefill_refuses(kda, over, status):
    a = block(kda.LinPrefillArgs, kda, **over)
    assert kda.lib().kda_lin_prefill_workspace_size(ctypes.byref(a)) == 0
    assert kda.lib().kda_lin_prefill(ctypes.byref(a), 0x100, 1 << 40, None) == status


@pytest.mark.parametrize("over,status", HEADS + [
    (dict(batch=-1), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(state=None), INVALID),
    (dict(state_out=None), INVALID), (dict(state_out=PTR + 4), INVALID)])
def test_lin_decode_refuses(kda, over, status):
    assert kda.lib().kda_lin_decode(ctypes.byref(block(kda.LinDecodeArgs, kda, **over)), None) == status


@pytest.mark.parametrize("over,status", HEADS + TOKENS + TREES + [(dict(q=None), INVALID), (dict(o=None), INVALID)])
def test_lin_draft_refuses(kda, over, status):
    assert kda.lib().kda_lin_draft(ctypes.byref(block(kda.LinDraftArgs, kda, **over)), None) == status


@pytest.mark.parametrize("over,status", HEADS + TOKENS + TREES + [
    (dict(last=None), INVALID), (dict(state_out=None), INVALID), (dict(state_out=PTR + 8), INVALID)])
def test_lin_commit_refuses(kda, over, status):
    assert kda.lib().kda_lin_commit(ctypes.byref(block(kda.LinCommitArgs, kda, **over)), None) == status


def test_null_argument_blocks(kda):
    L = kda.lib()
    assert L.kda_lin_prefill_workspace_size(None) == 0
    assert L.kda_lin_prefill(None, 0x100, 1 << 40, None) == INVALID
    for name in ("kda_lin_decode", "kda_lin_draft", "kda_lin_commit"):
        assert getattr(L, name)(None, None) == INVALID


@pytest.mark.parametrize("over", [{}, dict(in_dtype=0), dict(initial_state=None, final_state=None, num_states=0),
                                  dict(total_tokens=0, q=None, k=None, v=None, o=None), dict(total_tokens=100000)])
def test_workspace_is_checked(kda, over):
    a, L = block(kda.LinPrefillArgs, kda, **over), kda.lib()
    n = L.kda_lin_prefill_workspace_size(ctypes.byref(a))
    assert n >= 256 and n % 256 == 0
    assert L.kda_lin_prefill(ctypes.byref(a), None, n, None) == WORKSPACE
    assert L.kda_lin_prefill(ctypes.byref(a), 0x100, n - 1, None) == WORKSPACE
    assert L.kda_lin_prefill(ctypes.byref(a), 0x140, n, None) == WORKSPACE


@pytest.mark.parametrize("tokens", [100, 5000, 100000])
def test_workspace_is_enough_for_any_alignment(kda, tokens):
    size = kda.lib().kda_lin_prefill_workspace_size
    args = [block(kda.LinPrefillArgs, kda, total_tokens=tokens, q=PTR + off) for off in (0, 2)]
    assert size(ctypes.byref(args[0])) == size(ctypes.byref(args[1])) > 0
    # and a call that takes the other path still refuses less than that
    assert kda.lib().kda_lin_prefill(ctypes.byref(args[1]), 0x100, size(ctypes.byref(args[0])) - 1, None) == WORKSPACE


def test_binding_refuses(kda, monkeypatch):
    # (shapes and numbers are looked at before anything that needs a GPU)
    monkeypatch.setattr(kda, "_same_device", lambda **t: torch.device("cpu"))
    monkeypatch.setattr(kda, "_ptr", lambda t, dtype=None, name="": None if t is None else t.data_ptr())
    monkeypatch.setattr(kda._CacheCall, "_plan", lambda self, dev, a, keep, status: None)
    q, k, v = torch.zeros(6, 2, 16), torch.zeros(6, 2, 16), torch.zeros(6, 4, 32)
    cu, g, state = torch.tensor([0, 2, 6]), torch.zeros(6, 4), torch.zeros(3, 4, 16, 32)
    slots, last = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kda.LinPrefill(q, k, v, cu, g=g)
    kda.LinPrefill(q, k, v, cu, g=g, initial_state=state, state_slots=slots)
    kda.LinDraft(q, k, v, cu, state, g=g, max_seqlen=4)
    kda.LinCommit(k, v, cu, last, state, slope=torch.zeros(4))
    bad = [lambda: kda.LinPrefill(q, k, v, cu),                                     # no decay
           lambda: kda.LinPrefill(q, k, v, cu, g=g[:, :2]),
           lambda: kda.LinPrefill(q, k, v, cu, slope=torch.zeros(2)),
           lambda: kda.LinPrefill(q[:5], k, v, cu, g=g),
           lambda: kda.LinPrefill(q, k, v[:, :3], cu, g=g[:, :3]),                  # 3 heads over 2
           lambda: kda.LinPrefill(q, k, v, cu, g=g, o=v[:5]),
           lambda: kda.LinPrefill(q, k, v, cu, g=g, initial_state=state[:1]),       # fewer rows than sequences
           lambda: kda.LinPrefill(q, k, v, cu, g=g, initial_state=state, final_state=state[:2]),
           lambda: kda.LinPrefill(q, k, v, cu, g=g, initial_state=state[:, :2]),
           lambda: kda.LinPrefill(q, k, v, cu, g=g, state_slots=slots),             # rows not known
           lambda: kda.LinPrefill(q, k, v, cu, g=g, initial_state=state, state_slots=slots[:1]),
           lambda: kda.LinPrefill(q, k, v, cu[:1], g=g),
           lambda: kda.LinDecode(q, k, v, state, g=g),                              # 6 rows, 3 states
           lambda: kda.LinDecode(q, k, v, state, g=g, state_slots=slots),
           lambda: kda.LinDraft(q, k, v, cu, state, g=g, max_seqlen=65),
           lambda: kda.LinDraft(q, k, v, cu, state, g=g, max_seqlen=(1 << 32) + 1),
           lambda: kda.LinDraft(q, k, v, cu, state, g=g, max_seqlen=-1),
           lambda: kda.LinDraft(q, k, v, cu, state, g=g, parents=slots),
           lambda: kda.LinCommit(k, v, cu, last[:1], state, g=g)]
    for make in bad:
        with pytest.raises(ValueError):
            make()


def test_binding_refuses_host_tensors(kda):
    x, cu = torch.zeros(2, 2, 16), torch.tensor([0, 2])
    with pytest.raises(ValueError, match="CUDA"):
        kda.LinPrefill(x, x, x, cu, slope=torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        kda.LinDecode(x, x, x, torch.zeros(2, 2, 16, 16), slope=torch.zeros(2))
