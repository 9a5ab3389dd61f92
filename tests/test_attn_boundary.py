"""Host-side checks of the full-attention and paged-cache entry points (no GPU):
structure layouts against a C program, refusals before any launch, workspace
sizes, and the Python binding's checks of shapes and types.
"""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def kda():
    from linear_attention_serving_delta_gb300 import build, kda as binding
    build.build()
    binding.lib()
    return binding


def structs(kda):
    return {"kda_attn_prefill_args": kda.AttnPrefillArgs, "kda_attn_paged_args": kda.AttnPagedArgs,
            "kda_kv_plan_args": kda.KvPlanArgs, "kda_kv_release_args": kda.KvReleaseArgs,
            "kda_kv_write_args": kda.KvWriteArgs}


def test_struct_layouts_match_c(kda, tmp_path):
    body = []
    for name, cls in structs(kda).items():
        body.append(f'printf("{name} %zu\\n", sizeof({name}));')
        body += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    c = tmp_path / "layout.c"
    c.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kda.h"\nint main(void) {\n'
                 + "\n".join(body) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = dict(line.rsplit(" ", 1) for line in out.splitlines())
    want = {}
    for name, cls in structs(kda).items():
        want[name] = ctypes.sizeof(cls)
        want.update({f"{name}.{f}": getattr(cls, f).offset for f, _ in cls._fields_})
    assert {k: int(v) for k, v in got.items()} == want


PTR = 0x1000  # never dereferenced: every call below is refused before a launch


def prefill_args(kda, **over):
    a = kda.AttnPrefillArgs()
    a.num_seqs, a.num_heads, a.num_kv_heads, a.head_dim, a.total_tokens = 2, 8, 2, 64, 100
    a.in_dtype, a.scale = kda.KDA_BF16, 0.125
    a.cu_seqlens = a.q = a.k = a.v = a.o = PTR
    for k, v in over.items():
        setattr(a, k, v)
    return a


def paged_args(kda, **over):
    a = kda.AttnPagedArgs()
    a.num_seqs, a.num_heads, a.num_kv_heads, a.head_dim, a.total_tokens = 2, 8, 2, 64, 2
    a.in_dtype, a.scale, a.max_seqlen = kda.KDA_BF16, 0.125, 1
    a.num_pages, a.page_size, a.num_rows, a.max_pages = 40, 16, 2, 20
    a.cu_seqlens = a.q = a.k_cache = a.v_cache = a.o = a.block_table = a.kv_lens = PTR
    for k, v in over.items():
        setattr(a, k, v)
    return a


def plan_args(kda, **over):
    a = kda.KvPlanArgs()
    a.num_seqs, a.total_tokens, a.page_size, a.num_pages, a.num_rows, a.max_pages = 2, 10, 16, 40, 2, 20
    a.cu_seqlens = a.block_table = a.kv_lens_in = a.kv_lens_out = a.free_pages = PTR
    a.free_count_in = a.free_count_out = a.slot_map = PTR
    for k, v in over.items():
        setattr(a, k, v)
    return a


def release_args(kda, **over):
    a = kda.KvReleaseArgs()
    a.num_release, a.page_size, a.num_pages, a.num_rows, a.max_pages = 2, 16, 40, 2, 20
    a.rows = a.block_table = a.kv_lens = a.free_pages = a.free_count = PTR
    for k, v in over.items():
        setattr(a, k, v)
    return a


def write_args(kda, **over):
    a = kda.KvWriteArgs()
    a.total_tokens, a.num_kv_heads, a.head_dim, a.in_dtype, a.num_slots = 4, 2, 64, kda.KDA_BF16, 64
    a.k = a.v = a.slot_map = a.k_cache = a.v_cache = PTR
    for k, v in over.items():
        setattr(a, k, v)
    return a


HEADS = [(dict(num_heads=0), INVALID), (dict(num_kv_heads=0), INVALID), (dict(num_kv_heads=3), INVALID),
         (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(in_dtype=2), INVALID),
         (dict(num_heads=129, num_kv_heads=1), UNSUPPORTED), (dict(num_seqs=0), INVALID),
         (dict(total_tokens=-1), INVALID), (dict(total_tokens=1 << 30), UNSUPPORTED),
         (dict(cu_seqlens=None), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID)]
PAGES = [(dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
         (dict(num_pages=-1), INVALID), (dict(num_rows=-1), INVALID), (dict(max_pages=-1), INVALID),
         (dict(max_pages=1 << 27), UNSUPPORTED)]  # positions past int32


@pytest.mark.parametrize("over,status", HEADS + [(dict(k=None), INVALID), (dict(v=None), INVALID)])
def test_attn_prefill_refuses(kda, over, status):
    a = prefill_args(kda, **over)
    assert kda.lib().kda_attn_prefill_workspace_size(ctypes.byref(a)) == 0
    assert kda.lib().kda_attn_prefill(ctypes.byref(a), 0x100, 1 << 40, None) == status


@pytest.mark.parametrize("over,status", HEADS + PAGES + [
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(block_table=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(max_seqlen=-1), INVALID), (dict(num_rows=1), INVALID)])
def test_attn_paged_refuses(kda, over, status):
    a = paged_args(kda, **over)
    assert kda.lib().kda_attn_paged_workspace_size(ctypes.byref(a)) == 0
    assert kda.lib().kda_attn_paged(ctypes.byref(a), 0x100, 1 << 40, None) == status


@pytest.mark.parametrize("over,status", PAGES + [
    (dict(num_seqs=0), INVALID), (dict(total_tokens=-1), INVALID), (dict(cu_seqlens=None), INVALID),
    (dict(num_rows=1), INVALID), (dict(block_table=None), INVALID), (dict(kv_lens_in=None), INVALID),
    (dict(kv_lens_out=None), INVALID), (dict(free_pages=None), INVALID), (dict(free_count_in=None), INVALID),
    (dict(free_count_out=None), INVALID), (dict(slot_map=None), INVALID)])
def test_kv_plan_refuses(kda, over, status):
    a = plan_args(kda, **over)
    assert kda.lib().kda_kv_plan_workspace_size(ctypes.byref(a)) == 0
    assert kda.lib().kda_kv_plan(ctypes.byref(a), 0x100, 1 << 40, None) == status


@pytest.mark.parametrize("over,status", PAGES + [
    (dict(num_release=-1), INVALID), (dict(rows=None), INVALID), (dict(free_count=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(block_table=None), INVALID), (dict(free_pages=None), INVALID)])
def test_kv_release_refuses(kda, over, status):
    a = release_args(kda, **over)
    assert kda.lib().kda_kv_release_workspace_size(ctypes.byref(a)) == 0
    assert kda.lib().kda_kv_release(ctypes.byref(a), 0x100, 1 << 40, None) == status


@pytest.mark.parametrize("over,status", [
    (dict(total_tokens=-1), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=48), UNSUPPORTED),
    (dict(in_dtype=7), INVALID), (dict(num_slots=-1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(slot_map=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID)])
def test_kv_write_refuses(kda, over, status):
    a = write_args(kda, **over)
    assert kda.lib().kda_kv_write(ctypes.byref(a), None) == status


def test_null_argument_blocks(kda):
    L = kda.lib()
    for name in ("kda_attn_prefill", "kda_attn_paged", "kda_kv_plan", "kda_kv_release"):
        assert getattr(L, name + "_workspace_size")(None) == 0
        assert getattr(L, name)(None, 0x100, 1 << 40, None) == INVALID
    assert L.kda_kv_write(None, None) == INVALID


def test_workspace_is_checked(kda):
    L = kda.lib()
    for name, a in (("kda_attn_prefill", prefill_args(kda)), ("kda_attn_paged", paged_args(kda)),
                    ("kda_kv_plan", plan_args(kda)), ("kda_kv_release", release_args(kda))):
        n = getattr(L, name + "_workspace_size")(ctypes.byref(a))
        assert n >= 256 and n % 256 == 0
        call = getattr(L, name)
        assert call(ctypes.byref(a), None, n, None) == WORKSPACE
        assert call(ctypes.byref(a), 0x100, n - 1, None) == WORKSPACE
        assert call(ctypes.byref(a), 0x140, n, None) == WORKSPACE


def test_binding_refuses_host_tensors_and_shapes(kda):
    q, k = torch.zeros(4, 8, 64), torch.zeros(4, 2, 64)
    cu = torch.tensor([0, 4])
    with pytest.raises(ValueError):
        kda.AttnPrefill(q, k, k, cu)            # host tensors
    with pytest.raises(ValueError):
        kda.AttnPrefill(q, k[:3], k, cu)        # shapes
    with pytest.raises(ValueError):
        kda.AttnPrefill(q, torch.zeros(4, 3, 64), torch.zeros(4, 3, 64), cu)  # 8 heads over 3
    cache = torch.zeros(4, 16, 2, 64)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        kda.AttnPaged(q, cache, cache, table, lens, cu)
    with pytest.raises(ValueError):
        kda.AttnPaged(q, cache, cache[:, :, :1], table, lens, cu)
    with pytest.raises(ValueError):
        kda.KvWrite(k, k, torch.zeros(3, dtype=torch.int64), cache, cache)
    with pytest.raises(ValueError):
        kda.KvPlan(cu, 4, table, lens, torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                   page_size=16)
    with pytest.raises(ValueError):
        kda.KvRelease(torch.zeros(1, 1, dtype=torch.int32), table, lens, torch.zeros(4, dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32), page_size=16)
