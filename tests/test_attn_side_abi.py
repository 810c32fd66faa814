"""Argument checks of the attention-side operators (on the host, no GPU)."""
import ctypes

import pytest

import expert_cache_host_gb300 as ft
from expert_cache_host_gb300 import build as ftbuild

PTR = 1 << 20  # never dereferenced: every call below is refused (or has no rows) before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    ftbuild.build()
    return ft.load()


def cache(**kw):
    a = dict(k=PTR, v=2 * PTR, dtype=ft.FT_DTYPE_BF16, num_pages=4, page_size=16, kv_heads=2, head_dim=128,
             k_page_stride=16 * 256, k_token_stride=256, k_head_stride=128,
             v_page_stride=16 * 256, v_token_stride=256, v_head_stride=128)
    a.update(kw)
    return ft.make_kv_cache(**a)


def plan(**kw):
    a = dict(ctx_len=PTR, new_len=PTR, free_pages=PTR, free_count=PTR, block_table=PTR, q_start=PTR, slots=PTR,
             positions=PTR, free_left=2 * PTR, num_reqs=2, page_size=16, table_width=4, max_tokens=8, mask_words=0)
    a.update(kw)
    return ft.make_plan_args(**a)


def qk(cache_kw=None, **kw):
    a = dict(q=PTR, k=PTR, v=PTR, q_weight=PTR, k_weight=PTR, cos_sin=PTR, positions=PTR, slots=PTR, q_out=2 * PTR,
             q_stride=1024, k_stride=256, v_stride=256, q_out_stride=1024, T=3, q_heads=8, rot_dim=128, max_pos=64,
             interleaved=0, eps=1e-6, cache=cache(**(cache_kw or {})))
    a.update(kw)
    return ft.make_qk_args(**a)


def attn(cache_kw=None, **kw):
    a = dict(q=PTR, out=PTR, q_start=PTR, ctx_len=PTR, block_table=PTR, workspace=PTR, q_stride=1024, out_stride=1024,
             workspace_bytes=1 << 40, max_tokens=3, num_reqs=2, q_heads=8, table_width=4, mask_words=0, scale=0.1,
             cache=cache(**(cache_kw or {})))
    a.update(kw)
    return ft.make_attn_args(**a)


def logprob(**kw):
    a = dict(logits=PTR, tokens=PTR, logprob=PTR, entropy=PTR, top_ids=PTR, top_logprobs=PTR, row_stride=100,
             dtype=ft.FT_DTYPE_BF16, T=2, V=100, top_n=5)
    a.update(kw)
    return ft.make_logprob_args(**a)


def refused(call, args, code=ft.FT_E_ARG):
    with pytest.raises(ft.FtError) as ei:
        call(args)
    assert ei.value.code == code, ei.value


@pytest.mark.parametrize("kw", [
    dict(num_reqs=-1), dict(max_tokens=-1), dict(table_width=-1), dict(mask_words=-1), dict(page_size=0),
    dict(page_size=24), dict(ctx_len=0), dict(new_len=0), dict(block_table=0), dict(free_pages=0), dict(q_start=0),
    dict(free_count=0), dict(free_left=0), dict(slots=0), dict(positions=0), dict(free_left=PTR),
    dict(parents=PTR), dict(parents=PTR, mask=PTR), dict(mask_words=1), dict(reserved=1), dict(max_tokens=(1 << 30) + 1)],
    ids=str)
def test_plan_refusals(kw):
    refused(ft.ft_kv_plan, plan(**kw))


BAD_CACHE = [(dict(k=0), ft.FT_E_ARG), (dict(v=0), ft.FT_E_ARG), (dict(dtype=ft.FT_DTYPE_MXFP4), ft.FT_E_ARG),
             (dict(dtype=ft.FT_DTYPE_F32), ft.FT_E_ARG), (dict(num_pages=0), ft.FT_E_ARG), (dict(kv_heads=0), ft.FT_E_ARG),
             (dict(page_size=0), ft.FT_E_ARG), (dict(page_size=4), ft.FT_E_UNSUPPORTED),
             (dict(page_size=24), ft.FT_E_UNSUPPORTED), (dict(page_size=8192), ft.FT_E_UNSUPPORTED),
             (dict(head_dim=96), ft.FT_E_UNSUPPORTED), (dict(k=PTR + 2), ft.FT_E_ARG), (dict(v=PTR + 8), ft.FT_E_ARG),
             (dict(k_token_stride=130), ft.FT_E_ARG), (dict(v_page_stride=-8), ft.FT_E_ARG),
             (dict(v_head_stride=1 << 38), ft.FT_E_ARG), (dict(k_token_stride=0), ft.FT_E_ARG),
             (dict(k_head_stride=0), ft.FT_E_ARG), (dict(v_page_stride=0), ft.FT_E_ARG), (dict(reserved=1), ft.FT_E_ARG)]


@pytest.mark.parametrize("kw,code", BAD_CACHE, ids=str)
def test_cache_refusals(kw, code):
    refused(ft.ft_qk_norm_rope, qk(cache_kw=kw), code)
    refused(ft.ft_tree_attention, attn(cache_kw=kw), code)
    refused(ft.ft_tree_attention_workspace, attn(cache_kw=kw), code)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), ft.FT_E_ARG), (dict(q_heads=0), ft.FT_E_ARG), (dict(max_pos=0), ft.FT_E_ARG), (dict(q=0), ft.FT_E_ARG),
    (dict(k=0), ft.FT_E_ARG), (dict(v=0), ft.FT_E_ARG), (dict(q_weight=0), ft.FT_E_ARG), (dict(k_weight=0), ft.FT_E_ARG),
    (dict(cos_sin=0), ft.FT_E_ARG), (dict(positions=0), ft.FT_E_ARG), (dict(slots=0), ft.FT_E_ARG),
    (dict(q_out=0), ft.FT_E_ARG), (dict(rot_dim=-16), ft.FT_E_ARG), (dict(rot_dim=144), ft.FT_E_ARG),
    (dict(rot_dim=24), ft.FT_E_UNSUPPORTED), (dict(cos_sin=PTR + 4), ft.FT_E_ARG), (dict(q_weight=PTR + 2), ft.FT_E_ARG),
    (dict(eps=-1.0), ft.FT_E_ARG), (dict(eps=float("nan")), ft.FT_E_ARG), (dict(q_out=PTR, q_out_stride=2048), ft.FT_E_ARG),
    (dict(q_stride=-1), ft.FT_E_ARG)], ids=str)
def test_qk_refusals(kw, code):
    refused(ft.ft_qk_norm_rope, qk(**kw), code)


@pytest.mark.parametrize("name", ["q", "k", "v", "q_out"])
def test_qk_refuses_rows_between_elements(name):
    refused(ft.ft_qk_norm_rope, qk(**{name: PTR + 1}), ft.FT_E_ARG)


@pytest.mark.parametrize("kw,code", [
    (dict(max_tokens=-1), ft.FT_E_ARG), (dict(num_reqs=-1), ft.FT_E_ARG), (dict(q_heads=0), ft.FT_E_ARG),
    (dict(q_heads=7), ft.FT_E_ARG), (dict(q_heads=2 * 129), ft.FT_E_UNSUPPORTED), (dict(q=0), ft.FT_E_ARG),
    (dict(out=0), ft.FT_E_ARG), (dict(q_start=0), ft.FT_E_ARG), (dict(ctx_len=0), ft.FT_E_ARG),
    (dict(block_table=0), ft.FT_E_ARG), (dict(workspace=0), ft.FT_E_ARG), (dict(workspace=PTR + 4), ft.FT_E_ARG),
    (dict(workspace_bytes=0), ft.FT_E_ARG), (dict(q=PTR + 2), ft.FT_E_ARG), (dict(out=PTR + 2), ft.FT_E_ARG),
    (dict(q_stride=1023), ft.FT_E_ARG), (dict(out_stride=1020), ft.FT_E_ARG), (dict(mask=PTR), ft.FT_E_ARG),
    (dict(mask_words=2), ft.FT_E_ARG), (dict(table_width=0), ft.FT_E_ARG), (dict(scale=float("nan")), ft.FT_E_ARG),
    (dict(scale=float("inf")), ft.FT_E_ARG)], ids=str)
def test_attention_refusals(kw, code):
    refused(ft.ft_tree_attention, attn(**kw), code)


@pytest.mark.parametrize("kw", [
    dict(dtype=ft.FT_DTYPE_MXFP4), dict(T=-1), dict(V=0), dict(top_n=-1), dict(top_n=33), dict(top_n=5, V=4),
    dict(logits=0), dict(logits=PTR + 1), dict(row_stride=-1), dict(top_ids=0), dict(top_logprobs=0), dict(tokens=0),
    dict(logprob=0), dict(dtype=ft.FT_DTYPE_F32, logits=PTR + 2)], ids=str)
def test_logprob_refusals(kw):
    refused(ft.ft_token_logprobs, logprob(**kw))


def test_null_args_and_unknown_fields():
    lib = ft.load()
    for name in ("ft_kv_plan", "ft_qk_norm_rope", "ft_tree_attention", "ft_token_logprobs"):
        assert getattr(lib, name)(None, None) == ft.FT_E_ARG
    assert lib.ft_tree_attention_workspace(None, None) == ft.FT_E_ARG
    with pytest.raises(TypeError):
        ft.make_attn_args(no_such_field=1)


def test_no_rows_is_ok_without_a_launch():
    ft.ft_qk_norm_rope(qk(T=0))
    ft.ft_tree_attention(attn(max_tokens=0))
    ft.ft_tree_attention(attn(num_reqs=0))
    ft.ft_token_logprobs(logprob(T=0))


def test_workspace_grows_with_nothing_but_sizes():
    a = attn(workspace=0, workspace_bytes=0, q=0, out=0, q_start=0, ctx_len=0, block_table=0)
    n = ft.ft_tree_attention_workspace(a)
    assert n > 0 and n % 16 == 0
    assert ft.ft_tree_attention_workspace(a) == n


def test_struct_sizes_match_the_header():
    """The binding's structures lie as C lays out the header's."""
    import os
    import subprocess
    import tempfile
    names = ["ft_kv_cache", "ft_plan_args", "ft_qk_args", "ft_attn_args", "ft_logprob_args"]
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "ft_moe.h"\nint main(void) {\n'
    for n in names:
        src += f'  printf("%zu\\n", sizeof({n}));\n'
        for f in getattr(ft, n)._fields_:
            src += f'  printf("%zu\\n", offsetof({n}, {f[0]}));\n'
    src += "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c = os.path.join(d, "sizes.c")
        with open(c, "w") as f:
            f.write(src)
        exe = os.path.join(d, "sizes")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for n in names:
        s = getattr(ft, n)
        want += [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def test_workspace_follows_the_head_size_alone():
    size = lambda **kw: ft.ft_tree_attention_workspace(attn(workspace=0, workspace_bytes=0, **kw))
    n = size()
    for kw in (dict(max_tokens=1), dict(max_tokens=100000), dict(num_reqs=1), dict(num_reqs=5000), dict(q_heads=2),
               dict(q_heads=256), dict(mask=PTR, mask_words=4), dict(cache_kw=dict(dtype=ft.FT_DTYPE_F16)),
               dict(cache_kw=dict(num_pages=100000)), dict(cache_kw=dict(page_size=64)), dict(cache_kw=dict(kv_heads=1))):
        assert size(**kw) == n, kw
    half = size(cache_kw=dict(head_dim=64))
    # a part's maximum and sum (8 bytes a row) and the joins' list do not shrink with the head
    assert n // 2 < half < n // 2 + n // 50
