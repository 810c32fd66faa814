"""Argument checks of the 8-bit cache's operators (on the host, no GPU)."""
import ctypes

import numpy as np
import pytest

import expert_cache_host_gb300 as ft
import kv8_reference as ref
from expert_cache_host_gb300 import build as ftbuild

PTR = 1 << 20  # never dereferenced: every call below is refused (or has no rows) before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    ftbuild.build()
    return ft.load()


def cache(**kw):
    a = dict(k=PTR, v=2 * PTR, k_scale=3 * PTR, v_scale=4 * PTR, num_pages=4, page_size=32, block_size=16, kv_heads=2,
             head_dim=128, k_page_stride=32 * 256, k_token_stride=256, k_head_stride=128,
             v_page_stride=32 * 256, v_token_stride=256, v_head_stride=128)
    a.update(kw)
    return ft.make_kv8_cache(**a)


def store(cache_kw=None, **kw):
    a = dict(k=PTR, v=PTR, q_start=PTR, ctx_len=PTR, block_table=PTR, k_stride=256, v_stride=256, dtype=ft.FT_DTYPE_BF16,
             max_tokens=3, num_reqs=2, table_width=4, cache=cache(**(cache_kw or {})))
    a.update(kw)
    return ft.make_kv8_store_args(**a)


def load(cache_kw=None, **kw):
    a = dict(k=PTR, v=PTR, slots=PTR, k_stride=256, v_stride=256, dtype=ft.FT_DTYPE_F16, T=3, cache=cache(**(cache_kw or {})))
    a.update(kw)
    return ft.make_kv8_load_args(**a)


def attn(cache_kw=None, **kw):
    a = dict(q=PTR, out=PTR, q_start=PTR, ctx_len=PTR, block_table=PTR, workspace=PTR, q_stride=1024, out_stride=1024,
             workspace_bytes=1 << 40, dtype=ft.FT_DTYPE_BF16, max_tokens=3, max_new=0, num_reqs=2, q_heads=8, table_width=4,
             mask_words=0, scale=0.1, cache=cache(**(cache_kw or {})))
    a.update(kw)
    return ft.make_kv8_attn_args(**a)


def refused(call, args, code=ft.FT_E_ARG):
    with pytest.raises(ft.FtError) as ei:
        call(args)
    assert ei.value.code == code, ei.value


BAD_CACHE = [(dict(k=0), ft.FT_E_ARG), (dict(v=0), ft.FT_E_ARG), (dict(k_scale=0), ft.FT_E_ARG),
             (dict(v_scale=0), ft.FT_E_ARG), (dict(num_pages=0), ft.FT_E_ARG), (dict(kv_heads=0), ft.FT_E_ARG),
             (dict(page_size=0), ft.FT_E_ARG), (dict(block_size=0), ft.FT_E_ARG), (dict(block_size=-16), ft.FT_E_ARG),
             (dict(page_size=8), ft.FT_E_UNSUPPORTED), (dict(page_size=48), ft.FT_E_UNSUPPORTED),
             (dict(page_size=8192), ft.FT_E_UNSUPPORTED), (dict(block_size=8), ft.FT_E_UNSUPPORTED),
             (dict(block_size=24), ft.FT_E_UNSUPPORTED), (dict(block_size=64), ft.FT_E_UNSUPPORTED),
             (dict(page_size=256, block_size=256), ft.FT_E_UNSUPPORTED), (dict(head_dim=96), ft.FT_E_UNSUPPORTED),
             (dict(head_dim=256), ft.FT_E_UNSUPPORTED), (dict(kv_heads=20000), ft.FT_E_UNSUPPORTED),
             (dict(k=PTR + 2), ft.FT_E_ARG), (dict(v=PTR + 8), ft.FT_E_ARG), (dict(k_token_stride=264), ft.FT_E_ARG),
             (dict(v_page_stride=-16), ft.FT_E_ARG), (dict(v_head_stride=1 << 38), ft.FT_E_ARG),
             (dict(k_token_stride=0), ft.FT_E_ARG), (dict(k_head_stride=0), ft.FT_E_ARG),
             (dict(v_page_stride=0), ft.FT_E_ARG), (dict(reserved=1), ft.FT_E_ARG)]


@pytest.mark.parametrize("kw,code", BAD_CACHE, ids=str)
def test_cache_refusals(kw, code):
    refused(ft.ft_kv8_store, store(cache_kw=kw), code)
    refused(ft.ft_kv8_load, load(cache_kw=kw), code)
    refused(ft.ft_kv8_attention, attn(cache_kw=kw), code)
    refused(ft.ft_kv8_attention_workspace, attn(cache_kw=kw), code)


ROWS = [dict(k=0), dict(v=0), dict(k=PTR + 2), dict(v=PTR + 8), dict(k_stride=-8), dict(v_stride=257),
        dict(k_stride=1 << 38), dict(dtype=ft.FT_DTYPE_F32), dict(dtype=ft.FT_DTYPE_MXFP4)]


@pytest.mark.parametrize("kw", ROWS + [dict(max_tokens=-1), dict(num_reqs=-1), dict(table_width=-1), dict(table_width=0),
                                       dict(q_start=0), dict(ctx_len=0), dict(block_table=0)], ids=str)
def test_store_refusals(kw):
    refused(ft.ft_kv8_store, store(**kw))


@pytest.mark.parametrize("kw", ROWS + [dict(T=-1), dict(slots=0), dict(k_stride=248), dict(v_stride=0)], ids=str)
def test_load_refusals(kw):
    refused(ft.ft_kv8_load, load(**kw))


@pytest.mark.parametrize("kw,code", [
    (dict(max_tokens=-1), ft.FT_E_ARG), (dict(max_new=-1), ft.FT_E_ARG), (dict(num_reqs=-1), ft.FT_E_ARG),
    (dict(q_heads=0), ft.FT_E_ARG), (dict(q_heads=7), ft.FT_E_ARG), (dict(q_heads=2 * 129), ft.FT_E_UNSUPPORTED),
    (dict(dtype=ft.FT_DTYPE_F32), ft.FT_E_ARG), (dict(q=0), ft.FT_E_ARG), (dict(out=0), ft.FT_E_ARG),
    (dict(q_start=0), ft.FT_E_ARG), (dict(ctx_len=0), ft.FT_E_ARG), (dict(block_table=0), ft.FT_E_ARG),
    (dict(workspace=0), ft.FT_E_ARG), (dict(workspace=PTR + 4), ft.FT_E_ARG), (dict(workspace_bytes=0), ft.FT_E_ARG),
    (dict(q=PTR + 2), ft.FT_E_ARG), (dict(out=PTR + 2), ft.FT_E_ARG), (dict(q_stride=1023), ft.FT_E_ARG),
    (dict(out_stride=1020), ft.FT_E_ARG), (dict(mask=PTR), ft.FT_E_ARG), (dict(mask_words=2), ft.FT_E_ARG),
    (dict(table_width=0), ft.FT_E_ARG), (dict(scale=float("nan")), ft.FT_E_ARG), (dict(scale=float("inf")), ft.FT_E_ARG)],
    ids=str)
def test_attention_refusals(kw, code):
    refused(ft.ft_kv8_attention, attn(**kw), code)


def test_null_args_unknown_fields_and_no_rows():
    lib = ft.load()
    for name in ("ft_kv8_store", "ft_kv8_load", "ft_kv8_attention"):
        assert getattr(lib, name)(None, None) == ft.FT_E_ARG
    with pytest.raises(TypeError):
        ft.make_kv8_store_args(no_such_field=1)
    ft.ft_kv8_store(store(max_tokens=0))
    ft.ft_kv8_store(store(num_reqs=0))
    ft.ft_kv8_load(load(T=0))
    ft.ft_kv8_attention(attn(max_tokens=0))
    ft.ft_kv8_attention(attn(num_reqs=0))
    assert lib.ft_kv8_attention_workspace(None, None) == ft.FT_E_ARG


def test_workspace_follows_the_head_size_alone():
    size = lambda **kw: ft.ft_kv8_attention_workspace(attn(workspace=0, workspace_bytes=0, **kw))
    n = size()
    for kw in (dict(max_tokens=1), dict(max_tokens=100000), dict(max_new=1), dict(num_reqs=5000), dict(q_heads=256),
               dict(mask=PTR, mask_words=4), dict(dtype=ft.FT_DTYPE_F16), dict(cache_kw=dict(num_pages=100000)),
               dict(cache_kw=dict(page_size=64)), dict(cache_kw=dict(kv_heads=1))):
        assert size(**kw) == n, kw
    assert n % 16 == 0 and n // 2 <= size(cache_kw=dict(head_dim=64)) < n


def struct_layout(names):
    """Sizes and offsets as C lays out the header's structures, and as the binding does."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "ft_moe.h"\nint main(void) {\n'
    want = []
    for n in names:
        s = getattr(ft, n)
        src += f'  printf("%zu\\n", sizeof({n}));\n'
        want.append(ctypes.sizeof(s))
        for f in s._fields_:
            src += f'  printf("%zu\\n", offsetof({n}, {f[0]}));\n'
            want.append(getattr(s, f[0]).offset)
    src += "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "sizes.c"), os.path.join(d, "sizes")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    return got, want


def test_struct_sizes_match_the_header():
    got, want = struct_layout(["ft_kv8_cache", "ft_kv8_store_args", "ft_kv8_load_args", "ft_kv8_attn_args"])
    assert got == want


def test_every_declared_symbol_is_exported():
    """Names with a digit too."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "ft_moe.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(ft_[a-z0-9_]+)\s*\(", src))
    assert names == set(ft.EXPORTS) | set(ft.EXPORTS_KV8)
    for n in names:
        assert hasattr(ft.load(), n), n


def test_reference_codes():
    """The reference rounds to the nearest of all 253 numbers, ties to the even code."""
    codes = np.arange(256, dtype=np.uint8)
    fin = ~np.isnan(ref.VALUE)
    assert np.array_equal(ref.encode(ref.VALUE[fin]), codes[fin])
    assert ref.VALUE[126] == 448 and ref.VALUE[1] == 2.0 ** -9 and ref.VALUE[8] == 2.0 ** -6
    pos = ref.VALUE[:127]
    mid = (pos[:-1] + pos[1:]) / 2
    even = np.where(codes[:126] % 2 == 0, codes[:126], codes[1:127])
    assert np.array_equal(ref.encode(mid), even)
    assert np.array_equal(ref.encode(np.nextafter(mid, 0)), codes[:126])
    assert np.array_equal(ref.encode(np.nextafter(mid, 1000)), codes[1:127])
    assert ref.least_byte(0.0) == 0 and ref.least_byte(448.0) == 127 and ref.least_byte(448.5) == 128
