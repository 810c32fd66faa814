"""Argument checks of ft_verify_drafts (on the host, no GPU)."""
import pytest

import expert_cache_host_gb300 as ft
from expert_cache_host_gb300 import build as ftbuild
from test_kv8_abi import refused, struct_layout

PTR = 1 << 20  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    ftbuild.build()
    return ft.load()


def verify(**kw):
    a = dict(probs=PTR, draft_probs=PTR, tokens=PTR, parents=PTR, accept_u=PTR, draw_u=PTR, q_start=PTR, accepted=PTR,
             n_accepted=PTR, next_token=PTR, probs_stride=100, draft_stride=100, dtype=ft.FT_DTYPE_F32, max_tokens=8,
             num_reqs=2, V=100)
    a.update(kw)
    return ft.make_verify_args(**a)


@pytest.mark.parametrize("kw", [
    dict(dtype=ft.FT_DTYPE_MXFP4), dict(max_tokens=-1), dict(num_reqs=-1), dict(V=0), dict(V=(1 << 30) + 1), dict(probs=0),
    dict(tokens=0), dict(accept_u=0), dict(draw_u=0), dict(q_start=0), dict(accepted=0), dict(n_accepted=0),
    dict(next_token=0), dict(probs=PTR + 2), dict(draft_probs=PTR + 1), dict(dtype=ft.FT_DTYPE_F16, probs=PTR + 1),
    dict(probs_stride=-1), dict(draft_stride=-4)], ids=str)
def test_refusals(kw):
    refused(ft.ft_verify_drafts, verify(**kw))


def test_null_args_unknown_fields_and_no_requests():
    assert ft.load().ft_verify_drafts(None, None) == ft.FT_E_ARG
    with pytest.raises(TypeError):
        ft.make_verify_args(no_such_field=1)
    ft.ft_verify_drafts(verify(num_reqs=0))


def test_struct_size_matches_the_header():
    got, want = struct_layout(["ft_verify_args"])
    assert got == want
