"""Calls that read what the call before them has just written, one after another
without a pause and in a graph: a step's plan, its rows stored where the plan says,
read back by the plan's slots and attended to."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_verify import ft  # noqa: E402, F401


def test_plan_store_load_attention(ft):
    B, n, HKV, HQ, D, P, width, rounds = 40, 5, 4, 8, 64, 16, 16, 24
    T, pages = B * n, 1024
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    at = lambda t: t.data_ptr()
    codes = torch.zeros((2, pages, P, HKV, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, pages, 1, HKV), dtype=torch.uint8, device="cuda")
    s = [codes.stride(1), codes.stride(2), codes.stride(3)]
    cache = ft.make_kv8_cache(k=at(codes[0]), v=at(codes[1]), k_scale=at(scales[0]), v_scale=at(scales[1]), num_pages=pages,
                              page_size=P, block_size=16, kv_heads=HKV, head_dim=D, k_page_stride=s[0], k_token_stride=s[1],
                              k_head_stride=s[2], v_page_stride=s[0], v_token_stride=s[1], v_head_stride=s[2])
    # every round has its inputs and outputs; the plan's, the scratch rows and the workspace are shared, as in a step's layers
    ctx = torch.zeros((rounds, B), **i32)
    for r in range(rounds):
        ctx[r] = torch.tensor(np.random.default_rng(r).integers(0, 2, B) * 16, **i32)
    new = torch.full((B,), n, **i32)
    free, count = torch.zeros((rounds, pages), **i32), torch.full((1,), pages, **i32)
    for r in range(rounds):
        free[r] = torch.randperm(pages, generator=g, device="cuda").int()
    table, q_start, slots = torch.zeros((B, width), **i32), torch.zeros(B + 1, **i32), torch.zeros(T, dtype=torch.int64, device="cuda")
    positions, left, status = torch.zeros(T, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    q = torch.randn((T, HQ, D), generator=g, device="cuda").bfloat16()
    # whole numbers up to 15 are exact in e4m3 at any of its scales
    kv = torch.randint(-15, 16, (rounds, 2, T, HKV, D), generator=g, device="cuda").bfloat16()
    back = torch.zeros_like(kv)
    out = torch.zeros((rounds, T, HQ, D), dtype=torch.bfloat16, device="cuda")
    args = ft.make_kv8_attn_args(
        q=at(q), q_start=at(q_start), ctx_len=at(ctx), block_table=at(table), status=at(status), q_stride=HQ * D,
        out_stride=HQ * D, dtype=ft.FT_DTYPE_BF16, max_tokens=T, max_new=n, num_reqs=B, q_heads=HQ, table_width=width,
        scale=0.01, cache=cache)
    ws = torch.zeros(ft.ft_kv8_attention_workspace(args), dtype=torch.uint8, device="cuda")
    args.workspace, args.workspace_bytes = at(ws), ws.numel()

    def everything(pause):
        st = torch.cuda.current_stream().cuda_stream
        for r in range(rounds):
            calls = [
                lambda: ft.ft_kv_plan(ft.make_plan_args(
                    ctx_len=at(ctx[r]), new_len=at(new), free_pages=at(free[r]), free_count=at(count), block_table=at(table),
                    q_start=at(q_start), slots=at(slots), positions=at(positions), free_left=at(left), status=at(status),
                    num_reqs=B, page_size=P, table_width=width, max_tokens=T), st),
                lambda: ft.ft_kv8_store(ft.make_kv8_store_args(
                    k=at(kv[r, 0]), v=at(kv[r, 1]), q_start=at(q_start), ctx_len=at(ctx[r]), block_table=at(table),
                    status=at(status), k_stride=HKV * D, v_stride=HKV * D, dtype=ft.FT_DTYPE_BF16, max_tokens=T, num_reqs=B,
                    table_width=width, cache=cache), st),
                lambda: ft.ft_kv8_load(ft.make_kv8_load_args(
                    k=at(back[r, 0]), v=at(back[r, 1]), slots=at(slots), status=at(status), k_stride=HKV * D,
                    v_stride=HKV * D, dtype=ft.FT_DTYPE_BF16, T=T, cache=cache), st),
                lambda: attend(r, st)]
            for call in calls:
                call()
                if pause:
                    torch.cuda.synchronize()

    def attend(r, st):
        args.ctx_len, args.out = at(ctx[r]), at(out[r])
        args.max_new = n * (r % 2)  # (the kernel of few rows, that of many)
        ft.ft_kv8_attention(args, st)

    everything(True)
    want = out.clone()
    assert torch.equal(back, kv) and status.item() == 0 and bool(torch.isfinite(want.float()).all())
    for mode in ("eager", "graph"):
        graph = torch.cuda.CUDAGraph()
        if mode == "graph":
            with torch.cuda.graph(graph):
                everything(False)
        for _ in range(5):
            for t in (codes, scales, back, out):
                t.zero_()
            table.zero_()
            graph.replay() if mode == "graph" else everything(False)
            torch.cuda.synchronize()
            assert torch.equal(back, kv) and torch.equal(out, want) and status.item() == 0
