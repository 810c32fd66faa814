"""Drafted trees sampled as the model itself would, over a cache held in 8 bits.

The decoder of draft_verify.py with two things changed.  Keys and values live in
an 8-bit paged cache: a layer's ft_qk_norm_rope leaves the step's rows in a
16-bit scratch, ft_kv8_store quantises them into the cache and ft_kv8_attention
reads it.  And tokens are sampled: ft_verify_drafts accepts drafted tokens
against the model's probabilities by given random numbers and draws the token
that follows, so that what is said is distributed as without drafts.  The rows
of the accepted tokens are read back with ft_kv8_load and stored again right
after the context.

    python examples/draft_sample.py [--steps N] [--seed S] [--temperature T]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import draft_verify as dv  # noqa: E402
from draft_verify import HEAD, HKV, HQ, L, PAGE, VOCAB, ft, i32, ptr  # noqa: E402

BLOCK = 16  # tokens that share a scale


class Engine(dv.Engine):
    def make_cache(self, pages):
        self.pages = pages
        self.codes = torch.zeros((2, L, pages, PAGE, HKV, HEAD), dtype=torch.uint8, device="cuda")  # keys, values
        self.scales = torch.zeros((2, L, pages, PAGE // BLOCK, HKV), dtype=torch.uint8, device="cuda")

    def layer_cache(self, l):
        page = PAGE * HKV * HEAD
        return ft.make_kv8_cache(
            k=ptr(self.codes[0, l]), v=ptr(self.codes[1, l]), k_scale=ptr(self.scales[0, l]), v_scale=ptr(self.scales[1, l]),
            num_pages=self.pages, page_size=PAGE, block_size=BLOCK, kv_heads=HKV, head_dim=HEAD, k_page_stride=page,
            k_token_stride=HKV * HEAD, k_head_stride=HEAD, v_page_stride=page, v_token_stride=HKV * HEAD, v_head_stride=HEAD)

    def store(self, l, rows, q_start, ctx_len, st):
        """rows: keys and values [2, T, HKV * HEAD] of the requests' new tokens."""
        ft.ft_kv8_store(ft.make_kv8_store_args(
            k=ptr(rows[0]), v=ptr(rows[1]), q_start=ptr(q_start), ctx_len=ptr(ctx_len), block_table=ptr(self.table),
            status=ptr(self.status), k_stride=HKV * HEAD, v_stride=HKV * HEAD, dtype=ft.FT_DTYPE_BF16,
            max_tokens=rows.shape[1], num_reqs=self.B, table_width=self.table.shape[1], cache=self.layer_cache(l)), st)

    def attend(self, l, p, qkv, q, att):
        # a scratch in the shape of a 16-bit cache, the step's rows one after another
        pages = -(-p.T // PAGE)
        rows = torch.empty((2, pages * PAGE, HKV * HEAD), dtype=torch.bfloat16, device="cuda")
        page = PAGE * HKV * HEAD
        scratch = ft.make_kv_cache(k=ptr(rows[0]), v=ptr(rows[1]), dtype=ft.FT_DTYPE_BF16, num_pages=pages, page_size=PAGE,
                                   kv_heads=HKV, head_dim=HEAD, k_page_stride=page, k_token_stride=HKV * HEAD,
                                   k_head_stride=HEAD, v_page_stride=page, v_token_stride=HKV * HEAD, v_head_stride=HEAD)
        self.queries_and_keys(l, p, qkv, q, scratch, torch.arange(p.T, device="cuda"))
        self.store(l, rows[:, :p.T], p.q_start, p.ctx_len, p.st)
        args = ft.make_kv8_attn_args(
            q=ptr(q), out=ptr(att), q_start=ptr(p.q_start), ctx_len=ptr(p.ctx_len), block_table=ptr(self.table),
            mask=ptr(p.mask), status=ptr(self.status), q_stride=HQ * HEAD, out_stride=HQ * HEAD, dtype=ft.FT_DTYPE_BF16,
            max_tokens=p.T, max_new=p.longest, num_reqs=self.B, q_heads=HQ, table_width=self.table.shape[1],
            mask_words=p.words, scale=HEAD ** -0.5, cache=self.layer_cache(l))
        if self.workspace is None:
            self.workspace = torch.empty(ft.ft_kv8_attention_workspace(args), dtype=torch.uint8, device="cuda")
        args.workspace, args.workspace_bytes = ptr(self.workspace), self.workspace.numel()
        ft.ft_kv8_attention(args, p.st)

    def keep(self, slots, paths, new):
        """Keep of every request the new tokens paths[b] (indices among its rows, ascending): read back and stored again
        right after the context."""
        st = torch.cuda.current_stream().cuda_stream
        starts = [0]
        for p in paths:
            starts.append(starts[-1] + len(p))
        first = [sum(new[:b]) for b in range(self.B)]
        src = slots[[f + i for f, p in zip(first, paths) for i in p]].contiguous()
        q_start, ctx_len = i32(starts), i32(self.ctx)
        rows = torch.empty((2, starts[-1], HKV * HEAD), dtype=torch.bfloat16, device="cuda")
        for l in range(L):
            ft.ft_kv8_load(ft.make_kv8_load_args(
                k=ptr(rows[0]), v=ptr(rows[1]), slots=ptr(src), status=ptr(self.status), k_stride=HKV * HEAD,
                v_stride=HKV * HEAD, dtype=ft.FT_DTYPE_BF16, T=starts[-1], cache=self.layer_cache(l)), st)
            self.store(l, rows, q_start, ctx_len, st)
        for b, p in enumerate(paths):
            self.advance(b, len(p), new[b])

    def sample(self, tokens, parents, accept_u, draw_u, temperature):
        """One pass over each request's tree: for every request the rows it keeps and the token that follows."""
        p, logits = self.forward(tokens, parents)
        probs = torch.softmax(logits.float() / temperature, 1)
        accepted, count, following = i32([0] * p.T), i32([0] * self.B), i32([0] * self.B)
        ft.ft_verify_drafts(ft.make_verify_args(
            probs=ptr(probs), tokens=ptr(p.tokens), parents=ptr(p.parents), accept_u=ptr(accept_u), draw_u=ptr(draw_u),
            q_start=ptr(p.q_start), accepted=ptr(accepted), n_accepted=ptr(count), next_token=ptr(following),
            status=ptr(self.status), probs_stride=probs.stride(0), dtype=ft.FT_DTYPE_F32, max_tokens=p.T, num_reqs=self.B,
            V=VOCAB), p.st)
        self.check()
        accepted, paths, at = accepted.tolist(), [], 0
        for t, n in zip(tokens, count.tolist()):
            paths.append([0] + accepted[at:at + n])
            at += len(t)
        return p.slots, paths, following.tolist()


def generate(model, prompts, steps, seed=0, temperature=0.7, engine=Engine):
    """Sampled decoding with drafts.  Returns what each request said and the engine."""
    eng = engine(model, prompts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    random = lambda n: torch.rand(n, device="cuda", generator=g)
    new = [len(p) - 1 for p in prompts]
    p, _ = eng.forward([p[:-1] for p in prompts], None)
    eng.check()
    for b, n in enumerate(new):
        eng.advance(b, n, n)
    for _ in range(steps):
        trees = [dv.draft(s) for s in eng.said]
        tokens, parents = [t for t, _ in trees], [p for _, p in trees]
        new = [len(t) for t in tokens]
        slots, paths, following = eng.sample(tokens, parents, random(sum(new)), random(len(prompts)), temperature)
        eng.keep(slots, paths, new)
        for b, path in enumerate(paths):
            eng.said[b] += [tokens[b][i] for i in path[1:]] + [following[b]]
    return eng.said, eng


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--temperature", type=float, default=0.7)
    a = ap.parse_args(argv)
    prompts = dv.make_prompts(a.seed)
    model = dv.Model(a.seed)
    try:
        said, _ = generate(model, prompts, a.steps, a.seed, a.temperature)
    finally:
        model.close()
    told = sum(len(s) - len(p) for s, p in zip(said, prompts))
    print(f"{told} tokens in {a.steps} steps of {len(prompts)} requests: {told / a.steps / len(prompts):.2f} a request and step")
    return told, a.steps


if __name__ == "__main__":
    main()
