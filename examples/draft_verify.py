"""A small MoE decoder that verifies trees of drafted tokens in one step.

Every step runs the library end to end: ft_kv_plan lays the step's tokens out
in the paged cache, each layer runs ft_qk_norm_rope, ft_tree_attention and the
expert cache (ft_cache_step, ft_moe_forward), and ft_token_logprobs scores the
logits.  The drafter looks the last two tokens up in what the request has said
so far; the tree is a few such continuations.  The longest drafted path the
model agrees with (its most likely token at every node) is kept, its keys and
values are moved together, and pages that only dropped tokens used go back.

Weights are random (seeded), projections are plain torch products.

    python examples/draft_verify.py [--steps N] [--seed S]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import expert_cache_host_gb300 as ft  # noqa: E402
import ftsynth  # noqa: E402

L, D_MODEL, E, TOP_K, INTER = 2, 256, 16, 2, 128
HQ, HKV, HEAD, PAGE, VOCAB, MAX_POS = 8, 2, 64, 16, 1024, 4096
T_MAX, WORDS = 128, 1


def ptr(t):
    return 0 if t is None else t.data_ptr()


class Model:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s, std=0.06: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()
        self.embed = w(VOCAB, D_MODEL, std=1.0)
        self.qkv = [w(D_MODEL, (HQ + 2 * HKV) * HEAD) for _ in range(L)]
        self.o = [w(HQ * HEAD, D_MODEL) for _ in range(L)]
        self.head = w(D_MODEL, VOCAB)
        self.q_norm = [1 + w(HEAD) for _ in range(L)]
        self.k_norm = [1 + w(HEAD) for _ in range(L)]
        self.router = [w(D_MODEL, E).float() for _ in range(L)]
        half = HEAD // 2
        angle = torch.arange(MAX_POS, device="cuda")[:, None] * 10000.0 ** (-torch.arange(half, device="cuda") / half)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        pool = ftsynth.make_pool(seed, L, E, D_MODEL, INTER, 0, 0.06)
        self.pool = ft.HostPool(pool.nbytes)
        self.pool.array[:] = pool.view(np.uint8).reshape(-1)
        cfg = ft.make_config(num_layers=L, num_experts=E, top_k=TOP_K, hidden=D_MODEL, inter=INTER, num_slots=2 * E,
                             k_max=E, t_max=T_MAX)
        self.ctx = ft.ft_moe_init(cfg, self.pool.ptr, self.pool.nbytes)

    def close(self):
        ft.ft_moe_destroy(self.ctx)
        self.pool.free()


class Engine:
    """Requests over one paged cache.  Host lists hold what was said; the device holds the block table."""

    def __init__(self, model, prompts, pages=256):
        self.m, self.B = model, len(prompts)
        self.said = [list(p) for p in prompts]  # the last token of each is not in the cache yet
        self.ctx = [0] * self.B
        self.k, self.v = (torch.zeros((L, pages, PAGE, HKV, HEAD), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.full((self.B, MAX_POS // PAGE), -1, dtype=torch.int32, device="cuda")
        self.free = list(range(pages))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = None

    def plan(self, args, mask, st):
        """Lays the step out; `mask` is the tensor behind args.mask."""
        ft.ft_kv_plan(args, st)

    def step(self, tokens, parents, given=None):
        """One pass over each request's new tokens (parents: None where they follow one another).  Returns the plan's
        slots and, for every row, its most likely token, that token's log probability, and the log probability of
        given[row] (NaN where that is -1; None without `given`)."""
        new = [len(t) for t in tokens]
        T, st = sum(new), torch.cuda.current_stream().cuda_stream
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        flat, ctx_len, new_len = i32(sum(tokens, [])), i32(self.ctx), i32(new)
        tree = parents is not None
        par = i32(sum(parents, [])) if tree else None
        stack, count, left = i32(self.free), i32([len(self.free)]), i32([0])
        q_start, positions = i32([0] * (self.B + 1)), i32([0] * T)
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        mask = torch.zeros((T, WORDS), dtype=torch.int32, device="cuda") if tree else None
        self.plan(ft.make_plan_args(
            ctx_len=ptr(ctx_len), new_len=ptr(new_len), parents=ptr(par), free_pages=ptr(stack), free_count=ptr(count),
            block_table=ptr(self.table), q_start=ptr(q_start), slots=ptr(slots), positions=ptr(positions), mask=ptr(mask),
            free_left=ptr(left), status=ptr(self.status), num_reqs=self.B, page_size=PAGE,
            table_width=self.table.shape[1], max_tokens=T, mask_words=WORDS if tree else 0), mask, st)
        x = self.m.embed[flat.long()].float()
        q = torch.empty((T, HQ * HEAD), dtype=torch.bfloat16, device="cuda")
        att = torch.empty_like(q)
        y = torch.empty((T, D_MODEL), dtype=torch.float32, device="cuda")
        for l in range(L):
            h = norm(x)
            qkv = h @ self.m.qkv[l]
            cache = ft.make_kv_cache(
                k=ptr(self.k[l]), v=ptr(self.v[l]), dtype=ft.FT_DTYPE_BF16, num_pages=self.k.shape[1], page_size=PAGE,
                kv_heads=HKV, head_dim=HEAD, k_page_stride=PAGE * HKV * HEAD, k_token_stride=HKV * HEAD,
                k_head_stride=HEAD, v_page_stride=PAGE * HKV * HEAD, v_token_stride=HKV * HEAD, v_head_stride=HEAD)
            ld = qkv.stride(0)
            ft.ft_qk_norm_rope(ft.make_qk_args(
                q=ptr(qkv), k=ptr(qkv) + 2 * HQ * HEAD, v=ptr(qkv) + 2 * (HQ + HKV) * HEAD, q_weight=ptr(self.m.q_norm[l]),
                k_weight=ptr(self.m.k_norm[l]), cos_sin=ptr(self.m.cos_sin), positions=ptr(positions), slots=ptr(slots),
                q_out=ptr(q), status=ptr(self.status), q_stride=ld, k_stride=ld, v_stride=ld, q_out_stride=HQ * HEAD, T=T,
                q_heads=HQ, rot_dim=HEAD, max_pos=MAX_POS, interleaved=0, eps=1e-6, cache=cache), st)
            args = ft.make_attn_args(
                q=ptr(q), out=ptr(att), q_start=ptr(q_start), ctx_len=ptr(ctx_len), block_table=ptr(self.table),
                mask=ptr(mask), status=ptr(self.status), q_stride=HQ * HEAD, out_stride=HQ * HEAD, max_tokens=T,
                num_reqs=self.B, q_heads=HQ, table_width=self.table.shape[1], mask_words=WORDS if tree else 0,
                scale=HEAD ** -0.5, cache=cache)
            if self.workspace is None:
                self.workspace = torch.empty(ft.ft_tree_attention_workspace(args), dtype=torch.uint8, device="cuda")
            args.workspace, args.workspace_bytes = ptr(self.workspace), self.workspace.numel()
            ft.ft_tree_attention(args, st)
            x = x + (att @ self.m.o[l]).float()
            h = norm(x)
            logits = (h.float() @ self.m.router[l]).contiguous()
            ft.ft_cache_step(self.m.ctx, l, ptr(logits), T, st)
            ft.ft_moe_forward(self.m.ctx, l, ft.FT_DECODE_CACHED, 0, ptr(h), T, 0, ptr(y), st)
            x = x + y
        logits = norm(x) @ self.m.head
        best = torch.empty((T, 1), dtype=torch.int32, device="cuda")
        best_lp = torch.empty((T, 1), dtype=torch.float32, device="cuda")
        entropy = torch.empty(T, dtype=torch.float32, device="cuda")
        asked = None if given is None else i32(given)
        given_lp = None if given is None else torch.empty(T, dtype=torch.float32, device="cuda")
        ft.ft_token_logprobs(ft.make_logprob_args(
            logits=ptr(logits), tokens=ptr(asked), logprob=ptr(given_lp), entropy=ptr(entropy), top_ids=ptr(best), top_logprobs=ptr(best_lp), status=ptr(self.status),
            row_stride=logits.stride(0), dtype=ft.FT_DTYPE_BF16, T=T, V=VOCAB, top_n=1), st)
        self.free = self.free[:int(left.item())]
        if int(self.status.item()) or ft.ft_get_status(self.m.ctx):
            raise RuntimeError(f"device status {int(self.status.item())}")
        return slots, best[:, 0].tolist(), best_lp[:, 0].tolist(), None if given is None else given_lp.tolist()

    def keep(self, b, slots, path, new):
        """Keep the new tokens `path` (indices, ascending) of request b: their keys and values move to the places
        right after the context; pages that only dropped tokens began go back to the stack."""
        src = slots[path]
        dst = slots[:len(path)]
        for c in (self.k, self.v):
            rows = c.view(L, -1, HKV, HEAD)
            rows[:, dst] = rows[:, src].clone()
        was, self.ctx[b] = self.ctx[b], self.ctx[b] + len(path)
        held = -(-self.ctx[b] // PAGE)
        self.free += reversed(self.table[b, held:max(held, -(-(was + new) // PAGE))].tolist())


def norm(x):
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).bfloat16()


def draft(said, branches=3, depth=4):
    """A tree of continuations: the last token, then up to `branches` distinct continuations of its latest
    occurrences, each up to `depth` tokens, sharing prefixes."""
    tokens, parents, children = [said[-1]], [-1], [{}]
    found = 0
    for i in range(len(said) - 2, 0, -1):
        if said[i - 1:i + 1] != said[-2:]:
            continue
        at = 0
        for t in said[i + 1:i + 1 + depth]:
            if t not in children[at]:
                if len(tokens) == 32 * WORDS:
                    break
                children[at][t] = len(tokens)
                tokens.append(t)
                parents.append(at)
                children.append({})
            at = children[at][t]
        found += 1
        if found == branches:
            break
    return tokens, parents


def generate(model, prompts, steps, drafting=True, forced=None, engine=Engine):
    """Greedy decoding.  Returns what each request said, the log probability of each generated token, the steps taken,
    and how many tokens were not the model's own choice.  forced: tokens to say instead of the model's own, one a step
    (to score a given continuation)."""
    eng = engine(model, prompts)
    lps = [[] for _ in prompts]
    # the prompt but its last token, then one step per iteration
    slots, _, _, _ = eng.step([p[:-1] for p in prompts], None)
    at = 0
    for b, p in enumerate(prompts):
        eng.keep(b, slots[at:at + len(p) - 1], list(range(len(p) - 1)), len(p) - 1)
        at += len(p) - 1
    taken = other = 0
    while taken < steps:
        taken += 1
        trees = [draft(s) if drafting and forced is None else ([s[-1]], [-1]) for s in eng.said]
        given = None
        if forced is not None:  # a row a request
            given = [f[len(s)] if len(s) < len(f) else -1 for f, s in zip(forced, eng.said)]
        slots, best, best_lp, given_lp = eng.step([t for t, _ in trees], [p for _, p in trees], given)
        at = 0
        for b, (tokens, parents) in enumerate(trees):
            path = [0]
            while True:  # follow the model's choice down the tree
                node = path[-1]
                told = given is not None and given[b] >= 0
                say = given[b] if told else best[at + node]
                other += say != best[at + node]
                eng.said[b].append(say)
                lps[b].append(given_lp[at + node] if told else best_lp[at + node])
                nxt = [i for i in range(node + 1, len(tokens)) if parents[i] == node and tokens[i] == say]
                if not nxt:
                    break
                path.append(nxt[0])
            eng.keep(b, slots[at:at + len(tokens)], path, len(tokens))
            at += len(tokens)
    return eng.said, lps, taken, other


def verify(model, prompts, steps, engine=Engine):
    """Drafted decoding, then what it said scored one token at a time.  Returns the tokens told, the steps, the largest
    difference of a token's log probability between the two, and how many of the tokens the second pass would not have
    chosen."""
    said, lps, steps, _ = generate(model, prompts, steps, engine=engine)
    longest = max(len(s) - len(p) for s, p in zip(said, prompts))
    _, one_lps, _, other = generate(model, prompts, longest, forced=said)
    told = sum(len(s) - len(p) for s, p in zip(said, prompts))
    far = max(abs(x - y) for a, b in zip(lps, one_lps) for x, y in zip(a, b))
    return told, steps, far, other


def make_prompts(seed):
    rng = np.random.default_rng(seed)
    motif = rng.integers(0, VOCAB, 6).tolist()
    return [motif * 3, rng.integers(0, VOCAB, 9).tolist() * 2, rng.integers(0, VOCAB, 21).tolist()]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    prompts = make_prompts(a.seed)
    model = Model(a.seed)
    try:
        told, steps, far, other = verify(model, prompts, a.steps)
    finally:
        model.close()
    print(f"{told} tokens in {steps} steps of {len(prompts)} requests: {told / steps / len(prompts):.2f} a request and step")
    print(f"largest difference of a token's log probability from one token at a time: {far:.4f} "
          f"({other} tokens not its choice)")
    return told, steps, far


if __name__ == "__main__":
    main()
