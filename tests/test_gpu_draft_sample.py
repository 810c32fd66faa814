"""The 8-bit cache's operators and the verification of drafts run together."""
import os
import sys

import numpy as np
import pytest

import kv8_reference as ref
from test_gpu_verify import reference as verify_reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    from expert_cache_host_gb300 import build as ftbuild
    ftbuild.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import draft_sample
    model = draft_sample.dv.Model(0)
    yield draft_sample, model, draft_sample.dv.make_prompts(0)
    model.close()


def test_sampled_trees_run(example):
    ds, model, prompts = example
    said, eng = ds.generate(model, prompts, 20)
    assert all(len(s) >= len(p) + 20 for s, p in zip(said, prompts))  # at least one token a request and step
    assert all(0 <= t < ds.VOCAB for s in said for t in s)
    assert [len(s) - 1 for s in said] == eng.ctx  # the last token of each is not in the cache yet
    again, _ = ds.generate(model, prompts, 20)
    assert again == said
    # pages: those the contexts need, and no page twice
    held = [-(-c // ds.PAGE) for c in eng.ctx]
    used = [p for b, h in enumerate(held) for p in eng.table[b, :h].tolist()]
    assert sorted(used + eng.free) == list(range(eng.pages))


class Checked:
    """An engine whose every step is followed by plain implementations: the cache block by block, attention in 64 bits,
    the verification, and the tokens moved together."""

    @staticmethod
    def make(ds):
        class Engine(ds.Engine):
            def make_cache(self, pages):
                super().make_cache(pages)
                self.mirror = [ref.Cache([c.cpu().numpy() for c in self.codes[:, l]], [s.cpu().numpy() for s in self.scales[:, l]],
                                         ds.BLOCK) for l in range(ds.L)]
                self.checked = 0

            def store(self, l, rows, q_start, ctx_len, st):
                super().store(l, rows, q_start, ctx_len, st)
                torch.cuda.synchronize()
                start = q_start.tolist()
                new = [b - a for a, b in zip(start, start[1:])]
                x = rows.double().cpu().numpy().reshape(2, -1, ds.HKV, ds.HEAD)
                assert not self.mirror[l].store(list(x), "bf16", ctx_len.tolist(), new, self.table.cpu().numpy())
                for kv in range(2):
                    assert np.array_equal(self.codes[kv, l].cpu().numpy(), self.mirror[l].codes[kv])
                    assert np.array_equal(self.scales[kv, l].cpu().numpy(), self.mirror[l].scale[kv])

            def attend(self, l, p, qkv, q, att):
                super().attend(l, p, qkv, q, att)
                torch.cuda.synchronize()
                start, ctx, table = p.q_start.tolist(), p.ctx_len.tolist(), self.table.cpu().numpy()
                k, v = (self.mirror[l].values(kv) for kv in range(2))
                qq = q.double().cpu().numpy().reshape(p.T, ds.HQ, ds.HEAD)
                got = att.double().cpu().numpy().reshape(p.T, ds.HQ, ds.HEAD)
                masks = None if p.mask is None else p.mask.cpu().numpy().view(np.uint32)
                for b, c in enumerate(ctx):
                    n = start[b + 1] - start[b]
                    at = np.arange(c + n)
                    page, row = table[b, at // ds.PAGE], at % ds.PAGE
                    for i in range(n):
                        seen = [j <= i if masks is None else bool(masks[start[b] + i, 0] >> j & 1) for j in range(n)]
                        keys = np.concatenate([np.arange(c), c + np.nonzero(seen)[0]]).astype(int)
                        for h in range(ds.HQ):
                            kk, vv = (x[page[keys], row[keys], h * ds.HKV // ds.HQ] for x in (k, v))
                            s = kk @ qq[start[b] + i, h] * ds.HEAD ** -0.5
                            w = np.exp(s - s.max())
                            w /= w.sum()
                            out, mag = w @ vv, w @ np.abs(vv)
                            # probabilities and output rounded to bf16 (2^-8 each), fp32 steps
                            tol = 2.0 ** -8 * (mag + np.abs(out)) + 2.0 ** -16 * mag + 1e-30
                            assert (np.abs(got[start[b] + i, h] - out) <= tol).all()
                            self.checked += 1

            def sample(self, tokens, parents, accept_u, draw_u, temperature):
                seen = {}
                forward = self.forward

                def keep_logits(*a):
                    seen["p"], seen["logits"] = forward(*a)
                    return seen["p"], seen["logits"]
                self.forward = keep_logits
                slots, paths, following = super().sample(tokens, parents, accept_u, draw_u, temperature)
                self.forward = forward
                probs = torch.softmax(seen["logits"].float() / temperature, 1).double().cpu().numpy()
                new = [len(t) for t in tokens]
                start = np.concatenate([[0], np.cumsum(new)])
                accepted, counts, want = verify_reference(probs, None, sum(tokens, []), sum(parents, []),
                                                          accept_u.double().cpu().numpy(), draw_u.double().cpu().numpy(), start)
                assert want.tolist() == following
                assert [[0] + accepted[s:s + c].tolist() for s, c in zip(start, counts)] == paths
                return slots, paths, following
        return Engine


@pytest.mark.parametrize("eager", [False, True])
def test_every_step_against_plain_implementations(example, eager):
    """Plan, norms, store, attention over the 8-bit cache, experts, verification, and the kept tokens' way back.
    eager: every second step accepts whatever is drafted (its random numbers are 0), so that rows move."""
    ds, model, prompts = example

    class Engine(Checked.make(ds)):
        step = 0

        def sample(self, tokens, parents, accept_u, draw_u, temperature):
            self.step += 1
            if eager and self.step % 2:
                accept_u = torch.zeros_like(accept_u)
            return super().sample(tokens, parents, accept_u, draw_u, temperature)

    said, eng = ds.generate(model, [prompts[0], prompts[1]], 8, seed=3, engine=Engine)
    assert eng.checked > 8 * 2 * ds.L * ds.HQ
    told = sum(len(s) for s in said) - len(prompts[0]) - len(prompts[1])
    assert told > 2 * 8 if eager else told >= 2 * 8


def test_a_wrong_mask_bit_shows(example):
    """The same with one bit wrong, the first token's in every other row's mask, as the attention gets it."""
    ds, model, prompts = example

    class Wrong(Checked.make(ds)):
        def attend(self, l, p, qkv, q, att):
            right = p.mask
            if right is not None:
                p.mask = torch.where(((right & 1) == 1) & (right != 1), right - 1, right)
            ds.Engine.attend(self, l, p, qkv, q, att)
            p.mask = right
            told = att.clone()
            super().attend(l, p, qkv, q, att)
            if right is not None and bool((right != 1).any()):
                self.apart = max(getattr(self, "apart", 0.0), float((told.float() - att.float()).abs().max()))

    _, eng = ds.generate(model, [prompts[0]], 3, seed=3, engine=Wrong)
    assert eng.apart > 2.0 ** -6
