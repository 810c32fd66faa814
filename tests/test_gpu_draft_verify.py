"""The drafted-token example end to end: attention side and expert cache in one step.

Verifying a tree gives every kept token the log probability it has when decoded
one at a time.  The two differ by bf16 roundings of the activations in other
orders (2^-8 relative each, tens of them on logits of a few units): 0.25.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_drafted_trees_score_like_single_tokens():
    from expert_cache_host_gb300 import build as ftbuild
    ftbuild.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import draft_verify
    told, steps, far = draft_verify.main(["--steps", "40"])
    assert told >= 3 * steps  # every request says at least one token a step
    assert far < 0.25


# What the two passes may differ by: about 14 roundings to bf16 (2^-8 of the number at most, uniform: a root mean
# square of 2^-8 / sqrt 3 or less) on the way through two layers, in either pass, all of them different, make
# sqrt(28) 2^-8 / sqrt 3 = 0.012 of a logit of size 1; 4 of that for the largest of some hundreds, and the two logits'
# own rounding, a spacing of 2^-5 below 8.
APART = 4 * 0.012 + 2.0 ** -5


@pytest.fixture(scope="module")
def example():
    from expert_cache_host_gb300 import build as ftbuild
    ftbuild.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import draft_verify
    model = draft_verify.Model(0)
    yield draft_verify, model, draft_verify.make_prompts(0)
    model.close()


def test_drafted_tokens_are_accepted_and_score_as_given_one_at_a_time(example):
    """The tokens that the trees' pass kept, given to a pass of one token a step: the same log probability each."""
    dv, model, prompts = example
    told, steps, far, other = dv.verify(model, prompts, 40)
    assert told > 3 * steps  # more than a token a request and step: drafts were accepted
    assert far <= APART
    assert other <= told // 50  # ties and near ties of bf16 logits only


def test_a_wrong_mask_bit_shows(example):
    """The same with one bit wrong, the first token's in every other row's mask: beyond what roundings do."""
    dv, model, prompts = example

    class Wrong(dv.Engine):
        def plan(self, args, mask, st):
            super().plan(args, mask, st)
            if mask is not None:
                mask[((mask & 1) == 1) & (mask != 1)] -= 1

    assert dv.verify(model, prompts, 40, engine=Wrong)[2] > APART


def test_given_tokens_are_scored(example):
    """A continuation the model would not choose gets its own log probabilities, not those of the model's choice."""
    dv, model, prompts = example
    said, lps, _, _ = dv.generate(model, prompts, 6, drafting=False)
    forced = [p + [(t + 1) % dv.VOCAB for t in s[len(p):len(p) + 6]] for p, s in zip(prompts, said)]
    got, forced_lps, _, other = dv.generate(model, prompts, 6, forced=forced)
    assert got == forced and other >= 6
    for a, b in zip(lps, forced_lps):
        assert b[0] < a[0] - 0.5  # the same row of logits, another token
