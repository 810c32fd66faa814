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
