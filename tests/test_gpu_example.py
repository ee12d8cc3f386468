"""The example of a whole round: replayed from a graph it gives the eager rounds' tokens, and the
drafts that it accepts follow the drafter."""
import os
import sys

import pytest
import torch

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("prompt", [1, 2, 63, 64, 65, 700])
def test_rounds_from_a_graph_equal_eager_ones(prompt):
    need_gpu()
    import speculative_round as s
    model = s.Model()
    tokens = torch.randint(0, s.VOCAB, (prompt,), generator=torch.Generator().manual_seed(prompt)).int().cuda()
    log(f"example, prompt of {prompt}")
    eager, accepted, _ = s.decode(model, tokens, 12, False)
    replayed, again, _ = s.decode(model, tokens, 12, True)
    assert eager == replayed and accepted == again
    assert len(eager) == sum(accepted) + 12 and sum(accepted) > 0
    # an accepted draft is the one that follows the token before it
    follows, at = model.follows.tolist(), [int(tokens[-1])] + eager
    i = 0
    for n in accepted:
        for _ in range(n):
            assert at[i + 1] == follows[at[i]]
            i += 1
        i += 1
