"""The decoding example runs the whole step; its tokens, lengths and counts fit together."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("greedy", [False, True])
def test_verify_step_example(greedy):
    import torch

    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import verify_step
    finally:
        sys.path.pop(0)
    steps, batch, prompt, vocab = 12, 4, 96, 200
    tokens, lens, accepted = verify_step.decode(steps=steps, greedy=greedy, batch=batch,
                                                vocab=vocab, prompt=prompt)
    torch.cuda.synchronize()
    assert accepted.shape == (steps, batch) and int(accepted.min()) >= 0
    # every step emits its accepted tokens and one more, the prompt one
    assert lens.tolist() == (prompt + 1 + steps + accepted.sum(0)).tolist()
    for b in range(batch):
        row = tokens[b, :int(lens[b])]
        assert int(row.min()) >= 0 and int(row.max()) < vocab
        assert not tokens[b, int(lens[b]):].any()
    again = verify_step.decode(steps=steps, greedy=greedy, batch=batch, vocab=vocab,
                               prompt=prompt)
    assert torch.equal(again[0], tokens) and torch.equal(again[2], accepted)
