"""The gated-delta example: it learns, and serving it token by token gives the
training pass's logits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


def test_example_trains_and_serves():
    import gated_delta

    torch.manual_seed(0)
    model = gated_delta.Model(128).cuda()
    # untrained: the served logits are the full pass's up to bf16 roundings of
    # two layers' outs, and of q, k, v where a product's shape changes them
    # (2^-8 of a row's size each, a handful of them in a chain)
    diff, _ = gated_delta.serve(model)
    assert diff <= 16 * 2.0 ** -8
    # 64 values: a model that recalls nothing stays at ln 64 = 4.16 and answers
    # one in 64
    losses = gated_delta.train(model, 300, log=None)
    assert all(torch.isfinite(torch.tensor(losses)))
    assert max(losses[-10:]) < 2.08
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all())
               for p in model.parameters())
    diff, right = gated_delta.serve(model)
    assert diff <= 16 * 2.0 ** -8 and right > 0.5


def test_slots_outside_the_call_keep_their_states():
    import gated_delta

    torch.manual_seed(1)
    model = gated_delta.Model(128).cuda()
    states = model.new_states(5)
    for s in states:
        s.normal_()
    before = [s.clone() for s in states]
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    two = torch.tensor([5, 9], device="cuda")
    model.step(two, two, torch.tensor([7, 2], device="cuda"), states, slots)
    for s, b in zip(states, before):
        assert torch.equal(s[[0, 2, 4]], b[[0, 2, 4]])
        assert not torch.equal(s[1], b[1]) and not torch.equal(s[3], b[3])
