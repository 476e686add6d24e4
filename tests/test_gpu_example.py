"""The example that runs the rollout attention, the policy loss, the adapter's backward and AdamW together learns: the
reward (the share of even tokens) starts at one half, within 0.5 / sqrt(128 x 12) = 0.013 a standard deviation, and after
ten steps lies ten of them above."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_grpo_example_learns():
    import grpo_step
    rewards = grpo_step.train(steps=12, log=lambda *_: None)
    assert abs(rewards[0] - 0.5) < 5 * 0.013
    assert min(rewards[-2:]) > 0.5 + 10 * 0.013


def test_grpo_example_repeats():
    """Two runs from one seed: the same rewards (no kernel's result depends on the order of its blocks)."""
    import grpo_step
    assert grpo_step.train(steps=3, log=lambda *_: None) == grpo_step.train(steps=3, log=lambda *_: None)
