"""The student's policy loss: temperatures other than 1, the loss that is printed."""

import importlib.util
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("student_training_step", os.path.join(ROOT, "examples", "student_training_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("temperature", [0.8, 1.0, 2.0])
def test_an_unmoved_policy_has_a_ratio_of_one(example, temperature):
    """Its loss is -A, without a KL term: log_probs are those that the loss compares with."""
    with example.ns.Handle() as h:
        s = example.Student(h.value, hidden=256, intermediate=128, experts=8, top_k=2, vocab=1003, seed=4)
        g = torch.Generator("cuda").manual_seed(11)
        x = torch.randn(40, 256, generator=g, device="cuda").bfloat16()
        actions = torch.randint(0, 1003, (40,), generator=g, device="cuda", dtype=torch.int32)
        adv = torch.randn(40, generator=g, device="cuda")
        old = s.log_probs(x, actions, temperature=temperature)
        loss, _ = s.policy(x, actions, adv, old, old, temperature=temperature, kl_coef=0.1)
        # Loss alone and loss with gradient may add up a row in another order: either log
        # probability is within 300 half steps of FP32 (tests/loss_reference.py: 141 of the
        # sum, 6 of each of the numbers around 7 in it), and the ratio within both.
        np.testing.assert_allclose(loss.cpu().numpy(), -adv.cpu().numpy(), rtol=2.0**-14)
        example.ns.muon_last_device_error(h.value)


def test_the_printed_loss_is_that_of_the_tokens_that_count(example, monkeypatch, capsys):
    """Of what is trained: the mask's tokens are not zeros among the others."""
    seen = []
    policy = example.Student.policy

    def spy(self, x, actions, adv, old, ref, mask=None, **options):
        loss, grad = policy(self, x, actions, adv, old, ref, mask, **options)
        seen.append(float(loss[mask != 0].double().mean()))
        return loss, grad

    monkeypatch.setattr(example.Student, "policy", spy)
    monkeypatch.setattr(sys, "argv", ["student_training_step.py", "--loss", "policy", "--hidden", "128", "--intermediate", "64",
                                      "--experts", "4", "--top-k", "2", "--vocab", "777", "--tokens", "33", "--steps", "2"])
    example.main()
    printed = [float(line.split("loss")[1]) for line in capsys.readouterr().out.splitlines() if "loss" in line]
    # Five decimals are printed; 25 values of about 1 in FP32, whose weights are rounded too.
    assert len(printed) == len(seen) == 2 and min(abs(s) for s in seen) > 1e-3
    assert all(abs(a - b) <= 0.5e-5 + 2.0**-19 for a, b in zip(printed, seen))
