"""examples/delta_recall.py: the dense operators together, trained and then answering token by token."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def recall():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_recall.py")
    spec = importlib.util.spec_from_file_location("delta_recall", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trains_and_answers(gpu, recall):
    """The loss falls below a quarter of its start (log of 16 values), and single steps from the states that the pairs left
    give the whole sequence's logits: float32 throughout, two layers of 2e-5 each at most, ten times that for the products
    around them."""
    model, losses = recall.train(gpu, 150)
    assert losses[-1] < 0.25 * losses[0]
    tokens, before, _ = (t.to(gpu) for t in recall.batch(32, 8, 15, torch.Generator().manual_seed(2)))
    with torch.no_grad():
        whole = model(tokens, before, model.states(32, gpu), recall.train_form)[:, -15:]
    steps = recall.answer(model, tokens, before, 15)
    assert (steps - whole).norm() <= 4e-4 * whole.norm()


def test_gradients_match_plain_rule(gpu, recall):
    """One training step's gradients against the same model over the rule written out with torch (float32, differentiated
    by torch): both carry float32 sums, so 1e-3 of each gradient's norm."""
    torch.manual_seed(3)
    model = recall.Model().to(gpu)
    tokens, before, answers = (t.to(gpu) for t in recall.batch(4, 4, 3, torch.Generator().manual_seed(3)))

    def plain(state, k, v, beta, log_decay, q):
        n, scale = v.shape[2] // k.shape[2], k.shape[-1] ** -0.5
        k, q = (t.repeat_interleave(n, 2) for t in (k, q))
        S, outs = state, []
        for t in range(k.shape[1]):
            S = log_decay[:, t].exp()[..., None, None] * S
            u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(-2))
            S = S + k[:, t, :, :, None] * u[:, :, None]
            outs.append(scale * (q[:, t, :, :, None] * S).sum(-2))
        return torch.stack(outs, 1)

    grads = []
    for form in (recall.train_form, plain):
        logits = model(tokens, before, model.states(4, gpu), form)[:, -3:]
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), answers.flatten())
        grads.append(torch.autograd.grad(loss, list(model.parameters())))
    for (name, _), a, b in zip(model.named_parameters(), *grads):
        assert (a - b).norm() <= 1e-3 * b.norm() + 1e-8, name
