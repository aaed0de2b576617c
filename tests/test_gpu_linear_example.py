"""examples/delta_recall.py with linear attention layers: linear attention and group norm together, trained and then answering
token by token."""

import pytest
import torch

from tests.test_gpu_delta_example import recall  # noqa: F401

pytestmark = pytest.mark.gpu


def test_trains_and_answers(gpu, recall):
    """Training runs, and single steps from the states that the pairs left give the whole sequence's logits: float32
    throughout, two layers of 64 * 2^-23 of their terms each, a norm of each head's readings after either (which may make
    small readings' errors larger, hence against ten times that) and the products around them."""
    model, losses = recall.train(gpu, 5, layer=recall.LinearLayer)
    assert len(losses) == 5 and all(torch.isfinite(torch.tensor(losses)))
    tokens, before, _ = (t.to(gpu) for t in recall.batch(32, 8, 15, torch.Generator().manual_seed(2)))
    with torch.no_grad():
        whole = model(tokens, before, model.states(32, gpu), recall.linear_train_form)[:, -15:]
    steps = recall.answer(model, tokens, before, 15)
    assert (steps - whole).norm() <= 2 * 64 * 2.0 ** -23 * 20 * whole.norm()


def test_gradients_match_plain_layers(gpu, recall, monkeypatch):
    """One training step's gradients against the same model over the definitions written out with torch (float32,
    differentiated by torch): both carry float32 sums, so 1e-3 of each gradient's norm."""
    torch.manual_seed(3)
    model = recall.Model(layer=recall.LinearLayer).to(gpu)
    tokens, before, answers = (t.to(gpu) for t in recall.batch(4, 4, 3, torch.Generator().manual_seed(3)))

    def plain(state, k, v, log_decay, q):
        n, scale = v.shape[2] // k.shape[2], k.shape[-1] ** -0.5
        k, q = (t.repeat_interleave(n, 2) for t in (k, q))
        S, outs = state, []
        for t in range(k.shape[1]):
            S = log_decay.exp()[:, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None]
            outs.append(scale * (q[:, t, :, :, None] * S).sum(-2))
        return torch.stack(outs, 1)

    def plain_norm(x, groups, weight, bias, activation):
        assert activation == "silu"
        h = x.unflatten(-1, (groups, -1))
        d = h - h.mean(-1, keepdim=True)
        z = (d * (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt()).flatten(-2) * weight + bias
        return z * torch.sigmoid(z)

    grads = []
    for form in (recall.linear_train_form, plain):
        if form is plain:
            monkeypatch.setattr(recall.sdm, "group_norm", plain_norm)
        logits = model(tokens, before, model.states(4, gpu), form)[:, -3:]
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), answers.flatten())
        grads.append(torch.autograd.grad(loss, list(model.parameters())))
    for (name, _), a, b in zip(model.named_parameters(), *grads):
        assert (a - b).norm() <= 1e-3 * b.norm() + 1e-8, name
