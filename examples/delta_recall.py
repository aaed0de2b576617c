"""Trains a small model of pre-norm gated delta layers on associative recall, then answers with it token by token.

    python examples/delta_recall.py [--steps 300] [--layer linear]

A sequence is pairs (key, value) and then, again and again, one of the keys, each to be answered with its value. Training
runs layer_norm and gated_delta_rule with their gradients. Answering runs the pairs through gated_delta_fwd once, which leaves
each layer's state, and then one token at a time through gated_delta_step on the states in place. With --layer linear the
layers are linear attention with a decay for each head and a norm of each head's readings with an activation: linear_attention and
group_norm with their gradients, then linear_attention_fwd and linear_attention_step.
"""

import argparse
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_sparse_delta_amd as sdm  # noqa: E402

KEYS = 16       # of keys and of values in the vocabulary


class Norm(nn.Module):
    def __init__(self, width):
        super().__init__()
        self.weight, self.bias = nn.Parameter(torch.ones(width)), nn.Parameter(torch.zeros(width))

    def forward(self, x):
        return sdm.layer_norm(x, self.weight, self.bias)


class DeltaLayer(nn.Module):
    """x + Wo delta(Wi norm(x)): key_heads heads of q and k, each shared by value_heads / key_heads heads of v."""

    def __init__(self, width, key_heads=2, value_heads=4, head_dim=32, value_dim=32):
        super().__init__()
        self.sizes = [key_heads * head_dim, key_heads * head_dim, value_heads * value_dim, value_heads, value_heads]
        self.heads, self.shape = (key_heads, head_dim), (value_heads, value_dim)
        self.norm = Norm(width)
        self.inputs = nn.Linear(width, sum(self.sizes))
        self.output = nn.Linear(value_heads * value_dim, width)

    def state(self, streams, device):
        return torch.zeros((streams, self.shape[0], self.heads[1], self.shape[1]), device=device)

    def forward(self, x, state, form):
        q, k, v, beta, decay = self.inputs(self.norm(x)).split(self.sizes, -1)
        q, k = (nn.functional.normalize(nn.functional.silu(t.unflatten(-1, self.heads).float()), dim=-1).to(x.dtype) for t in (q, k))
        v = v.unflatten(-1, self.shape)
        beta, decay = beta.float().sigmoid(), -0.05 * nn.functional.softplus(decay.float())
        out = form(state, k, v, beta.contiguous(), decay.contiguous(), q)
        return x + self.output(out.flatten(-2))


class LinearLayer(nn.Module):
    """x + Wo silu(heads' norm(linear attention(Wi norm(x)))), decays fixed for each head."""

    def __init__(self, width, key_heads=2, value_heads=4, head_dim=32, value_dim=32):
        super().__init__()
        self.sizes = [key_heads * head_dim, key_heads * head_dim, value_heads * value_dim]
        self.heads, self.shape = (key_heads, head_dim), (value_heads, value_dim)
        self.norm = Norm(width)
        self.inputs = nn.Linear(width, sum(self.sizes))
        self.weight, self.bias = nn.Parameter(torch.ones(value_heads * value_dim)), nn.Parameter(torch.zeros(value_heads * value_dim))
        self.output = nn.Linear(value_heads * value_dim, width)
        # memories of 8, 32, 128, ... tokens
        self.register_buffer("log_decay", torch.log1p(-0.125 * 0.25 ** torch.arange(value_heads)))

    state = DeltaLayer.state

    def forward(self, x, state, form):
        q, k, v = self.inputs(self.norm(x)).split(self.sizes, -1)
        q, k = (nn.functional.silu(t).unflatten(-1, self.heads) for t in (q, k))
        out = form(state, k, v.unflatten(-1, self.shape), self.log_decay, q)
        out = sdm.group_norm(out.flatten(2).flatten(0, 1), self.shape[0], self.weight, self.bias, activation="silu")
        return x + self.output(out.unflatten(0, x.shape[:2]))


class Model(nn.Module):
    def __init__(self, width=128, layers=2, layer=DeltaLayer):
        super().__init__()
        self.embed = nn.Embedding(2 * KEYS, width)
        # a value's token also sees the key before it: what a short convolution gives such models
        self.before = nn.Embedding(2 * KEYS, width)
        self.layers = nn.ModuleList(layer(width) for _ in range(layers))
        self.norm, self.head = Norm(width), nn.Linear(width, KEYS)

    def states(self, streams, device):
        return [layer.state(streams, device) for layer in self.layers]

    def forward(self, tokens, before, states, form):
        x = self.embed(tokens) + self.before(before)
        for layer, state in zip(self.layers, states):
            x = layer(x, state, form)
        return self.head(self.norm(x))


def train_form(state, *inputs):
    return sdm.gated_delta_rule(None, *inputs)[0]


def linear_train_form(state, *inputs):
    return sdm.linear_attention(None, *inputs)[0]


# a layer's forms: for training, for a prompt and for single tokens
FORMS = {DeltaLayer: (train_form, sdm.gated_delta_fwd, sdm.gated_delta_step),
         LinearLayer: (linear_train_form, sdm.linear_attention_fwd, sdm.linear_attention_step)}


def batch(streams, pairs, asked, gen):
    """Tokens [streams, 2 pairs + asked], the token before each, and the answers to the last `asked`."""
    keys = torch.rand((streams, KEYS), generator=gen).argsort(1)[:, :pairs]
    values = torch.randint(KEYS, (streams, pairs), generator=gen)
    which = torch.randint(pairs, (streams, asked), generator=gen)
    tokens = torch.cat([torch.stack([keys, KEYS + values], 2).flatten(1), keys.gather(1, which)], 1)
    before = torch.cat([tokens[:, :1], tokens[:, :-1]], 1)
    return tokens, before, values.gather(1, which)


def train(device, steps, streams=64, pairs=8, asked=15, seed=0, layer=DeltaLayer):
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    model = Model(layer=layer).to(device)
    opt = torch.optim.AdamW(model.parameters(), lr=2e-3)
    losses = []
    for _ in range(steps):
        tokens, before, answers = (t.to(device) for t in batch(streams, pairs, asked, gen))
        logits = model(tokens, before, model.states(streams, device), FORMS[layer][0])[:, -asked:]
        loss = nn.functional.cross_entropy(logits.flatten(0, 1), answers.flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return model, torch.stack(losses).tolist()


@torch.no_grad()
def answer(model, tokens, before, asked):
    """Logits of the last `asked` tokens, one step each after one pass over the others; the states advance in place."""
    states = model.states(len(tokens), tokens.device)
    n = tokens.shape[1] - asked
    _, prompt, step = FORMS[type(model.layers[0])]
    model(tokens[:, :n], before[:, :n], states, prompt)
    return torch.cat([model(tokens[:, t:t + 1], before[:, t:t + 1], states, step)
                      for t in range(n, n + asked)], 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--layer", choices=("delta", "linear"), default="delta")
    args = ap.parse_args(argv)
    device = torch.device("cuda:0")
    model, losses = train(device, args.steps, layer=LinearLayer if args.layer == "linear" else DeltaLayer)
    tokens, before, answers = (t.to(device) for t in batch(256, 8, 15, torch.Generator().manual_seed(1)))
    logits = answer(model, tokens, before, 15)
    right = (logits.argmax(-1) == answers).float().mean().item()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps; {100 * right:.1f} % of answers right, token by token")
    return losses, right


if __name__ == "__main__":
    main()
