"""A token model of expert layers, forward and backward, on the library's calls:

    tokens -> embedding -> [norm -> expert layer -> + residual] * L -> norm -> vocabulary loss

The residual sums are taken inside the norms (moe_layer_norm_forward adds the
expert layer's output to the stream), the stream's gradient is carried through
their backward, and the logits of the head exist only a piece at a time.  There
is no mixing between positions: the model predicts a label from the token at its
own position.

    python -m moe_expert_layer_05_gb300.lm --steps 60      # train it on a made-up task
"""
from __future__ import annotations

import argparse
import math

import torch

from . import api


class MoEModel:
    """Weights (bf16, in ``params``), activations and gradients (in ``grads``) for batches of T tokens.

    tied: the embedding's table is the head's weight too; its gradient is then
    the sum of both.  Gradients are fp32, except an untied head's (bf16, as
    moe_cross_entropy_backward writes it).
    """

    def __init__(self, T: int, H: int, E: int, k: int, F: int, V: int, layers: int = 1, S: int = 0,
                 score: str = "softmax", tied: bool = True, eps: float = 1e-5, seed: int = 0, device="cuda"):
        self.T, self.H, self.V, self.layers, self.tied, self.eps = T, H, V, layers, tied, eps
        self.embed_scale = math.sqrt(H)
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            t = torch.empty(shape, dtype=torch.float32, device=device).normal_(0.0, std, generator=gen)
            return t.to(torch.bfloat16)

        p = {"table": normal(V, H, std=H ** -0.5)}
        if not tied:
            p["head"] = normal(V, H, std=H ** -0.5)
        cfg = api.make_config(T, H, E, k, F, S, score)
        self.blocks = []
        for i in range(layers):
            w = {"w_router": normal(E, H, std=0.02), "w1": normal(E, 2 * F, H, std=H ** -0.5),
                 "w2": normal(E, H, F, std=F ** -0.5)}
            if S > 0:
                w["w1_shared"], w["w2_shared"] = normal(2 * S, H, std=H ** -0.5), normal(H, S, std=S ** -0.5)
            p.update({f"layer{i}.{n}": t for n, t in w.items()})
            self.blocks.append(api.MoELayer(cfg, w, with_backward=True, device=device))
        for i in range(layers + 1):
            p[f"norm{i}.weight"] = torch.ones(H, dtype=torch.bfloat16, device=device)
            p[f"norm{i}.bias"] = torch.zeros(H, dtype=torch.bfloat16, device=device)
        self.params = p
        self.grads = {n: torch.empty(t.shape, dtype=torch.bfloat16 if n == "head" else torch.float32, device=device)
                      for n, t in p.items()}

        def rows(n):
            return [torch.empty(T, H, dtype=torch.bfloat16, device=device) for _ in range(n)]

        self.stream, self.normed, self.branch = rows(layers + 1), rows(layers + 1), rows(layers)
        self.mean, self.rstd = ([torch.empty(T, device=device) for _ in range(layers + 1)] for _ in range(2))
        self.loss, self.lse = (torch.empty(T, device=device) for _ in range(2))
        self.d_normed, self.d_stream = rows(1)[0], rows(2)
        self.d_head = torch.empty(V, H, dtype=torch.bfloat16, device=device) if tied else self.grads["head"]
        self.dgate = torch.empty(T, k, dtype=torch.float32, device=device)
        self.ws = torch.empty(max(api.moe_embedding_workspace_bytes(T, V, H), api.moe_layer_norm_workspace_bytes(T, H),
                                  api.moe_cross_entropy_workspace_bytes(T, H, V)), dtype=torch.uint8, device=device)
        api.moe_workspace_init(self.ws)

    @property
    def head(self) -> torch.Tensor:
        return self.params["table" if self.tied else "head"]

    def _norm(self, i: int, x, residual=None) -> None:
        p = self.params
        api.moe_layer_norm_forward(x, p[f"norm{i}.weight"], p[f"norm{i}.bias"], self.normed[i], self.mean[i],
                                   self.rstd[i], residual=residual, eps=self.eps,
                                   sum_out=None if residual is None else self.stream[i])

    def forward(self, tokens: torch.Tensor, labels: torch.Tensor) -> torch.Tensor:
        """Per-token losses [T] (0 where labels is -1); tokens, labels int32 [T]."""
        api.moe_embedding_forward(tokens, self.params["table"], self.stream[0], self.ws, scale=self.embed_scale)
        self._norm(0, self.stream[0])
        for i, block in enumerate(self.blocks):
            block.forward(self.normed[i], self.branch[i])
            self._norm(i + 1, self.branch[i], residual=self.stream[i])
        api.moe_cross_entropy_forward(self.normed[-1], self.head, labels, self.loss, self.lse, self.ws)
        return self.loss

    def backward(self, tokens: torch.Tensor, labels: torch.Tensor, dloss: torch.Tensor) -> dict:
        """Gradients of sum_t dloss[t] * loss[t] for the batch that forward() ran last (fp32 dloss [T])."""
        p, g = self.params, self.grads
        api.moe_cross_entropy_backward(self.normed[-1], self.head, labels, self.lse, dloss, self.d_normed, self.d_head,
                                       self.ws)
        d_out = None                       # gradient of the stream that later layers left
        for i in range(self.layers, -1, -1):
            d_in = self.d_stream[i % 2]
            api.moe_layer_norm_backward(self.d_normed, self.stream[i], p[f"norm{i}.weight"], self.mean[i], self.rstd[i],
                                        d_in, g[f"norm{i}.weight"], g[f"norm{i}.bias"], self.ws, dsum=d_out)
            d_out = d_in
            if i > 0:
                grads = {"d" + n: g[f"layer{i - 1}.{n}"] for n in ("w_router", "w1", "w2", "w1_shared", "w2_shared")
                         if f"layer{i - 1}.{n}" in g}
                self.blocks[i - 1].backward(self.normed[i - 1], d_out, grads=grads, dx=self.d_normed, dgate=self.dgate)
        api.moe_embedding_backward(tokens, d_out, g["table"], self.ws, scale=self.embed_scale,
                                   base=self.d_head if self.tied else None)
        return g

    def step(self, tokens: torch.Tensor, labels: torch.Tensor) -> torch.Tensor:
        """Forward and backward of the mean loss over the scored positions; the mean, on the device."""
        loss = self.forward(tokens, labels)
        share = (labels >= 0).float()
        share /= share.sum().clamp(min=1.0)
        self.backward(tokens, labels, share)
        return torch.dot(loss, share)

    def status(self) -> int:
        """First device error of any call (0: none).  Synchronises."""
        codes = [api.moe_read_device_status(w) for w in (self.ws, *(b.ws for b in self.blocks))]
        return next((c for c in codes if c != 0), 0)


def main(argv=None) -> list[float]:
    ap = argparse.ArgumentParser(description="Train a small token model of expert layers on a made-up task.")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=2003)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--untied", action="store_true")
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args(argv)
    model = MoEModel(a.tokens, a.hidden, a.experts, 2, 2 * a.hidden, a.vocab, layers=a.layers, tied=not a.untied)
    # fp32 copies of the weights are what is optimised; the model computes on their bf16 roundings
    master = {n: t.float().requires_grad_() for n, t in model.params.items()}
    opt = torch.optim.Adam(master.values(), lr=a.lr)
    gen = torch.Generator(device="cuda").manual_seed(1)
    next_token = torch.randperm(a.vocab, device="cuda", generator=gen).to(torch.int32)   # the rule to learn
    losses = []
    for step in range(a.steps):
        tokens = torch.randint(0, a.vocab, (a.tokens,), device="cuda", generator=gen, dtype=torch.int32)
        labels = next_token[tokens.long()]
        labels[:: 16] = -1                                     # some positions are not scored
        losses.append(float(model.step(tokens, labels)))
        for n, t in master.items():
            t.grad = model.grads[n].float()
        opt.step()
        with torch.no_grad():
            for n, t in master.items():
                model.params[n].copy_(t)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {losses[-1]:.4f}  (uniform guess {math.log(a.vocab):.4f})")
    if model.status() != 0:
        raise api.MoeError(model.status(), "lm")
    return losses


if __name__ == "__main__":
    main()
