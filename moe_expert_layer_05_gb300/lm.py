"""A token model of expert layers, forward and backward, on the library's calls:

    tokens -> embedding -> [norm -> expert layer -> + residual] * L -> norm -> vocabulary loss

and with attention heads, a transformer:

    tokens -> embedding -> [norm -> attention -> + residual, norm -> expert layer -> + residual] * L -> ...

The residual sums are taken inside the norms (moe_layer_norm_forward adds the
layer's output to the stream), the stream's gradient is carried through
their backward, and the logits of the head exist only a piece at a time.  Without
heads there is no mixing between positions: the model predicts a label from the
token at its own position.  With them a batch is sequences packed one after the other,
queries and keys turned by their positions.  The routers may have a balance loss, and
the gradients of a step may be clipped to a norm.

    python -m moe_expert_layer_05_gb300.lm --steps 60                           # train it on a made-up task
    python -m moe_expert_layer_05_gb300.lm --heads 4 --balance 0.01 --clip 1    # one that needs attention
"""
from __future__ import annotations

import argparse
import math

import torch

from . import api


class Attention:
    """One attention layer of a model: projections (weights [(q + 2 kv) D, H] and [H, q D]), rotary positions, attention."""

    def __init__(self, T: int, H: int, heads: int, kv_heads: int, head_dim: int, wqkv, wo, freq, device):
        self.heads, self.kv, self.D, self.wqkv, self.wo, self.freq = heads, kv_heads, head_dim, wqkv, wo, freq
        n = heads + 2 * kv_heads
        self.qkv = torch.zeros(T, n, head_dim, dtype=torch.bfloat16, device=device)
        self.out = torch.zeros(T, heads, head_dim, dtype=torch.bfloat16, device=device)
        self.lse = torch.zeros(heads, T, device=device)

    def _parts(self, t):
        return t[:, :self.heads], t[:, self.heads:self.heads + self.kv], t[:, self.heads + self.kv:]

    def forward(self, x, branch, positions, cu_seqlens, ws) -> None:
        T = x.shape[0]
        torch.mm(x, self.wqkv.t(), out=self.qkv.view(T, -1))
        turned = self.qkv[:, :self.heads + self.kv]
        api.moe_rotary(turned, positions, self.freq, turned)
        self.out.zero_()                                       # (rows of no sequence)
        api.moe_attention_forward(*self._parts(self.qkv), cu_seqlens, self.out, self.lse, ws)
        torch.mm(self.out.view(T, -1), self.wo.t(), out=branch)

    def backward(self, x, d_branch, dx, dwqkv, dwo, positions, cu_seqlens, d_out, dqkv, ws) -> None:
        """dx [T, H] and the weights' gradients (bf16); d_out, dqkv: scratch of out's and qkv's shapes."""
        T = x.shape[0]
        torch.mm(d_branch.t(), self.out.view(T, -1), out=dwo)
        torch.mm(d_branch, self.wo, out=d_out.view(T, -1))
        dqkv.zero_()
        api.moe_attention_backward(*self._parts(self.qkv), cu_seqlens, self.out, self.lse, d_out, *self._parts(dqkv), ws)
        turned = dqkv[:, :self.heads + self.kv]
        api.moe_rotary(turned, positions, self.freq, turned, inverse=True)
        torch.mm(dqkv.view(T, -1).t(), x, out=dwqkv)
        torch.mm(dqkv.view(T, -1), self.wqkv, out=dx)


class MoEModel:
    """Weights (bf16, in ``params``), activations and gradients (in ``grads``) for batches of T tokens.

    tied: the embedding's table is the head's weight too; its gradient is then
    the sum of both.  heads > 0: an attention layer in front of every expert layer, kv_heads
    (default: heads) key-value heads of head_dim (default: H / heads).  balance: the factor of the routers'
    balance loss (0: none).  Gradients are fp32, except an untied head's (bf16, as moe_cross_entropy_backward
    writes it) and those of the attention's projections (bf16).
    """

    def __init__(self, T: int, H: int, E: int, k: int, F: int, V: int, layers: int = 1, S: int = 0,
                 score: str = "softmax", tied: bool = True, eps: float = 1e-5, seed: int = 0, device="cuda",
                 heads: int = 0, kv_heads: int = 0, head_dim: int = 0, rotary_base: float = 10000.0,
                 balance: float = 0.0):
        self.T, self.H, self.V, self.layers, self.tied, self.eps = T, H, V, layers, tied, eps
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads or heads, head_dim or (H // heads if heads else 0)
        self.balance, self.score = balance, score
        self.embed_scale = math.sqrt(H)
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            t = torch.empty(shape, dtype=torch.float32, device=device).normal_(0.0, std, generator=gen)
            return t.to(torch.bfloat16)

        p = {"table": normal(V, H, std=H ** -0.5)}
        if not tied:
            p["head"] = normal(V, H, std=H ** -0.5)
        cfg = api.make_config(T, H, E, k, F, S, score)
        freq = api.moe_rotary_frequencies(self.head_dim, rotary_base, device=device)[0] if heads else None
        self.blocks, self.attentions, self.sublayers = [], [], []
        for i in range(layers):
            if heads:
                n, D = (heads + 2 * self.kv_heads) * self.head_dim, heads * self.head_dim
                p[f"layer{i}.wqkv"], p[f"layer{i}.wo"] = normal(n, H, std=H ** -0.5), normal(H, D, std=D ** -0.5)
                self.attentions.append(Attention(T, H, heads, self.kv_heads, self.head_dim, p[f"layer{i}.wqkv"],
                                                 p[f"layer{i}.wo"], freq, device))
                self.sublayers.append(("attention", i))
            w = {"w_router": normal(E, H, std=0.02), "w1": normal(E, 2 * F, H, std=H ** -0.5),
                 "w2": normal(E, H, F, std=F ** -0.5)}
            if S > 0:
                w["w1_shared"], w["w2_shared"] = normal(2 * S, H, std=H ** -0.5), normal(H, S, std=S ** -0.5)
            p.update({f"layer{i}.{n}": t for n, t in w.items()})
            self.blocks.append(api.MoELayer(cfg, w, with_backward=True, device=device))
            self.sublayers.append(("experts", i))
        subs = len(self.sublayers)
        for i in range(subs + 1):
            p[f"norm{i}.weight"] = torch.ones(H, dtype=torch.bfloat16, device=device)
            p[f"norm{i}.bias"] = torch.zeros(H, dtype=torch.bfloat16, device=device)
        self.params = p
        self.grads = {n: torch.empty(t.shape, dtype=torch.bfloat16 if n == "head" or n.endswith((".wqkv", ".wo"))
                                     else torch.float32, device=device) for n, t in p.items()}

        def rows(n):
            return [torch.empty(T, H, dtype=torch.bfloat16, device=device) for _ in range(n)]

        self.stream, self.normed, self.branch = rows(subs + 1), rows(subs + 1), rows(subs)
        self.mean, self.rstd = ([torch.empty(T, device=device) for _ in range(subs + 1)] for _ in range(2))
        self.loss, self.lse = (torch.empty(T, device=device) for _ in range(2))
        self.d_normed, self.d_stream = rows(1)[0], rows(2)
        self.d_head = torch.empty(V, H, dtype=torch.bfloat16, device=device) if tied else self.grads["head"]
        self.dgate = torch.empty(T, k, dtype=torch.float32, device=device)
        if heads:
            self.d_out, self.dqkv = torch.zeros_like(self.attentions[0].out), torch.zeros_like(self.attentions[0].qkv)
            self.one_sequence = (torch.tensor([0, T], dtype=torch.int32, device=device),
                                 torch.arange(T, dtype=torch.int32, device=device))
            self.cu_seqlens, self.positions = self.one_sequence
        if balance:
            self.balance_loss, self.slope = torch.zeros(layers, 1, device=device), torch.zeros(layers, E, device=device)
            self.counts = torch.zeros(layers, E, dtype=torch.int32, device=device)      # choices of each expert
            self.dlogits, self.factor = torch.zeros(T, E, device=device), torch.full((1,), balance, device=device)
        self.grad_norm = torch.zeros(1, device=device)
        self.ws = torch.empty(max(api.moe_embedding_workspace_bytes(T, V, H), api.moe_layer_norm_workspace_bytes(T, H),
                                  api.moe_cross_entropy_workspace_bytes(T, H, V),
                                  api.moe_attention_workspace_bytes(T, heads, self.kv_heads, self.head_dim) if heads else 0,
                                  api.moe_balance_loss_workspace_bytes(T, E),
                                  api.moe_grad_norm_workspace_bytes(len(p))), dtype=torch.uint8, device=device)
        api.moe_workspace_init(self.ws)

    @property
    def head(self) -> torch.Tensor:
        return self.params["table" if self.tied else "head"]

    def _norm(self, i: int, x, residual=None) -> None:
        p = self.params
        api.moe_layer_norm_forward(x, p[f"norm{i}.weight"], p[f"norm{i}.bias"], self.normed[i], self.mean[i],
                                   self.rstd[i], residual=residual, eps=self.eps,
                                   sum_out=None if residual is None else self.stream[i])

    def _routing(self, i: int):
        f = self.blocks[i].fields()
        return f["logits"], f["topk_idx"]

    def forward(self, tokens: torch.Tensor, labels: torch.Tensor, cu_seqlens: torch.Tensor | None = None) -> torch.Tensor:
        """Per-token losses [T] (0 where labels is -1); tokens, labels int32 [T].

        cu_seqlens (models with heads): the packed sequences' first rows and the last one's end, int32; one
        sequence of all tokens where it is not given.
        """
        if cu_seqlens is not None:
            if not self.heads:
                raise ValueError("cu_seqlens: this model has no attention, its tokens do not know of sequences")
            if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or len(cu_seqlens) == 0:
                raise ValueError(f"cu_seqlens: expected the sequences' first rows and the last one's end, int32, got "
                                 f"{tuple(cu_seqlens.shape)} of {cu_seqlens.dtype}")
        if self.heads:
            if cu_seqlens is None:
                self.cu_seqlens, self.positions = self.one_sequence
            else:
                at = torch.arange(self.T, dtype=torch.int32, device=tokens.device)
                first = cu_seqlens[torch.searchsorted(cu_seqlens, at, right=True).sub_(1).clamp_(min=0)]
                self.cu_seqlens, self.positions = cu_seqlens, at - first
        api.moe_embedding_forward(tokens, self.params["table"], self.stream[0], self.ws, scale=self.embed_scale)
        self._norm(0, self.stream[0])
        for j, (kind, i) in enumerate(self.sublayers):
            if kind == "attention":
                self.attentions[i].forward(self.normed[j], self.branch[j], self.positions, self.cu_seqlens, self.ws)
            else:
                self.blocks[i].forward(self.normed[j], self.branch[j])
                if self.balance:
                    logits, topk_idx = self._routing(i)
                    api.moe_balance_loss_forward(logits, topk_idx, self.balance_loss[i], self.counts[i], self.slope[i],
                                                 self.ws, tokens=tokens, score=self.score)
            self._norm(j + 1, self.branch[j], residual=self.stream[j])
        api.moe_cross_entropy_forward(self.normed[-1], self.head, labels, self.loss, self.lse, self.ws)
        return self.loss

    def _balance_backward(self, i: int, x, tokens) -> None:
        """The balance loss's gradients through the router, added to those of the expert layer (whose dx, bf16, is rounded a
        second time here)."""
        logits, _ = self._routing(i)
        api.moe_balance_loss_backward(logits, self.slope[i], self.factor, self.dlogits, tokens=tokens, score=self.score)
        self.d_normed.copy_(torch.addmm(self.d_normed.float(), self.dlogits, self.params[f"layer{i}.w_router"].float()))
        self.grads[f"layer{i}.w_router"].addmm_(self.dlogits.t(), x.float())

    def backward(self, tokens: torch.Tensor, labels: torch.Tensor, dloss: torch.Tensor) -> dict:
        """Gradients of sum_t dloss[t] * loss[t] (and of the balance losses times their factor) for the batch that
        forward() ran last (fp32 dloss [T])."""
        p, g = self.params, self.grads
        api.moe_cross_entropy_backward(self.normed[-1], self.head, labels, self.lse, dloss, self.d_normed, self.d_head,
                                       self.ws)
        d_out = None                       # gradient of the stream that later layers left
        for j in range(len(self.sublayers), -1, -1):
            d_in = self.d_stream[j % 2]
            api.moe_layer_norm_backward(self.d_normed, self.stream[j], p[f"norm{j}.weight"], self.mean[j], self.rstd[j],
                                        d_in, g[f"norm{j}.weight"], g[f"norm{j}.bias"], self.ws, dsum=d_out)
            d_out = d_in
            if j == 0:
                continue
            kind, i = self.sublayers[j - 1]
            x = self.normed[j - 1]
            if kind == "attention":
                self.attentions[i].backward(x, d_out, self.d_normed, g[f"layer{i}.wqkv"], g[f"layer{i}.wo"], self.positions,
                                            self.cu_seqlens, self.d_out, self.dqkv, self.ws)
            else:
                grads = {"d" + n: g[f"layer{i}.{n}"] for n in ("w_router", "w1", "w2", "w1_shared", "w2_shared")
                         if f"layer{i}.{n}" in g}
                self.blocks[i].backward(x, d_out, grads=grads, dx=self.d_normed, dgate=self.dgate)
                if self.balance:
                    self._balance_backward(i, x, tokens)
        api.moe_embedding_backward(tokens, d_out, g["table"], self.ws, scale=self.embed_scale,
                                   base=self.d_head if self.tied else None)
        return g

    def step(self, tokens: torch.Tensor, labels: torch.Tensor, cu_seqlens: torch.Tensor | None = None) -> torch.Tensor:
        """Forward and backward of the mean loss over the scored positions, plus the balance losses times their
        factor; that sum, on the device."""
        loss = self.forward(tokens, labels, cu_seqlens)
        share = (labels >= 0).float()
        share /= share.sum().clamp(min=1.0)
        self.backward(tokens, labels, share)
        mean = torch.dot(loss, share)
        return mean + self.balance * self.balance_loss.sum() if self.balance else mean

    def clip(self, limit: float) -> torch.Tensor:
        """Scale all gradients of the last step so that their norm is at most `limit`; the norm they had, on the device."""
        grads = list(self.grads.values())
        api.moe_grad_norm(grads, self.grad_norm, self.ws)
        api.moe_grad_clip(grads, self.grad_norm, limit)
        return self.grad_norm

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
    ap.add_argument("--heads", type=int, default=0, help="attention heads (0: no attention)")
    ap.add_argument("--kv-heads", type=int, default=0, help="key-value heads (0: as many)")
    ap.add_argument("--length", type=int, default=100, help="tokens of a sequence, with attention")
    ap.add_argument("--balance", type=float, default=0.0, help="factor of the routers' balance loss")
    ap.add_argument("--clip", type=float, default=0.0, help="limit of the gradients' norm (0: none)")
    a = ap.parse_args(argv)
    model = MoEModel(a.tokens, a.hidden, a.experts, 2, 2 * a.hidden, a.vocab, layers=a.layers, tied=not a.untied,
                     heads=a.heads, kv_heads=a.kv_heads, balance=a.balance)
    cu_seqlens = None
    if a.heads:
        cu_seqlens = torch.tensor([*range(0, a.tokens, a.length), a.tokens], dtype=torch.int32, device="cuda")
    # fp32 copies of the weights are what is optimised; the model computes on their bf16 roundings
    master = {n: t.float().requires_grad_() for n, t in model.params.items()}
    opt = torch.optim.Adam(master.values(), lr=a.lr)
    gen = torch.Generator(device="cuda").manual_seed(1)
    next_token = torch.randperm(a.vocab, device="cuda", generator=gen).to(torch.int32)   # the rule to learn
    losses = []
    for step in range(a.steps):
        tokens = torch.randint(0, a.vocab, (a.tokens,), device="cuda", generator=gen, dtype=torch.int32)
        labels = next_token[tokens.long()]
        if a.heads:
            labels = labels.roll(1)                            # the rule asks for the token before
            labels[cu_seqlens[:-1].long()] = -1
        labels[:: 16] = -1                                     # some positions are not scored
        losses.append(float(model.step(tokens, labels, cu_seqlens)))
        if a.clip > 0:
            model.clip(a.clip)
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
