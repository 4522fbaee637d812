"""One MoE block, trained for a few steps and then decoded with 4-bit experts.

    python examples/moe_block.py            # both, with the losses printed

The block, in the order its kernels run (residual stream r, [T, H]):

    n = norm(r) * w_pre                         block_norm
    scores = n @ router                         (a library product)
    idx, w = topk_gate(scores)                  topk_gate
    map = route_map(idx)                        route_map
    y_e = down(swiglu(up(n)))  per expert       training: library products;
                                                decoding: expert_matvec_fp4
    y = sum_j w_j y_e                           combine
    h = r + scale * g * norm(y) * w_post        block_norm

Training adds balance_loss over the packed sequences and runs the backward
passes: block_norm_backward, combine_backward, the experts', the router's
(balance_loss_backward, which takes the top-k weights' gradient with it) and
block_norm_backward again.  Decoding quantises the trained experts once with
the library's own FP4 cast and then runs every step in its kernels.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass, field

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_routing_precision_gb300 import _build, ops  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@dataclass
class Block:
    """Parameters: f32 masters, as an optimizer would keep them."""
    H: int = 256
    N: int = 128          # expert width
    E: int = 8
    k: int = 2
    scale: float = 0.7    # residual scale
    balance_coef: float = 0.02
    z_coef: float = 1e-3
    group: int = 32
    device: str = "cuda"
    seed: int = 0
    p: dict = field(default_factory=dict)

    def __post_init__(self):
        g = torch.Generator().manual_seed(self.seed)

        def randn(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(self.device)

        H, N, E = self.H, self.N, self.E
        self.p = dict(pre=torch.ones(H, device=self.device), post=torch.ones(H, device=self.device),
                      gate=torch.full((H,), 0.5, device=self.device),
                      router=randn(H, E, std=H ** -0.5),
                      up=randn(E, 2 * N, H, std=H ** -0.5),      # gate rows, then up rows
                      down=randn(E, H, N, std=N ** -0.5))


def swiglu(x):
    gate, up = x.float().chunk(2, -1)
    return gate * torch.sigmoid(gate) * up


def forward(b: Block, r, seq_offsets, token_mask=None):
    """The block's output h and what its backward pass needs."""
    p = b.p
    _, n, _, rstd_pre = ops.block_norm(r, pre_weight=p["pre"])
    scores = n.float() @ p["router"]
    idx, w = ops.topk_gate(scores, b.k)
    counts, offsets, pos, src = ops.route_map(idx, b.E)
    rows = n[(src // b.k).long()]
    ends = offsets.tolist()
    pre_act = torch.empty(rows.shape[0], 2 * b.N, dtype=BF, device=r.device)
    y_e = torch.empty_like(rows)
    for e in range(b.E):
        s = slice(ends[e], ends[e + 1])
        pre_act[s] = (rows[s].float() @ p["up"][e].T).to(BF)
        y_e[s] = (swiglu(pre_act[s]) @ p["down"][e].T).to(BF)
    y = ops.combine(y_e, w, pos)
    h, _, rstd_post, _ = ops.block_norm(r, y, post_weight=p["post"], gate=p["gate"],
                                        gate_act="sigmoid", scale=b.scale)
    losses = ops.balance_loss(scores, idx, seq_offsets=seq_offsets, token_mask=token_mask)
    saved = dict(r=r, n=n, rstd_pre=rstd_pre, scores=scores, idx=idx, w=w, ends=ends, pos=pos,
                 src=src, rows=rows, pre_act=pre_act, y_e=y_e, y=y, rstd_post=rstd_post, h=h,
                 losses=losses, seq_offsets=seq_offsets, token_mask=token_mask)
    return h, saved


def backward(b: Block, s: dict, grad_h):
    """Gradients of <grad_h, h> + balance_coef * mean balance + z_coef * mean z
    (means over the sequences) for every parameter and for r."""
    p, g = b.p, {}
    grad_r, grad_y, g["post"], g["gate"], _ = ops.block_norm_backward(
        grad_h, None, s["h"], y=s["y"], post_weight=p["post"], gate=p["gate"], gate_act="sigmoid",
        scale=b.scale, rstd_post=s["rstd_post"])
    grad_rows_out, grad_w = ops.combine_backward(grad_y, s["y_e"], s["w"], s["pos"])
    g["up"], g["down"] = torch.zeros_like(p["up"]), torch.zeros_like(p["down"])
    grad_rows = torch.empty_like(s["rows"])
    for e in range(b.E):
        q = slice(s["ends"][e], s["ends"][e + 1])
        gate, up = s["pre_act"][q].float().chunk(2, -1)
        sig = torch.sigmoid(gate)
        go = grad_rows_out[q].float()
        g["down"][e] = go.T @ (gate * sig * up)
        ga = go @ p["down"][e]
        g_pre = torch.cat([ga * up * sig * (1 + gate * (1 - sig)), ga * gate * sig], -1)
        g["up"][e] = g_pre.T @ s["rows"][q].float()
        grad_rows[q] = (g_pre @ p["up"][e]).to(BF)
    # a token's row went to its k experts: the gradients come back summed
    grad_n = ops.combine(grad_rows, torch.ones_like(s["w"]), s["pos"], F32)
    _, _, counts, _, tokens = s["losses"]
    S = tokens.numel()
    grad_scores = ops.balance_loss_backward(
        s["scores"], counts, tokens, torch.full((S,), b.balance_coef / S, device=grad_h.device),
        torch.full((S,), b.z_coef / S, device=grad_h.device), seq_offsets=s["seq_offsets"],
        token_mask=s["token_mask"], topk_idx=s["idx"], topk_weights=s["w"],
        grad_topk_weights=grad_w)
    g["router"] = s["n"].float().T @ grad_scores
    grad_n += grad_scores @ p["router"].T
    grad_r2, _, _, _, g["pre"] = ops.block_norm_backward(
        None, grad_n.to(BF), s["r"], pre_weight=p["pre"], rstd_pre=s["rstd_pre"])
    return grad_r + grad_r2, g


def train(b: Block, steps: int = 8, tokens: int = 192, lr: float = 0.5, say=print):
    """Fits the block to move a batch of three packed sequences towards a target
    with plain gradient steps; the loss of every step."""
    gen = torch.Generator().manual_seed(b.seed + 1)
    r = torch.randn(tokens, b.H, generator=gen).to(b.device)
    target = r + torch.tanh(torch.randn(tokens, b.H, generator=gen)).to(b.device) * 0.5
    cuts = torch.tensor([0, tokens // 5, tokens // 2, tokens], dtype=torch.int32, device=b.device)
    history = []
    for step in range(steps):
        h, s = forward(b, r, cuts)
        balance, z = s["losses"][0], s["losses"][1]
        err = h - target
        loss = 0.5 * err.square().mean()
        total = loss + b.balance_coef * balance.mean() + b.z_coef * z.mean()
        _, g = backward(b, s, err / err.numel())
        for name, grad in g.items():
            b.p[name] -= lr * grad * tokens ** 0.5
        history.append(float(total))
        say(f"step {step}: loss {float(loss):.5f}  balance {float(balance.mean()):.4f}  "
            f"z {float(z.mean()):.4f}  total {history[-1]:.5f}")
    return history


def quantise(b: Block, ue8m0: bool = True) -> dict:
    """The experts in 4 bits, once: the library's FP4 cast of every weight row."""
    flags = ops.SF_POW2 | ops.SF_UE8M0 if ue8m0 else 0
    out = {}
    for name in ("up", "down"):
        w = b.p[name].to(BF)
        E, M, K = w.shape
        rows = torch.arange(E * M, dtype=torch.int32, device=b.device).view(-1, 1)
        q, sf = ops.expand_cast_fp4(w.reshape(E * M, K), rows, group=b.group, sf_flags=flags)
        out[name] = (q.view(E, M, K // 2), sf.view(E, M, K // b.group))
    return out


def decode(b: Block, q: dict, r):
    """One decoding step of a small batch r [T, H]: every step of the block in the
    library's kernels but the router's product."""
    p = b.p
    _, n, _, _ = ops.block_norm(r, pre_weight=p["pre"])
    idx, w = ops.topk_gate((n.float() @ p["router"]).contiguous(), b.k)
    _, offsets, pos, src = ops.route_map(idx, b.E)
    act = ops.expert_matvec_fp4(n, *q["up"], offsets, sorted_src=src, k=b.k, group=b.group,
                                swiglu=True)
    y_e = ops.expert_matvec_fp4(act, *q["down"], offsets, k=b.k, group=b.group)
    y = ops.combine(y_e, w, pos)
    h, _, _, _ = ops.block_norm(r, y, post_weight=p["post"], gate=p["gate"], gate_act="sigmoid",
                                scale=b.scale)
    return h


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=192)
    a = ap.parse_args()
    _build.build()
    b = Block()
    train(b, a.steps, a.tokens)
    q = quantise(b)
    r = torch.randn(4, b.H, device=b.device)
    with_bf16, _ = forward(b, r, None)
    h = decode(b, q, r)
    rel = float((h - with_bf16).norm() / (with_bf16 - r).norm())
    print(f"decoded 4 tokens with 4-bit experts: relative to the bf16 block's update {rel:.3f}")
    assert ops.device_status() == 0


if __name__ == "__main__":
    main()
