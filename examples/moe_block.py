"""A decode step's mixture-of-experts block out of the library's calls: norm, router, choice of experts, experts in MXFP4.

    python examples/moe_block.py [--tokens 16 --hidden 2048 --width 1024 --experts 64]

For tokens x with a residual stream r:

    h = bf16(x + r);  y = norm(h)                       rmsnorm: y in bf16 and in MXFP4, and h, in one pass
    logits = y @ Wr^T                                   the router GEMM (fp32 logits)
    weights, ids = route(logits)                        sigmoid scores, balance bias, limited groups, top-k
    out[t] = sum over the chosen e of weight * down_e(silu(gate_e(y)) * up_e(y))
                                                        bf16_linear_mxfp4 on the norm's codes, _dynamic on the inner values

The experts run one after another on the rows that chose them; everything stays on the device but the list of experts
that have any.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import moe_router_gemm_gb300 as m


def make_weights(hidden, width, experts, seed=0, device="cuda"):
    """Random weights: router and norm in bf16, each expert's gate-and-up and down projections in MXFP4."""
    g = torch.Generator(device=device).manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).to(torch.bfloat16)

    return dict(norm=(1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(torch.bfloat16), router=w(experts, hidden),
                bias=0.05 * torch.randn(experts, generator=g, device=device),
                gate_up=[m.quant_mxfp4(w(2 * width, hidden)) for _ in range(experts)],
                down=[m.quant_mxfp4(w(hidden, width)) for _ in range(experts)])


def moe_block(x, residual, weights, k=4, groups=4, top_groups=2):
    """The block's output in bf16, the new residual stream, and what lies between (for a caller that looks)."""
    y = m.rmsnorm(x, weights["norm"], residual, quant="mxfp4")
    logits = m.bf16_linear_f32out(y.out, weights["router"])
    w, ids = m.route(logits, k, scoring="sigmoid", bias=weights["bias"], groups=groups, top_groups=top_groups, group_best=2)
    out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    inner = {}
    for e in ids.unique().tolist():
        token, slot = (ids == e).nonzero(as_tuple=True)
        gate, up = m.bf16_linear_mxfp4(y.codes[token], y.scales[token], *weights["gate_up"][e]).float().chunk(2, dim=-1)
        act = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
        down = m.bf16_linear_mxfp4_dynamic(act, *weights["down"][e])
        out.index_add_(0, token, down.float() * w[token, slot, None])
        inner[e] = (token, slot, act, down)
    return out.to(torch.bfloat16), y.residual, dict(norm=y, logits=logits, weights=w, ids=ids, experts=inner)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 16), ("hidden", 2048), ("width", 1024), ("experts", 64)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    weights = make_weights(a.hidden, a.width, a.experts)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, residual, between = moe_block(x, r, weights)
    torch.cuda.synchronize()
    used = sorted(between["experts"])
    print(f"{a.tokens} tokens through {len(used)} of {a.experts} experts: out {tuple(out.shape)}, rms {out.float().square().mean().sqrt():.4f}; "
          f"token 0 chose {between['ids'][0].tolist()} with weights {[round(v, 3) for v in between['weights'][0].tolist()]}")


if __name__ == "__main__":
    main()
