"""Trains a small MXFP8 mixture-of-experts layer on a fixed batch, then runs it on single tokens.

    python examples/moe_ffn.py [--steps 30]

Every step goes through routing, dispatch, the grouped products, the gated activation with its 8-bit checkpoint, combine,
and all of their gradients; the last part is the same layer as a decoder calls it, a token at a time and in one call for a few.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B  # noqa: E402
from mxfp8_precision_gemms_fp8bw_gb300.moe import MxMoEFFN  # noqa: E402


def main(steps: int = 30, tokens: int = 1000, dim: int = 256, hidden: int = 512, experts: int = 8, top_k: int = 2):
    torch.manual_seed(0)
    layer = MxMoEFFN(dim, hidden, experts, top_k, score="sigmoid", groups=4, groups_kept=2, group_top=2, device="cuda")
    x = torch.randn(tokens, dim, device="cuda").bfloat16()
    want = x.float().roll(1, dims=1)
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for step in range(steps):
        loss = (layer(x).float() - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        layer.update_balance()
        losses.append(loss.detach())
        if step % 10 == 0 or step + 1 == steps:
            print(f"step {step:3d}  mean square error {float(losses[-1]):.4f}  loads {layer.counts.tolist()}")
    with torch.no_grad():
        codes = layer.weight_codes(colwise=False)  # the weights stay as they are from here on
        together = layer(x[:4], codes)
        alone = torch.cat([layer(x[i:i + 1], codes) for i in range(4)])
        few = layer.decode(x[:4], layer.weight_codes(bits=4))  # for up to 32 tokens, weights in 4 bits
    B.fp8bw_sync_status()
    print("tokens one at a time equal the batch:", bool(torch.equal(together, alone)))
    print(f"with weights in 4 bits {float((few - together).float().norm() / together.float().norm()):.3f} of the result away")
    return [float(v) for v in losses], together, alone


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    main(ap.parse_args().steps)
