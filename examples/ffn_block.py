"""The feed-forward half of a transformer block, forward and backward, on the
library's operators: the norm before it, the gated up projections in one NVFP4
kernel, the down projection, and the norm after it with the residual's scale
and a gate per channel, and back.  The recipe is that of an NVFP4 linear layer
(1x16 activations, 16x16 weights, gradients rounded stochastically, the
Hadamard transform on both Wgrad operands); what the backward pass needs of
gate, up and the block's output is kept in 8 bits.

  python examples/ffn_block.py [--tokens 16384] [--keep e4m3] [--activation silu]

runs it at the 3B model's sizes (hidden 3072, FFN 9216) on random data and
prints the time of each operator and the memory kept.
"""
import argparse
import os
import sys
from dataclasses import dataclass, field
from typing import Dict, Tuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp4_gemm_nvfp4_gb300 import build, capi, ops  # noqa: E402


@dataclass
class FeedForwardBlock:
    """Weights and what one step keeps between its forward and backward pass."""
    w_up: torch.Tensor                  # bf16 [2 * ffn, hidden]: the gate's rows, then the up projection's
    w_down: torch.Tensor                # bf16 [hidden, ffn]
    pre_norm: torch.Tensor              # float32 [hidden], before the block
    post_norm: torch.Tensor             # after it
    gate: torch.Tensor                  # float32 [hidden]
    next_norm: torch.Tensor             # before the next block
    residual_scale: float = 1.0
    activation: str = "silu"
    keep: str = "e4m3"
    rht_mask: int = 0x5A5A
    seed: int = 0
    saved: Dict[str, object] = field(default_factory=dict)

    @staticmethod
    def random(hidden=3072, ffn=9216, seed=0, device="cuda", **kw):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * 0.02).to(torch.bfloat16)

        ones = torch.ones(hidden, device=device)
        return FeedForwardBlock(weight(2 * ffn, hidden), weight(hidden, ffn), ones.clone(), ones.clone(), 0.5 * ones,
                                ones.clone(), **kw)

    def forward(self, residual: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """residual bf16 or float32 [tokens, hidden] (tokens % 16 == 0) -> the residual after the block and the
        next block's input."""
        s, ffn = self.saved, self.w_down.shape[1]
        s["residual"], s["n"], _ = ops.block_norm(residual, pre_weight=self.pre_norm)
        s["nq"], s["nq_col"] = ops.quantize_row_col_rht(s["n"], self.rht_mask)
        s["wu"], s["wu_col"] = ops.quantize(self.w_up, two_d=True, colwise=True)
        s["wd"], s["wd_col"] = ops.quantize(self.w_down, two_d=True, colwise=True)
        amax = torch.empty(2, device=residual.device)
        h, s["g"], s["u"] = ops.gemm_gated(s["nq"], ops.operand_rows(s["wu"], 0, ffn),
                                           ops.operand_rows(s["wu"], ffn, 2 * ffn), activation=self.activation,
                                           keep=self.keep, amax=amax, rht_mask=self.rht_mask)
        s["hq"], s["hq_col"] = ops.quantize_row_col_rht_amax(h, self.rht_mask, amax)
        y = ops.gemm(s["hq"], s["wd"])
        s["out"], normed, s["y"] = ops.block_norm(residual, y, pre_weight=self.next_norm, post_weight=self.post_norm,
                                                  gate=self.gate, residual_scale=self.residual_scale, keep=self.keep)
        return s["out"], normed

    def backward(self, dout: torch.Tensor, dnormed: torch.Tensor) -> Dict[str, torch.Tensor]:
        """The gradients of forward's two results -> those of its input and of every weight."""
        s = self.saved
        after = ops.block_norm_backward(dout, dnormed, s["out"], s["y"], pre_weight=self.next_norm,
                                        post_weight=self.post_norm, gate=self.gate, residual_scale=self.residual_scale)
        dyq, dyq_col = ops.quantize_row_col_rht(after.dbranch, self.rht_mask, sr=True, seed=self.seed, stream_row=0,
                                                stream_col=1)
        dw_down = ops.gemm(dyq_col, s["hq_col"], out_dtype=torch.float32)
        amax = torch.empty(2, device=dout.device)
        dgu = ops.gemm_gated_backward(dyq, s["wd_col"], s["g"], s["u"], activation=self.activation, amax=amax,
                                      rht_mask=self.rht_mask)
        dgu_row, dgu_col = ops.quantize_row_col_rht_amax(dgu, self.rht_mask, amax, sr=True, seed=self.seed,
                                                         stream_row=2, stream_col=3)
        dw_up = ops.gemm(dgu_col, s["nq_col"], out_dtype=torch.float32)
        dn = ops.gemm(dgu_row, s["wu_col"])
        before = ops.block_norm_backward(after.dresidual, dn, s["residual"], pre_weight=self.pre_norm)
        return {"residual": before.dresidual, "w_up": dw_up, "w_down": dw_down, "pre_norm": before.dpre_weight,
                "post_norm": after.dpost_weight, "gate": after.dgate, "next_norm": after.dpre_weight,
                "y": after.dbranch, "gu": dgu, "n": dn, "stream": after.dresidual}

    def kept_bytes(self) -> int:
        """What gate, up and the block's output take until the backward pass."""
        return sum(self.saved[n].nbytes() for n in ("g", "u", "y"))


def _time(f, steps=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / steps * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16384)
    ap.add_argument("--keep", choices=("e4m3", "bf16"), default="e4m3")
    ap.add_argument("--activation", choices=("silu", "gelu"), default="silu")
    a = ap.parse_args()
    build.build()
    block = FeedForwardBlock.random(keep=a.keep, activation=a.activation)
    hidden, ffn = block.w_down.shape
    x = torch.randn((a.tokens, hidden), device="cuda").to(torch.bfloat16)
    dout, dn = ((torch.randn((a.tokens, hidden), device="cuda") * 1e-3).to(torch.bfloat16) for _ in range(2))
    out, _ = block.forward(x)
    grads = block.backward(dout, dn)
    torch.cuda.synchronize()
    capi.check(ops.device_error(), "feed-forward block")
    s = block.saved
    wg, wu = ops.operand_rows(s["wu"], 0, ffn), ops.operand_rows(s["wu"], ffn, 2 * ffn)
    dyq, _ = ops.quantize(grads["y"])
    around = dict(pre_weight=block.next_norm, post_weight=block.post_norm, gate=block.gate)
    rows = [
        ("forward pass", lambda: block.forward(x)),
        ("backward pass", lambda: block.backward(dout, dn)),
        ("  gated up projections", lambda: ops.gemm_gated(s["nq"], wg, wu, activation=a.activation, keep=a.keep)),
        ("  their backward pass", lambda: ops.gemm_gated_backward(dyq, s["wd_col"], s["g"], s["u"],
                                                                 activation=a.activation)),
        ("  norms around the block", lambda: ops.block_norm(x, grads["y"], keep=a.keep, **around)),
        ("  their backward pass", lambda: ops.block_norm_backward(dout, dn, s["out"], s["y"], **around)),
        ("  down projection", lambda: ops.gemm(s["hq"], s["wd"])),
    ]
    print(f"{a.tokens} tokens, hidden {hidden}, FFN {ffn}: |out| {out.float().norm().item():.4g}, "
          f"|dx| {grads['residual'].float().norm().item():.4g}, kept {block.kept_bytes() / 2 ** 20:.0f} MiB")
    for name, f in rows:
        print(f"{name:32s} {_time(f):9.1f} us")


if __name__ == "__main__":
    main()
