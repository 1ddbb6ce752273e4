"""The attention half of a transformer block, forward and backward, on the
library's operators: NVFP4 QKV projection, per-head norm with position
rotation, attention, NVFP4 O projection, and back, with the recipe of an
NVFP4 linear layer (1x16 activations, 16x16 weights, gradients rounded
stochastically, the Hadamard transform on both Wgrad operands).

  python examples/attention_block.py [--tokens 8192] [--context 2048] [--softcap 0]

runs it at the 3B model's sizes (hidden 3072, 24 query and 12 key/value heads
of 128) on random data, packed sequences of --context tokens, and prints the
time of each operator.
"""
import argparse
import os
import sys
from dataclasses import dataclass, field
from typing import Dict, Optional

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp4_gemm_nvfp4_gb300 import build, capi, ops  # noqa: E402


@dataclass
class AttentionBlock:
    """Weights and what one step keeps between its forward and backward pass."""
    hidden: int
    q_heads: int
    kv_heads: int
    head_dim: int
    w_qkv: torch.Tensor                 # bf16 [(q_heads + 2 kv_heads) * head_dim, hidden]
    w_o: torch.Tensor                   # bf16 [hidden, q_heads * head_dim]
    q_norm: torch.Tensor                # float32 [head_dim]
    k_norm: torch.Tensor
    cos: torch.Tensor                   # ops.rope_tables
    sin: torch.Tensor
    softcap: float = 0.0
    slopes: Optional[torch.Tensor] = None
    rht_mask: int = 0x5A5A
    seed: int = 0
    saved: Dict[str, object] = field(default_factory=dict)

    @staticmethod
    def random(hidden=3072, q_heads=24, kv_heads=12, head_dim=128, positions=2048, softcap=0.0, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * 0.02).to(torch.bfloat16)

        ones = torch.ones(head_dim, device=device)
        return AttentionBlock(hidden, q_heads, kv_heads, head_dim, weight((q_heads + 2 * kv_heads) * head_dim, hidden),
                              weight(hidden, q_heads * head_dim), ones.clone(), ones.clone(),
                              *ops.rope_tables(positions, head_dim, device=device), softcap=softcap)

    def forward(self, x: torch.Tensor, positions: torch.Tensor, spans: torch.Tensor) -> torch.Tensor:
        """x bf16 [tokens, hidden] (tokens % 16 == 0) -> y bf16 [tokens, hidden]."""
        s = self.saved
        s["positions"], s["spans"] = positions, spans
        s["xq"], s["xq_col"] = ops.quantize_row_col_rht(x, self.rht_mask)
        s["wq"], s["wq_col"] = ops.quantize(self.w_qkv, two_d=True, colwise=True)
        s["wo"], s["wo_col"] = ops.quantize(self.w_o, two_d=True, colwise=True)
        qkv = s["qkv"] = ops.gemm(s["xq"], s["wq"])
        s["q"], s["k"] = ops.qk_norm_rope(qkv, self.q_norm, self.k_norm, self.cos, self.sin, positions,
                                          q_heads=self.q_heads, kv_heads=self.kv_heads)
        # the values stay where the projection wrote them
        s["v"] = qkv[:, (self.q_heads + self.kv_heads) * self.head_dim:].unflatten(1, (self.kv_heads, self.head_dim))
        s["o"], s["lse"] = ops.attention(s["q"], s["k"], s["v"], spans, softcap=self.softcap, slopes=self.slopes)
        s["oq"], s["oq_col"] = ops.quantize_row_col_rht(s["o"].flatten(1), self.rht_mask)
        return ops.gemm(s["oq"], s["wo"])

    def backward(self, dy: torch.Tensor) -> Dict[str, torch.Tensor]:
        """dy bf16 [tokens, hidden] -> gradients of x and of every weight."""
        s, d = self.saved, self.head_dim
        dyq, dyq_col = ops.quantize_row_col_rht(dy, self.rht_mask, sr=True, seed=self.seed, stream_row=0, stream_col=1)
        do = ops.gemm(dyq, s["wo_col"])
        dw_o = ops.gemm(dyq_col, s["oq_col"], out_dtype=torch.float32)
        dqkv = torch.empty_like(s["qkv"])
        dv = dqkv[:, (self.q_heads + self.kv_heads) * d:].unflatten(1, (self.kv_heads, d))
        dq, dk, _ = ops.attention_backward(do.unflatten(1, (self.q_heads, d)), s["q"], s["k"], s["v"], s["o"], s["lse"],
                                           s["spans"], softcap=self.softcap, slopes=self.slopes, dv=dv)
        _, dq_norm, dk_norm = ops.qk_norm_rope_backward(dq, dk, s["qkv"], self.q_norm, self.k_norm, self.cos, self.sin,
                                                        s["positions"], dqkv=dqkv)
        dq_row, dq_col = ops.quantize_row_col_rht(dqkv, self.rht_mask, sr=True, seed=self.seed, stream_row=2, stream_col=3)
        return {"x": ops.gemm(dq_row, s["wq_col"]),
                "w_qkv": ops.gemm(dq_col, s["xq_col"], out_dtype=torch.float32), "w_o": dw_o,
                "q_norm": dq_norm, "k_norm": dk_norm, "qkv": dqkv, "o": do}


def packed(tokens: int, context: int, device="cuda"):
    """Positions and key intervals of sequences of `context` tokens, packed and causal."""
    at = torch.arange(tokens, device=device, dtype=torch.int32)
    offsets = torch.tensor(list(range(0, tokens, context)) + [tokens], dtype=torch.int32, device=device)
    return at % context, ops.attention_spans(offsets, tokens)


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
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--context", type=int, default=2048)
    ap.add_argument("--softcap", type=float, default=0.0)
    a = ap.parse_args()
    build.build()
    block = AttentionBlock.random(positions=a.context, softcap=a.softcap)
    x = torch.randn((a.tokens, block.hidden), device="cuda").to(torch.bfloat16)
    dy = (torch.randn((a.tokens, block.hidden), device="cuda") * 1e-3).to(torch.bfloat16)
    positions, spans = packed(a.tokens, a.context)
    y = block.forward(x, positions, spans)
    grads = block.backward(dy)
    torch.cuda.synchronize()
    capi.check(ops.device_error(), "attention block")
    s, d = block.saved, block.head_dim
    do = grads["o"].unflatten(1, (block.q_heads, d))
    norm = (block.q_norm, block.k_norm, block.cos, block.sin, positions)
    rows = [
        ("forward pass", lambda: block.forward(x, positions, spans)),
        ("backward pass", lambda: block.backward(dy)),
        ("  norm and rotation", lambda: ops.qk_norm_rope(s["qkv"], *norm, q_heads=block.q_heads, kv_heads=block.kv_heads)),
        ("  attention", lambda: ops.attention(s["q"], s["k"], s["v"], spans, softcap=a.softcap)),
        ("  attention, backward", lambda: ops.attention_backward(do, s["q"], s["k"], s["v"], s["o"], s["lse"], spans,
                                                                  softcap=a.softcap)),
        ("  norm and rotation, backward", lambda: ops.qk_norm_rope_backward(do, s["k"], s["qkv"], *norm,
                                                                            dqkv=grads["qkv"])),
        ("  QKV projection", lambda: ops.gemm(s["xq"], s["wq"])),
    ]
    print(f"{a.tokens} tokens in sequences of {a.context}, hidden {block.hidden}, {block.q_heads}/{block.kv_heads} heads "
          f"of {d}: |y| {y.float().norm().item():.4g}, |dx| {grads['x'].float().norm().item():.4g}")
    for name, f in rows:
        print(f"{name:32s} {_time(f):9.1f} us")


if __name__ == "__main__":
    main()
