"""The entry points of a block's feed-forward half in the library's debug build
(NVFP4_BOUNDS_CHECK): run by tests/test_gpu_block_bounds.py in a process of
its own, so that the debug library is the only one loaded here.  Ragged shapes
in every mode leave the check's count at zero and equal the regular build's
values, which the parent passes in a file; with the declared ranges shortened
by 16 bytes the check fires.  Exits 0 when all holds."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from fp4_gemm_nvfp4_gb300 import build, capi, ops  # noqa: E402


def results():
    """{name: tensor} of every entry point on ragged shapes."""
    out = {}
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    for T, H, kind, gate in ((1, 8, torch.bfloat16, "channel"), (131, 264, torch.float32, "token"),
                             (37, 3072, torch.bfloat16, "token"), (20, 4104, torch.float32, "channel")):
        r, y = normal(T, H).to(kind), normal(T, H).to(torch.bfloat16)
        args = {"post_weight": normal(H), "pre_weight": normal(H),
                "gate": normal(H) if gate == "channel" else normal(T, H).to(torch.bfloat16)}
        o, n, kept = ops.block_norm(r, y, keep="e4m3", **args)
        grads = ops.block_norm_backward(r, y, o, kept, **args)
        for name, x in zip(("out", "normed", "codes", "scales", "dr", "dy", "dpost", "dpre", "dgate"),
                           (o, n, kept.data[:, :H], kept.scales[:, :(H + 31) // 32], *grads)):
            out[f"norm {T} {H} {name}"] = x
        kept = ops.checkpoint_encode(y)
        out[f"decoded {T} {H}"] = ops.checkpoint_decode(kept, torch.float32)
    for M, K, N in ((1, 64, 16), (150, 272, 208), (300, 512, 1040)):
        a, dy = (ops.quantize(normal(M, K).to(torch.bfloat16))[0] for _ in range(2))
        bg, bu, wd = (ops.quantize(normal(N, K).to(torch.bfloat16), two_d=True)[0] for _ in range(3))
        for keep in ("bf16", "e4m3"):
            h, gate, up = ops.gemm_gated(a, bg, bu, keep=keep)
            out[f"gated {M} {keep} h"] = h
            out[f"gated {M} {keep} gate"] = gate.data[:, :N]
            if keep == "e4m3":
                out[f"gated {M} scales"] = up.scales[:, :(N + 31) // 32]
            out[f"gated {M} {keep} dgu"] = ops.gemm_gated_backward(dy, wd, gate, up)
    torch.cuda.synchronize()
    return out


def violations():
    st, n = capi.nvfp4_testing_bounds_violations()
    assert st == capi.NVFP4_OK, capi.status_string(st)
    return n


def main():
    capi.load(build.build(debug=True))
    want = torch.load(sys.argv[1], weights_only=True)
    assert violations() == 0
    got = results()
    assert violations() == 0, "stores outside the declared ranges"
    assert ops.device_error() == capi.NVFP4_OK
    assert set(got) == set(want)
    for n, x in got.items():
        assert torch.equal(x.cpu(), want[n]), n
    capi.check(capi.nvfp4_testing_bounds_shrink(16))
    results()
    n = violations()
    capi.check(capi.nvfp4_testing_bounds_shrink(0))
    assert n > 0, "the shortened ranges produced no skipped store"
    print("block bounds check: clean in every mode, fires on shortened ranges")


if __name__ == "__main__":
    main()
