"""The attention and norm/rotation entry points in the library's debug build
(NVFP4_BOUNDS_CHECK): run by tests/test_gpu_attention_bounds.py in a process of
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

    def bf16(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    for T, HQ, HKV, D, cap, bias in ((1, 3, 3, 40, 0.0, False), (131, 4, 2, 72, 9.0, True), (300, 5, 1, 64, 0.0, False),
                                     (700, 2, 1, 128, 0.0, False)):
        q, k, v, do = bf16(T, HQ, D), bf16(T, HKV, D), bf16(T, HKV, D), bf16(T, HQ, D)
        slopes = torch.rand(HQ, generator=g, device="cuda") if bias else None
        offsets = torch.tensor([0, T // 3, T - T // 7], dtype=torch.int32, device="cuda")
        spans = ops.attention_spans(offsets, T, prefix=torch.tensor([2, 5], dtype=torch.int32, device="cuda"))
        o, lse = ops.attention(q, k, v, spans, softcap=cap, slopes=slopes)
        grads = ops.attention_backward(do, q, k, v, o, lse, spans, softcap=cap, slopes=slopes)
        for n, x in zip(("spans", "o", "lse", "dq", "dk", "dv"), (spans, o, lse, *grads)):
            out[f"attention {T} {D} {n}"] = x
        rot = 16 * (D // 32)
        qkv = bf16(T, (HQ + 2 * HKV) * D)
        cos, sin = ops.rope_tables(50, rot)
        w = torch.rand(2, D, generator=g, device="cuda")
        pos = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32)
        for inter in (False, True):
            a = (qkv, w[0].contiguous(), w[1].contiguous(), cos, sin, pos)
            r = ops.qk_norm_rope(*a, q_heads=HQ, kv_heads=HKV, interleaved=inter)
            r += ops.qk_norm_rope_backward(do, k, *a, interleaved=inter)
            for n, x in zip(("q", "k", "dqkv", "dwq", "dwk"), r):
                out[f"norm {T} {D} {inter} {n}"] = x
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
    print("attention bounds check: clean in every mode, fires on shortened ranges")


if __name__ == "__main__":
    main()
