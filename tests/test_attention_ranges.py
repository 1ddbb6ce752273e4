"""Scales and caps at the ends of what the constants made of them hold."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import attention_reference as ref

A16 = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return capi.load()


@pytest.mark.parametrize("backward", [False, True])
def test_refusals(backward):
    h, bad = capi.nvfp4_heads(A16, 512, 64), capi.nvfp4_heads(A16, 0, 64)   # a stride that is refused once the scalars are taken

    def status(scale, softcap):
        d = capi.nvfp4_attention_desc(64, 8, 4, 64, scale, softcap, None, A16)
        if backward:
            return capi.nvfp4_attention_backward(d, bad, h, h, h, bad, A16, h, h, h, A16, 1 << 30, None)
        return capi.nvfp4_attention(d, bad, h, h, h, A16, None)

    for scale in (2.0 ** 127, 3e38):              # times log2 e, which the scores are held in, it overflows
        for softcap in (0.0, 30.0):
            assert status(scale, softcap) == capi.NVFP4_ERR_INVALID_ARG, (scale, softcap)
    for scale, softcap in ((0.125, 0.0), (0.125, 30.0), (1e-38, 0.0), (1e-38, 10.0), (2.0 ** 126, 0.0), (0.125, 3.4e38), (0.125, 1e-45)):
        assert status(scale, softcap) == capi.NVFP4_ERR_SHAPE, (scale, softcap)


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1e-45, 1e-40, 2.0 ** -90, 1e-6, 1e6, 1e19, 1e20, 1e38, 3.4e38])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_far_from_the_scores(softcap, D):
    """Scores that are all at the cap, and scores that the cap leaves as they are; some products are 0."""
    T = 200
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, do = ((torch.randn((T, h, D), generator=g, device="cuda") * std).to(torch.bfloat16)
                   for h, std in ((4, 1.2), (2, 1.2), (2, 1.0), (4, 0.02)))
    q[7], k[5], k[140] = 0, 0, 0
    spans = ops.attention_spans(torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)
    o, lse = ops.attention(q, k, v, spans, softcap=softcap)
    grads = ops.attention_backward(do, q, k, v, o, lse, spans, softcap=softcap)
    r = ref.attention(q.double(), k.double(), v.double(), spans.long(), D ** -0.5, softcap, None, do.double())
    for name, got in zip(("o", "dq", "dk", "dv"), (o, *grads)):
        assert ((got.double() - r[name]).abs() <= r[name + "_tol"] + 1e-30).all(), name
    assert ((lse.double() - r["lse"]).abs() <= 2e-5 * (1 + r["lse"].abs())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-35, 1e-20, 1.0])
def test_small_scales(scale):
    T, D = 150, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((T, 2, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    spans = ops.attention_spans(torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)
    o, lse = ops.attention(q, k, v, spans, scale=scale)
    r = ref.attention(q.double(), k.double(), v.double(), spans.long(), scale)
    assert ((o.double() - r["o"]).abs() <= r["o_tol"] + 1e-30).all()
    assert ((lse.double() - r["lse"]).abs() <= 2e-5 * (1 + r["lse"].abs())).all()
