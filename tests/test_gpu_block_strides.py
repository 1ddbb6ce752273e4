"""Layouts of the feed-forward operators that the C interface allows and the
wrappers do not make themselves: gate and up kept in BF16 in wider memory,
dgate and dup as two matrices, a kept branch in wider memory, FP32 rows a
multiple of 16 bytes apart, no residual_out, and every call on a stream that is
handed to it.  All are the same values as in the plain layout."""
import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests.test_gpu_block_norm import _inputs
from tests.test_gpu_gemm_gated import _case

pytestmark = pytest.mark.gpu

FILL = 77


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


class Frame:
    """A [rows, cols] matrix inside a larger one of FILLs, `left` columns from its left end."""

    def __init__(self, rows, cols, dtype, left, right):
        self.whole = torch.full((rows + 2, left + cols + right), FILL, dtype=dtype, device="cuda")
        self.part = self.whole[1:-1, left:left + cols]
        self.left, self.cols = left, cols

    def holds(self, want):
        """The matrix is `want` and nothing around it was written."""
        w, a, b = self.whole, self.left, self.left + self.cols
        around = (w[[0, -1]] == FILL).all() and (w[:, :a] == FILL).all() and (w[:, b:] == FILL).all()
        return bool(around) and torch.equal(self.part, want)


@pytest.mark.parametrize("M,K,N", [(1, 64, 16), (150, 272, 208), (300, 64, 1040)])
@pytest.mark.parametrize("stream", [False, True])
def test_gated_products(M, K, N, stream):
    a, bg, bu, dy, wd = _case(M, K, N, 3)
    h, gate, up = ops.gemm_gated(a, bg, bu, keep="bf16")
    dgu = ops.gemm_gated_backward(dy, wd, gate, up)
    side = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    # (each with a leading dimension of its own)
    hf, gf, uf = (Frame(M, N, torch.bfloat16, 8 * i, 8 * (3 - i)) for i in (1, 2, 3))
    df, ef = Frame(M, N, torch.bfloat16, 24, 0), Frame(M, N, torch.bfloat16, 0, 40)
    if side is not None:
        side.wait_stream(torch.cuda.current_stream())   # (the frames are filled on the current one)
    handle = ops.stream_handle(side)
    g, u = (capi.nvfp4_checkpoint(f.part.data_ptr(), f.part.stride(0), None, 0) for f in (gf, uf))
    capi.check(capi.nvfp4_gemm_gated(a.struct(), bg.struct(), bu.struct(), 0, hf.part.data_ptr(), hf.part.stride(0), g, u,
                                     None, 0, handle))
    capi.check(capi.nvfp4_gemm_gated_backward(dy.struct(), wd.struct(), 0, g, u, df.part.data_ptr(), df.part.stride(0),
                                              ef.part.data_ptr(), ef.part.stride(0), None, 0, handle))
    if side is not None:
        again = torch.empty_like(dgu)
        side.wait_stream(torch.cuda.current_stream())
        ops.gemm_gated_backward(dy, wd, gate, up, out=again, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(again, dgu)
    torch.cuda.synchronize()
    assert hf.holds(h) and gf.holds(gate.data[:, :N]) and uf.holds(up.data[:, :N])
    assert df.holds(dgu[:, :N]) and ef.holds(dgu[:, N:])


@pytest.mark.parametrize("T,H", [(3, 8), (70, 264), (33, 3080)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_norms_around_a_block(T, H, kind):
    s = _inputs(T, H, kind, True, "token", True, T)
    args = {n: s[n] for n in ("post_weight", "pre_weight", "gate")}
    out, normed, kept = ops.block_norm(s["residual"], s["branch"], keep="e4m3", **args)
    grads = ops.block_norm_backward(s["dresidual_out"], s["dnormed"], out, kept, **args)
    step = 16 // s["residual"].element_size()   # 16 bytes

    def framed(x, i, unit):
        f = Frame(x.shape[0], x.shape[1], x.dtype, unit * i, unit * (5 - i))
        f.part.copy_(x)
        return f

    r, y, gate = framed(s["residual"], 1, step), framed(s["branch"], 2, 8), framed(s["gate"], 3, 8)
    of, nf = (Frame(T, H, k, u, 3 * u) for k, u in ((kind, step), (torch.bfloat16, 8)))
    blocks = (H + 31) // 32
    cf, sf = Frame(T, H, torch.uint8, 16, -H % 16), Frame(T, blocks, torch.uint8, 32, 64 - blocks % 16)
    desc = ops._block_norm_desc(T, H, kind, s["post_weight"], s["pre_weight"], gate.part, 1.0, 1e-6)
    where = capi.nvfp4_checkpoint(cf.part.data_ptr(), cf.part.stride(0), sf.part.data_ptr(), sf.part.stride(0))

    def at(f):
        return f.part.data_ptr(), f.part.stride(0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    capi.check(capi.nvfp4_block_norm(desc, *at(r), *at(y), *at(of), *at(nf), where, ops.stream_handle(side)))
    torch.cuda.synchronize()
    assert of.holds(out) and nf.holds(normed) and cf.holds(kept.data[:, :H]) and sf.holds(kept.scales[:, :blocks])
    # the norm alone
    nf.part.fill_(FILL)
    capi.check(capi.nvfp4_block_norm(desc, *at(r), *at(y), None, 0, *at(nf), None, ops.stream_handle()))
    assert nf.holds(normed) and of.holds(out)
    do, dn = framed(s["dresidual_out"], 2, step), framed(s["dnormed"], 1, 8)
    dr, db, dg = (Frame(T, H, k, u, 2 * u) for k, u in ((kind, step), (torch.bfloat16, 16), (torch.bfloat16, 8)))
    side.wait_stream(torch.cuda.current_stream())
    got = ops.block_norm_backward(do.part, dn.part, of.part, ops.Checkpoint(cf.part, sf.part, T, H),
                                  post_weight=s["post_weight"], pre_weight=s["pre_weight"], gate=gate.part,
                                  dresidual=dr.part, dbranch=db.part, dgate=dg.part, stream=side)
    torch.cuda.synchronize()
    assert dr.holds(grads.dresidual) and db.holds(grads.dbranch) and dg.holds(grads.dgate)
    assert torch.equal(got.dpost_weight, grads.dpost_weight) and torch.equal(got.dpre_weight, grads.dpre_weight)


def test_checkpoints_on_a_stream_that_is_handed_over():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(500, 1000, generator=g, device="cuda").to(torch.bfloat16)
    want = ops.checkpoint_decode(ops.checkpoint_encode(x), torch.float32)
    side = torch.cuda.Stream()
    kept, y = ops.alloc_checkpoint(500, 1000), torch.empty_like(want)
    side.wait_stream(torch.cuda.current_stream())
    ops.checkpoint_encode(x, out=kept, stream=side)
    ops.checkpoint_decode(kept, out=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
