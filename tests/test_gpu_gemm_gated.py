"""The gated pair of products and its backward pass against the 64-bit form on
the operands' decoded values.

Bounds: the products carry the documented bound of the GEMM (1e-4 sum |a b| +
1e-6), passed on through the formulas (|act'| <= 1.13).  The sigmoid's error:
e^-p with an argument rounded to 24 bits is off by at most (|p| + 2) 2^-22,
|p| < 89 before it leaves the type: 2^-15 of s or of 1 - s, 2^-14 with the
operations around it (FA).  Each result is rounded once: 2^-8 of its value,
2^-4 (or half the smallest code's step) in 8 bits."""
import math
import time

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops

pytestmark = pytest.mark.gpu

U, FA, TINY = 2.0 ** -8, 2.0 ** -14, 1e-30
REL, ABS = 1e-4, 1e-6
MASK = 0x3C5A


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _operand(rows, cols, seed, size=1.0, two_d=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * size
    pad = torch.zeros(-rows % 16, cols, device="cuda")   # 16x16 tiles take whole 16 rows
    q, _ = ops.quantize(torch.cat([x, pad]).to(torch.bfloat16), two_d=two_d)
    return _rows(q, rows)


def _rows(q, rows):
    return ops.NVFP4Operand(q.codes[:rows], q.scales, q.amax, q.global_scale, rows, q.cols)


def _product(a, b):
    """(A B^T in 64 bits, its bound)."""
    x, y = ops.dequantize(a).double(), ops.dequantize(b).double()
    return x @ y.t(), REL * (x.abs() @ y.abs().t()) + ABS


def _act(g, kind):
    """(act, act', the size of act' 's terms)."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), s + (g * s).abs()
    c, k = math.sqrt(2 / math.pi), 0.044715
    s = torch.sigmoid(2 * c * (g + k * g ** 3))
    slope = 2 * c * (1 + 3 * k * g ** 2)
    far = g.abs() > 14          # s is 0 or 1 to far beyond FP32
    return g * s, s + torch.where(far, 0.0, g * s * (1 - s) * slope), s + torch.where(far, 0.0, (g * s * slope).abs())


def _check_forward(a, bg, bu, h, kind):
    (g, ge), (u, ue) = _product(a, bg), _product(a, bu)
    f, _, _ = _act(g, kind)
    want = f * u
    # |act| <= |g|, |act'| <= 1.13; the errors' product too
    tol = 1.13 * ge * (u.abs() + ue) + f.abs() * ue + FA * want.abs() + U * (want.abs() + 1.13 * ge * u.abs() + f.abs() * ue)
    assert ((h.double() - want).abs() <= tol + TINY).all()
    return (g, ge), (u, ue)


def _values(kept):
    return (kept.data[:, :kept.cols] if kept.scales is None else ops.checkpoint_decode(kept, torch.float32)).double()


def _check_kept(kept, value, error):
    got = _values(kept)
    if kept.scales is None:
        tol = error + U * (value.abs() + error)
    else:
        b = kept.scales[:, :(kept.cols + 31) // 32].double().repeat_interleave(32, 1)[:, :kept.cols]
        tol = error + 2.0 ** -4 * (value.abs() + error) + torch.exp2(b - 137)
        # the scale is the smallest that takes the block: codes reach past half of the largest
        n = kept.cols // 32 * 32
        codes = kept.data[:, :n].reshape(kept.rows, n // 32, 32).view(torch.float8_e4m3fn).float().abs().amax(-1)
        assert ((codes > 216) | (kept.scales[:, :n // 32] == 10)).all()
    assert ((got - value).abs() <= tol + TINY).all()


def _check_backward(dy, wd, gate, up, dgu, kind):
    dh, e = _product(dy, wd)
    g, u = _values(gate), _values(up)
    f, df, dsize = _act(g, kind)
    n = g.shape[1]
    for got, factor, size in ((dgu[:, :n], u * df, (u * dsize).abs()), (dgu[:, n:], f, f.abs())):
        want = dh * factor
        tol = e * factor.abs() + FA * (dh.abs() + e) * size
        assert ((got.double() - want).abs() <= (1 + U) * tol + U * want.abs() + TINY).all()


def _case(M, K, N, seed=0, size=1.0):
    return (_operand(M, K, seed, size), _operand(N, K, seed + 1, 0.05, True), _operand(N, K, seed + 2, 0.05, True),
            _operand(M, K, seed + 3, 1e-3), _operand(N, K, seed + 4, 0.05, True))


SIZES = [(1, 16, 16), (1, 3072, 9216), (2, 64, 48), (16, 256, 128), (127, 272, 144), (129, 1040, 1056), (300, 64, 4112),
         (513, 3088, 240), (1000, 512, 1040), (4100, 128, 2064)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_sizes(M, K, N, kind):
    a, bg, bu, dy, wd = _case(M, K, N, M + K + N)
    plain, none, _ = ops.gemm_gated(a, bg, bu, activation=kind)
    assert none is None
    for keep in ("bf16", "e4m3"):
        h, gate, up = ops.gemm_gated(a, bg, bu, activation=kind, keep=keep)
        assert torch.equal(h, plain)
        (g, ge), (u, ue) = _check_forward(a, bg, bu, h, kind)
        _check_kept(gate, g, ge)
        _check_kept(up, u, ue)
        dgu = ops.gemm_gated_backward(dy, wd, gate, up, activation=kind)
        assert dgu.shape == (M, 2 * N)
        _check_backward(dy, wd, gate, up, dgu, kind)
    assert ops.device_error() == capi.NVFP4_OK


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_far_gates(kind):
    """Gates of thousands and 1e30, of both signs: the sigmoid at its ends, GELU's cube past the type."""
    for size in (300.0, 1e15, 1e30):
        a, bg, bu, dy, wd = _case(64, 256, 160, 5, size)
        bu = _operand(160, 256, 7, 0.05 / size, True)
        for keep in ("bf16", "e4m3"):
            h, gate, up = ops.gemm_gated(a, bg, bu, activation=kind, keep=keep)
            _check_forward(a, bg, bu, h, kind)
            _check_backward(dy, wd, gate, up, ops.gemm_gated_backward(dy, wd, gate, up, activation=kind), kind)


def test_gates_past_the_type_are_kept_as_nan():
    """Gates around FP32's end: what overflows is kept as NaN and leaves its block's scale to the others, what
    reaches 2^127 takes the last scale."""
    a, bg, bu = _operand(64, 256, 5, 3e37), _operand(160, 256, 6, 0.5), _operand(160, 256, 7, 1e-30)   # (finite in bf16)
    _, gate, _ = ops.gemm_gated(a, bg, bu, keep="e4m3")
    (g, ge), got = _product(a, bg), _values(gate)
    limit = float(torch.finfo(torch.float32).max)
    over, under = g.abs() - ge > limit, g.abs() + ge < limit
    assert over.any() and (g.abs() > 2.0 ** 127)[under].any()
    assert torch.isnan(got[over]).all() and torch.isfinite(got[under]).all()
    # 1.875 2^127 stands for what would round to 2^128
    want = g.clamp(-1.875 * 2.0 ** 127, 1.875 * 2.0 ** 127)
    b = gate.scales[:, :5].double().repeat_interleave(32, 1)
    tol = ge + 2.0 ** -4 * (want.abs() + ge) + torch.exp2(b - 137)
    assert ((got - want).abs() <= tol)[under].all()


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_a_nan_that_is_kept_stays_alone(keep):
    _, _, _, dy, wd = _case(70, 128, 112, 8)
    g = torch.Generator(device="cuda").manual_seed(9)
    x, y = (torch.randn(70, 112, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    kept = (lambda t: t) if keep == "bf16" else ops.checkpoint_encode
    clean = ops.gemm_gated_backward(dy, wd, kept(x), kept(y))
    x[3, 40], y[69, 111] = float("nan"), float("nan")
    dgu = ops.gemm_gated_backward(dy, wd, kept(x), kept(y))
    bad = torch.zeros_like(dgu, dtype=torch.bool)
    bad[3, 40] = bad[3, 152] = bad[69, 111] = True
    assert torch.isnan(dgu[bad]).all()
    if keep == "bf16":   # (in 8 bits the block's other values may have another scale)
        assert torch.equal(dgu[~bad], clean[~bad])
    assert torch.isfinite(dgu[~bad]).all()


def test_zeros():
    a, bg, bu, dy, wd = _case(48, 256, 96)
    zero = _operand(48, 256, 0, 0.0)
    h, gate, up = ops.gemm_gated(zero, bg, bu, keep="e4m3")
    assert (h == 0).all() and (_values(gate) == 0).all()
    assert (ops.gemm_gated_backward(dy, wd, gate, up) == 0).all()
    h, gate, up = ops.gemm_gated(a, bg, bu, keep="bf16")
    assert (ops.gemm_gated_backward(zero, wd, gate, up) == 0).all()


@pytest.mark.parametrize("M,K,N", [(16, 64, 32), (272, 512, 400), (1024, 1024, 1152)])
def test_amaxes_feed_the_quantizer(M, K, N):
    a, bg, bu, dy, wd = _case(M, K, N, 11)
    amax = torch.full((2,), 9e9, device="cuda")
    h, gate, up = ops.gemm_gated(a, bg, bu, keep="e4m3", amax=amax, rht_mask=MASK)
    assert torch.equal(h, ops.gemm_gated(a, bg, bu)[0])
    dmax = torch.full((2,), 9e9, device="cuda")
    dgu = ops.gemm_gated_backward(dy, wd, gate, up, amax=dmax, rht_mask=MASK)
    assert torch.equal(dgu, ops.gemm_gated_backward(dy, wd, gate, up))
    for x, m in ((h, amax), (dgu, dmax)):
        row, col = ops.quantize_row_col_rht(x, MASK)
        assert m[0] == row.amax[0] and m[1] == col.amax[0]
        got = ops.quantize_row_col_rht_amax(x, MASK, m)
        for p, q in zip(got, (row, col)):
            n = p.cols // 2   # (the padding of a row is not written)
            assert torch.equal(p.codes[:, :n], q.codes[:, :n]) and torch.equal(p.scales, q.scales)


def test_amaxes_of_calls_in_a_row():
    """A large product and then a small one into the same two floats, without a wait between."""
    M, K, N = 512, 512, 768
    _, bg, bu, dy, wd = _case(M, K, N, 12)
    big, small = _operand(M, K, 13, 50.0), _operand(M, K, 14, 0.01)
    _, gate, up = ops.gemm_gated(small, bg, bu, keep="bf16")
    amax, dmax = (torch.empty(2, device="cuda") for _ in range(2))
    for _ in range(10):
        for a in (big, small):
            h, _, _ = ops.gemm_gated(a, bg, bu, amax=amax, rht_mask=MASK)
            dgu = ops.gemm_gated_backward(dy, wd, gate, up, amax=dmax, rht_mask=MASK)
        assert amax[0] == h.abs().max().float() and dmax[0] == dgu.abs().max().float()


def test_halves_of_one_weight_matrix():
    M, K, N = 200, 512, 384
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(2 * N, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    q, _ = ops.quantize(w, two_d=True)
    a = _operand(M, K, 4)
    gate, up = ops.operand_rows(q, 0, N), ops.operand_rows(q, N, 2 * N)
    x = ops.dequantize(q)
    assert torch.equal(ops.dequantize(gate), x[:N]) and torch.equal(ops.dequantize(up), x[N:])
    h, _, _ = ops.gemm_gated(a, gate, up)
    _check_forward(a, gate, up, h, "silu")
    # the gate as its own up projection, and one projection as both
    h, kept_g, kept_u = ops.gemm_gated(a, gate, gate, keep="bf16")
    assert torch.equal(kept_g.data, kept_u.data)
    with pytest.raises(ValueError):
        ops.operand_rows(q, 64, N)


def test_strides_and_what_lies_around():
    M, K, N = 150, 256, 208
    a, bg, bu, dy, wd = _case(M, K, N, 21)
    h, gate, up = ops.gemm_gated(a, bg, bu, keep="e4m3")
    want = ops.gemm_gated_backward(dy, wd, gate, up)
    wide = torch.full((M + 2, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.gemm_gated(a, bg, bu, out=wide[1:-1, 16:16 + N])
    assert torch.equal(wide[1:-1, 16:16 + N], h)
    assert (wide[[0, -1]] == 7).all() and (wide[:, :16] == 7).all() and (wide[:, 16 + N:] == 7).all()
    wide = torch.full((M + 2, 2 * N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.gemm_gated_backward(dy, wd, gate, up, out=wide[1:-1, 8:8 + 2 * N])
    assert torch.equal(wide[1:-1, 8:8 + 2 * N], want)
    assert (wide[[0, -1]] == 7).all() and (wide[:, :8] == 7).all() and (wide[:, 8 + 2 * N:] == 7).all()

    def place(x, fill):
        w = torch.full((M + 2, x.shape[1] + 48), fill, dtype=x.dtype, device="cuda")
        return w, w[1:-1, 16:16 + x.shape[1]]

    # kept into wider memory, and read from there
    wg, kg = zip(*(place(x, 77) for x in (gate.data, gate.scales)))
    wu, ku = zip(*(place(x, 77) for x in (up.data, up.scales)))
    views = [ops.Checkpoint(*k, M, N) for k in (kg, ku)]
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    capi.check(capi.nvfp4_gemm_gated(a.struct(), bg.struct(), bu.struct(), 0, out.data_ptr(), N, views[0].struct(),
                                     views[1].struct(), None, 0, ops.stream_handle()))
    n = (N + 31) // 32
    for w, kept in ((wg, gate), (wu, up)):
        assert torch.equal(w[0][1:-1, 16:16 + N], kept.data[:, :N]) and torch.equal(w[1][1:-1, 16:16 + n], kept.scales[:, :n])
        for x, m in zip(w, (N, n)):
            assert (x[[0, -1]] == 77).all() and (x[:, :16] == 77).all() and (x[:, 16 + m:] == 77).all()
    assert torch.equal(ops.gemm_gated_backward(dy, wd, *views), want)
    both = torch.cat([_values(gate), _values(up)], 1).to(torch.bfloat16)
    assert torch.equal(ops.gemm_gated_backward(dy, wd, both[:, :N], both[:, N:]), want)   # bf16 holds the codes' values


def test_offsets_past_32_bits():
    M, K, N = 3, 64, 64
    a, bg, bu, dy, wd = _case(M, K, N, 31)
    h, gate, up = ops.gemm_gated(a, bg, bu, keep="bf16")
    want = ops.gemm_gated_backward(dy, wd, gate, up)
    far = torch.empty(M, 2 ** 31 + 1024, dtype=torch.bfloat16, device="cuda")
    at = [far[:, 128 * i:128 * i + n] for i, n in enumerate((64, 64, 64, 128))]
    ops.gemm_gated(a, bg, bu, out=at[0])
    assert torch.equal(at[0], h)
    at[1].copy_(gate.data)
    at[2].copy_(up.data)
    assert torch.equal(ops.gemm_gated_backward(dy, wd, at[1], at[2], out=at[3]), want)


def test_equal_bits_streams_and_graph():
    M, K, N = 700, 1024, 1552
    a, bg, bu, dy, wd = _case(M, K, N, 41)

    def both():
        h, gate, up = ops.gemm_gated(a, bg, bu, keep="e4m3")
        return h, gate.data[:, :N], up.data[:, :N], ops.gemm_gated_backward(dy, wd, gate, up)

    want = both()
    # calls in a row over the same and other buffers, on two streams at once
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got.append(both())
        with torch.cuda.stream(side):
            got.append(both())
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(x, y) for x, y in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = both()
    for x in r:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(r, want))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradients_against_differences(kind):
    M, K, N = 64, 128, 96
    a, bg, bu, dy, wd = _case(M, K, N, 51)
    _, gate, up = ops.gemm_gated(a, bg, bu, activation=kind, keep="bf16")
    dgu = ops.gemm_gated_backward(dy, wd, gate, up, activation=kind).double()
    dh, e = _product(dy, wd)
    at = torch.cat([_values(gate), _values(up)], 1)
    u = torch.randn(at.shape, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda", dtype=torch.float64)

    def loss(x):
        return (dh * _act(x[:, :N], kind)[0] * x[:, N:]).sum()

    step = 1e-5
    slope = (loss(at + step * u) - loss(at - step * u)) / (2 * step)
    f, df, dsize = _act(at[:, :N], kind)
    size = torch.cat([(at[:, N:] * dsize).abs(), f.abs()], 1)
    tol = ((U * dgu.abs() + (2 * e.repeat(1, 2) + 2 * FA * dh.abs().repeat(1, 2)) * size) * u.abs()).sum()
    assert abs(slope - (dgu * u).sum()) <= tol + 1e-6 * (dgu * u).abs().sum()


def test_empty():
    a, bg, bu, dy, wd = _case(0, 64, 32)
    amax = torch.ones(2, device="cuda")
    h, gate, up = ops.gemm_gated(a, bg, bu, keep="e4m3", amax=amax, rht_mask=MASK)
    assert h.shape == (0, 32) and (amax == 0).all()
    assert ops.gemm_gated_backward(dy, wd, gate, up).shape == (0, 64)


@pytest.mark.parametrize("backward", [False, True])
def test_a_wait_runs_out_and_the_next_call_is_correct(backward):
    a, bg, bu, dy, wd = _case(256, 512, 512, 61)
    h, gate, up = ops.gemm_gated(a, bg, bu, keep="bf16")
    dgu = ops.gemm_gated_backward(dy, wd, gate, up)
    torch.cuda.synchronize()
    assert ops.device_error() == capi.NVFP4_OK

    def call(out):
        return ops.gemm_gated_backward(dy, wd, gate, up, out=out) if backward else ops.gemm_gated(a, bg, bu, out=out)[0]

    out = torch.full_like(dgu if backward else h, 7.0)
    capi.check(capi.nvfp4_testing_arm_gemm_timeout(20000), "arm")     # 20 ms per wait
    t0 = time.perf_counter()
    call(out)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.5
    assert ops.device_error() == capi.NVFP4_ERR_TIMEOUT and ops.device_error() == capi.NVFP4_OK
    # the CTA pair whose barrier waits writes nothing; every pair's is withheld
    assert (out == 7).all()
    assert torch.equal(call(None), dgu if backward else h)
    assert ops.device_error() == capi.NVFP4_OK
