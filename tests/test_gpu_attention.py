"""Attention forward and backward against the plain 64-bit form: masks, head
layouts, lengths around the tiles, caps and biases, strides, streams and what
masked places hold."""
import math

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import attention_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _inputs(T, HQ, HKV, D, seed, std=1.2):
    g = _gen(seed)
    return _bf16(g, T, HQ, D, std=std), _bf16(g, T, HKV, D, std=std), _bf16(g, T, HKV, D), _bf16(g, T, HQ, D, std=0.02)


def _spans(rows):
    return torch.tensor(rows, dtype=torch.int32, device="cuda").reshape(-1, 2)


def _causal(T):
    return _spans([(0, i + 1) for i in range(T)])


def _within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = ((got - want).abs() - tol - 1e-30).max().item()
    assert worst <= 0, f"{what}: {worst} over its bound"


def _check(q, k, v, do, spans, softcap=0.0, slopes=None, scale=None, backward=True):
    T, HQ, D = q.shape
    sc = D ** -0.5 if scale is None else scale
    o, lse = ops.attention(q, k, v, spans, scale=scale, softcap=softcap, slopes=slopes)
    r = ref.attention(q.double(), k.double(), v.double(), spans.long(), sc, softcap,
                      None if slopes is None else slopes.double(), do.double() if backward else None)
    _within(o, r["o"], r["o_tol"], "out")
    empty = r["lse"] == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    off = (lse.double() - r["lse"]).abs()[~empty]
    assert not off.numel() or (off <= 2e-5 * (1 + r["lse"][~empty].abs())).all(), off.max()
    if backward:
        dq, dk, dv = ops.attention_backward(do, q, k, v, o, lse, spans, scale=scale, softcap=softcap, slopes=slopes)
        for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
            _within(got, r[name], r[name + "_tol"], name)
    torch.cuda.synchronize()
    assert ops.device_error() == capi.NVFP4_OK
    return o, lse


@pytest.mark.parametrize("T", [1, 2, 31, 64, 127, 128, 129, 255, 257, 385, 640])
@pytest.mark.parametrize("D", [64, 128])
def test_causal_lengths(T, D):
    _check(*_inputs(T, 4, 2, D, T), _causal(T))


@pytest.mark.parametrize("HQ,HKV", [(1, 1), (3, 3), (5, 1), (6, 2), (24, 12)])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 96, 120, 128])
def test_heads_and_dims(HQ, HKV, D):
    _check(*_inputs(200, HQ, HKV, D, HQ + D), _causal(200))


@pytest.mark.parametrize("softcap,bias", [(5.0, False), (30.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("T,D", [(77, 64), (300, 128), (300, 80)])
def test_cap_and_bias(softcap, bias, T, D):
    slopes = torch.tensor([0.5, 0.1, 0.0, 2.0], device="cuda") if bias else None
    _check(*_inputs(T, 4, 2, D, T + D), _causal(T), softcap=softcap, slopes=slopes)


def test_scores_far_beyond_the_cap():
    q, k, v, do = _inputs(150, 2, 1, 64, 5)
    _check(q * 20, k * 20, v, do, _causal(150), softcap=10.0)


def test_large_scores_need_the_running_maximum():
    """Scores that grow along the keys, by far more than exp can hold: every
    tile raises the maximum."""
    T, D = 700, 64
    q, k, v, do = _inputs(T, 2, 1, D, 6, std=0.5)
    q[..., 0], k[..., 0] = 8.0, (torch.arange(T, device="cuda") / 8.0)[:, None].to(torch.bfloat16)
    _check(q, k, v, do, _spans([(0, T)] * T), scale=1.0)
    _check(q, k.flip(0), v, do, _spans([(0, T)] * T), scale=1.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("with_prefix", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_documents(causal, with_prefix, D):
    """Packed documents of lengths that start and end inside tiles, empty ones
    among them, padding before and after."""
    lengths = [1, 130, 0, 128, 77, 3, 0, 200, 256]
    offsets = [5]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    T = offsets[-1] + 41
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    pre = torch.tensor([n * 2 // 3 for n in lengths], dtype=torch.int32, device="cuda") if with_prefix else None
    spans = ops.attention_spans(off, T, causal=causal, prefix=pre)
    want = [(0, 0)] * T
    for d, n in enumerate(lengths):
        for i in range(offsets[d], offsets[d] + n):
            hi = max(i + 1, offsets[d] + (n * 2 // 3 if with_prefix else 0)) if causal else offsets[d + 1]
            want[i] = (offsets[d], hi)
    assert torch.equal(spans, _spans(want))
    o, lse = _check(*_inputs(T, 4, 2, D, 9), spans)
    pad = torch.tensor([w == (0, 0) for w in want], device="cuda")
    assert (o[pad] == 0).all() and (lse[:, pad] == -math.inf).all()


def test_spans_of_no_documents_and_bad_offsets():
    none = ops.attention_spans(torch.zeros(1, dtype=torch.int32, device="cuda"), 10)
    assert (none == 0).all()
    # offsets past the tokens are cut
    s = ops.attention_spans(torch.tensor([0, 50], dtype=torch.int32, device="cuda"), 20, causal=False)
    assert torch.equal(s, _spans([(0, 20)] * 20))


@pytest.mark.parametrize("D", [64, 128])
def test_rows_with_nothing_and_arbitrary_intervals(D):
    """Intervals that no mask of documents gives: empty rows between others,
    windows, rows that see only the future, ends outside [0, tokens)."""
    T = 420
    g = torch.Generator().manual_seed(3)
    rows = []
    for i in range(T):
        kind = int(torch.randint(0, 6, (1,), generator=g))
        a, b = sorted(torch.randint(0, T + 1, (2,), generator=g).tolist())
        rows.append([(0, 0), (a, b), (max(0, i - 40), i + 1), (i, T + 7), (-5, i // 2), (b, a)][kind])
    _check(*_inputs(T, 3, 3, D, 12), _spans(rows))


def test_all_rows_empty():
    T = 300
    q, k, v, do = _inputs(T, 2, 1, 64, 2)
    spans = torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    o, lse = ops.attention(q, k, v, spans)
    grads = ops.attention_backward(do, q, k, v, o, lse, spans)
    assert (o == 0).all() and (lse == -math.inf).all()
    assert all((x == 0).all() for x in grads)


@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_masked_places_may_hold_anything(junk, D):
    """Padding rows of every input hold NaN, infinities or the type's largest
    values: nothing of it reaches a result."""
    T, first, end = 333, 19, 290
    q, k, v, do = _inputs(T, 4, 2, D, 21)
    pad = torch.ones(T, dtype=torch.bool, device="cuda")
    pad[first:end] = False
    clean = [x.clone() for x in (q, k, v, do)]
    for x in (q, k, v, do):
        x[pad] = junk
    off = torch.tensor([first, 100, end], dtype=torch.int32, device="cuda")
    for causal in (True, False):
        spans = ops.attention_spans(off, T, causal=causal)
        o, lse = ops.attention(q, k, v, spans)
        o2, lse2 = ops.attention(*clean[:3], spans)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        got = ops.attention_backward(do, q, k, v, o, lse, spans)
        want = ops.attention_backward(clean[3], *clean[:3], o2, lse2, spans)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
            assert torch.isfinite(a).all()


def test_strided_views_and_given_outputs():
    """q, k, v as columns of one matrix and in [heads][tokens] order, outputs
    into views whose surroundings keep their values."""
    T, HQ, HKV, D = 201, 4, 2, 64
    g = _gen(8)
    qkv = _bf16(g, T, (HQ + 2 * HKV) * D + 16)
    q = qkv[:, :HQ * D].unflatten(1, (HQ, D))
    k = _bf16(g, HKV, T, D).transpose(0, 1)
    v = qkv[:, (HQ + HKV) * D:(HQ + 2 * HKV) * D].unflatten(1, (HKV, D))
    do = _bf16(g, T, HQ, D)
    spans = _causal(T)
    o, lse = ops.attention(q, k, v, spans)
    want = ops.attention(q.contiguous(), k.contiguous(), v.contiguous(), spans)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    grads = ops.attention_backward(do, q.contiguous(), k.contiguous(), v.contiguous(), o, lse, spans)
    dqkv = torch.full_like(qkv, 7.0)
    dv = dqkv[:, (HQ + HKV) * D:(HQ + 2 * HKV) * D].unflatten(1, (HKV, D))
    dq = torch.empty((HQ, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    out = torch.full((T, HQ + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.attention(q, k, v, spans, out=out[:, :HQ])
    assert torch.equal(out[:, :HQ], o) and (out[:, HQ:] == 7.0).all()
    got = ops.attention_backward(do, q, k, v, out[:, :HQ], lse, spans, dq=dq, dv=dv)
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    assert (dqkv[:, :(HQ + HKV) * D] == 7.0).all() and (dqkv[:, (HQ + 2 * HKV) * D:] == 7.0).all()


def test_equal_inputs_give_equal_bits():
    q, k, v, do = _inputs(900, 6, 2, 128, 31)
    spans = _causal(900)
    first = None
    for _ in range(4):
        o, lse = ops.attention(q, k, v, spans, softcap=20.0)
        got = (o, lse, *ops.attention_backward(do, q, k, v, o, lse, spans, softcap=20.0))
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_other_stream_and_graph():
    q, k, v, do = _inputs(300, 4, 2, 64, 41)
    spans = _causal(300)
    o, lse = ops.attention(q, k, v, spans)
    want = (o, lse, *ops.attention_backward(do, q, k, v, o, lse, spans))
    ws = torch.empty(capi.nvfp4_attention_backward_workspace_size(300, 4, 2, 64), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(x) for x in want]

    def step(stream):
        ops.attention(q, k, v, spans, out=outs[0], lse=outs[1], stream=stream)
        ops.attention_backward(do, q, k, v, outs[0], outs[1], spans, dq=outs[2], dk=outs[3], dv=outs[4],
                               workspace=ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    for x in outs:
        x.zero_()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("softcap,bias", [(0.0, False), (8.0, True)])
def test_gradients_against_differences(softcap, bias):
    """The directional derivative of sum(out * dout) along random directions,
    by central differences of the 64-bit form, against the kernel's gradients;
    the bound is the gradients' own, summed along the direction."""
    T, HQ, HKV, D = 150, 4, 2, 64
    q, k, v, do = _inputs(T, HQ, HKV, D, 51)
    slopes = torch.tensor([0.3, 0.1, 0.05, 0.0], device="cuda") if bias else None
    spans = _causal(T)
    o, lse = ops.attention(q, k, v, spans, softcap=softcap, slopes=slopes)
    grads = ops.attention_backward(do, q, k, v, o, lse, spans, softcap=softcap, slopes=slopes)
    x = [t.double() for t in (q, k, v)]
    sl = None if slopes is None else slopes.double()
    r = ref.attention(*x, spans.long(), D ** -0.5, softcap, sl, do.double())
    g = _gen(52)
    eps = 1e-5
    for n, grad in enumerate(grads):
        u = torch.randn(x[n].shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(t):
            y = list(x)
            y[n] = y[n] + t * u
            return (ref.attention(*y, spans.long(), D ** -0.5, softcap, sl)["o"] * do.double()).sum()

        slope = (loss(eps) - loss(-eps)) / (2 * eps)
        name = ("dq", "dk", "dv")[n]
        assert abs(slope - (r[name] * u).sum()) <= 1e-6 * (r[name] * u).abs().sum()
        assert abs(slope - (grad.double() * u).sum()) <= (r[name + "_tol"] * u.abs()).sum()


@pytest.mark.parametrize("T,HQ,HKV,D,softcap", [(2048, 4, 2, 128, 0.0), (3001, 2, 2, 64, 30.0), (1537, 8, 2, 96, 0.0)])
def test_longer_sequences(T, HQ, HKV, D, softcap):
    _check(*_inputs(T, HQ, HKV, D, T), _causal(T), softcap=softcap)


@pytest.mark.parametrize("HQ,HKV,D", [(40, 20, 64), (40, 20, 128), (36, 6, 40), (33, 33, 96)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_tiles_per_sm(HQ, HKV, D, causal):
    """More tiles than SMs several times over, with documents from one token to
    many tiles, whole tiles of padding among them: what one tile leaves behind
    for the next on the same SM must not show, whatever their lengths.  Run
    three times over changing inputs, the repeats equal bit for bit."""
    lengths = [1, 3, 600, 1, 127, 130, 260, 40, 1, 1, 300, 5, 128, 128]
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    T = offsets[-1] + 300
    spans = ops.attention_spans(torch.tensor(offsets, dtype=torch.int32, device="cuda"), T, causal=causal)
    first, other = _inputs(T, HQ, HKV, D, D), _inputs(T, HQ, HKV, D, D + 1)

    def step(q, k, v, do):
        o, lse = ops.attention(q, k, v, spans)
        return (o, lse, *ops.attention_backward(do, q, k, v, o, lse, spans))

    want = step(*first)
    for _ in range(3):
        step(*other)
        again = step(*first)
        assert all(torch.equal(a, b) for a, b in zip(again, want))
    _check(*first, spans)


@pytest.mark.parametrize("T,HQ,HKV,D", [(1, 4, 2, 64), (150, 8, 2, 64), (700, 8, 4, 128), (2100, 24, 12, 128)])
def test_calls_in_a_row_over_the_same_buffers(T, HQ, HKV, D):
    """Kernels start under the tail of the one before: every call reads what the
    call before wrote, and overwrites what the one before that read.  The last
    step's results equal those of steps with the device idle between the calls."""
    g = _gen(31)
    qkvs = [_bf16(g, T, (HQ + 2 * HKV) * D) for _ in range(3)]
    douts = [_bf16(g, T, HQ, D, std=0.02) for _ in range(3)]
    wq, wk = (torch.rand(D, generator=g, device="cuda") + 0.5 for _ in range(2))
    cos, sin = ops.rope_tables(T, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    spans = ops.attention_spans(torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda"), T)
    new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k, o, lse = new(T, HQ, D), new(T, HKV, D), new(T, HQ, D), torch.empty((HQ, T), device="cuda")
    dq, dk, dqkv = new(T, HQ, D), new(T, HKV, D), new(T, (HQ + 2 * HKV) * D)
    size = capi.nvfp4_attention_backward_workspace_size(T, HQ, HKV, D)
    size = max(size, capi.nvfp4_qk_norm_rope_backward_workspace_size(D))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step(i, idle):
        wait = torch.cuda.synchronize if idle else (lambda: None)
        qkv, do = qkvs[i % 3], douts[i % 3]
        v = qkv.view(T, HQ + 2 * HKV, D)[:, HQ + HKV:]
        wait()
        ops.qk_norm_rope(qkv, wq, wk, cos, sin, pos, q_heads=HQ, kv_heads=HKV, out_q=q, out_k=k)
        wait()
        ops.attention(q, k, v, spans, out=o, lse=lse)
        wait()
        ops.attention_backward(do, q, k, v, o, lse, spans, dq=dq, dk=dk,
                               dv=dqkv.view(T, HQ + 2 * HKV, D)[:, HQ + HKV:], workspace=ws)
        wait()
        dw = ops.qk_norm_rope_backward(dq, dk, qkv, wq, wk, cos, sin, pos, dqkv=dqkv, workspace=ws)[1:]
        wait()
        return [x.clone() for x in (q, k, o, lse, dq, dk, dqkv, *dw)]

    want = [step(i, True) for i in range(3)]
    for steps in (2, 3, 4, 12):
        for i in range(steps):
            got = step(i, False)
        for a, b in zip(got, want[(steps - 1) % 3]):
            assert torch.equal(a, b)


# Enough heads that there are more pairs of query tiles than SMs: an item is two
# tiles then (two heads that share their keys, or two tiles of one head), where
# the few heads of the tests above give one tile whose keys are split.
MANY_HEADS = [(128, 64, 64), (128, 64, 128), (100, 100, 64), (100, 100, 96), (69, 23, 128)]


@pytest.mark.parametrize("HQ,HKV,D", MANY_HEADS)
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (5.0, False), (0.0, True), (5.0, True)])
def test_pairs_of_tiles(HQ, HKV, D, softcap, bias):
    """Intervals that differ between the two tiles of an item, empty rows, ends
    outside [0, tokens), an odd number of tiles."""
    T = 700 if HQ == 69 else 330
    g = torch.Generator().manual_seed(4)
    rows = []
    for i in range(T):
        kind = int(torch.randint(0, 5, (1,), generator=g))
        a, b = sorted(torch.randint(0, T + 1, (2,), generator=g).tolist())
        rows.append([(0, 0), (a, b), (max(0, i - 40), i + 1), (i, T + 7), (-5, i // 2)][kind])
    slopes = torch.rand(HQ, generator=_gen(5), device="cuda") * 0.2 if bias else None
    _check(*_inputs(T, HQ, HKV, D, 14), _spans(rows), softcap=softcap, slopes=slopes)
    _check(*_inputs(T, HQ, HKV, D, 15), _causal(T), softcap=softcap, slopes=slopes)


@pytest.mark.parametrize("junk", [math.nan, -math.inf])
@pytest.mark.parametrize("HQ,HKV,D", MANY_HEADS)
def test_pairs_of_tiles_masked_places(junk, HQ, HKV, D):
    T, first, end = 700, 150, 600
    q, k, v, do = _inputs(T, HQ, HKV, D, 22)
    pad = torch.ones(T, dtype=torch.bool, device="cuda")
    pad[first:end] = False
    clean = [x.clone() for x in (q, k, v, do)]
    for x in (q, k, v, do):
        x[pad] = junk
    spans = ops.attention_spans(torch.tensor([first, 260, end], dtype=torch.int32, device="cuda"), T)
    o, lse = ops.attention(q, k, v, spans)
    o2, lse2 = ops.attention(*clean[:3], spans)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.isfinite(o).all()
    got = ops.attention_backward(do, q, k, v, o, lse, spans)
    want = ops.attention_backward(clean[3], *clean[:3], o2, lse2, spans)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and torch.isfinite(a).all()


def test_no_tokens():
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    spans = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    o, lse = ops.attention(q, k, k, spans)
    assert o.shape == q.shape and lse.shape == (4, 0)
    assert [x.shape[0] for x in ops.attention_backward(q, q, k, k, o, lse, spans)] == [0, 0, 0]
