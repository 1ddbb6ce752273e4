"""What attention does with NaN and infinities: in places that no row sees
they reach nothing, in places that a row sees they reach its result."""
import math

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi, ops
from tests import attention_reference as ref

pytestmark = pytest.mark.gpu

# (query heads, key heads, dims): few heads, whose tiles are split over their
# keys, and heads enough that an item is two heads of one tile, or two tiles of one head
SPLIT = [(4, 2, 64), (4, 2, 96), (3, 3, 128)]
PAIRS = [(128, 64, 64), (128, 64, 128), (100, 100, 96)]
JUNK = [math.nan, math.inf, -math.inf]
FORMS = [(5.0, False), (0.0, True), (5.0, True), (40.0, False)]


@pytest.fixture(scope="module", autouse=True)
def library():
    libbuild.build()
    capi.load()


def _inputs(T, HQ, HKV, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def bf16(heads, std):
        return (torch.randn((T, heads, D), generator=g, device="cuda") * std).to(torch.bfloat16)

    return bf16(HQ, 1.2), bf16(HKV, 1.2), bf16(HKV, 1.0), bf16(HQ, 0.02)


def _both_passes(q, k, v, do, spans, **form):
    o, lse = ops.attention(q, k, v, spans, **form)
    return (o, lse, *ops.attention_backward(do, q, k, v, o, lse, spans, **form))


def _unseen(spans):
    """The keys that no row sees, the rows that see no key."""
    T = spans.shape[0]
    at = torch.arange(T, device=spans.device)
    ok = (at[None] >= spans[:, :1]) & (at[None] < spans[:, 1:])
    return ~ok.any(0), ~ok.any(1)


def _junk_changes_nothing(T, heads, spans, junk, seed, softcap=0.0, bias=False):
    HQ, HKV, D = heads
    clean = _inputs(T, HQ, HKV, D, seed)
    keys, rows = _unseen(spans)
    assert keys.any()
    q, k, v, do = (x.clone() for x in clean)
    q[rows], do[rows], k[keys], v[keys] = junk, junk, junk, junk
    form = dict(softcap=softcap, slopes=torch.linspace(0.0, 0.4, HQ, device="cuda") if bias else None)
    names = ("o", "lse", "dq", "dk", "dv")
    got = dict(zip(names, _both_passes(q, k, v, do, spans, **form)))
    assert all(torch.isfinite(got[n]).all() for n in names if n != "lse")
    assert torch.equal(got["lse"] == -math.inf, rows.expand(HQ, T))
    assert all((got[n][w] == 0).all() for n, w in (("o", rows), ("dq", rows), ("dk", keys), ("dv", keys)))
    if not softcap:
        want = dict(zip(names, _both_passes(*clean, spans, **form)))
        assert [n for n in names if not torch.equal(got[n], want[n])] == []
        return
    # which of the cap's forms a warp takes goes by its largest product, masked
    # ones among them: the same results but for the last bits
    q, k, v, do = (x.double() for x in clean)
    r = ref.attention(q, k, v, spans.long(), D ** -0.5, softcap, None if form["slopes"] is None else form["slopes"].double(), do)
    for n in ("o", "dq", "dk", "dv"):
        assert ((got[n].double() - r[n]).abs() <= r[n + "_tol"] + 1e-30).all(), n
    off = (got["lse"].double() - r["lse"]).abs()[:, ~rows]
    assert (off <= 2e-5 * (1 + r["lse"][:, ~rows].abs())).all()


@pytest.mark.parametrize("junk", JUNK)
@pytest.mark.parametrize("softcap,bias", FORMS)
@pytest.mark.parametrize("heads", SPLIT + PAIRS)
@pytest.mark.parametrize("causal", [True, False])
def test_caps_and_biases_of_padded_ends(heads, softcap, bias, junk, causal):
    """Documents with padding before and after them, scores capped and biased."""
    T, first, end = 333, 19, 290
    off = torch.tensor([first, 100, end], dtype=torch.int32, device="cuda")
    _junk_changes_nothing(T, heads, ops.attention_spans(off, T, causal=causal), junk, 21, softcap, bias)


def _padded(T, lengths, causal):
    """Sequences with padding after each: (tokens, padding) in turn."""
    rows, n = [(0, 0)] * T, 0
    while n < T:
        for keep, pad in lengths:
            for i in range(n, min(n + keep, T)):
                rows[i] = (n, i + 1 if causal else min(n + keep, T))
            n += keep + pad
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("junk", JUNK)
@pytest.mark.parametrize("softcap,bias", [(0.0, False), *FORMS[:3]])
@pytest.mark.parametrize("heads", SPLIT + PAIRS)
def test_padding_between_sequences(heads, softcap, bias, junk):
    """Each sequence padded: the padding lies between keys that rows of the same
    tiles see, within a tile and across the two tiles of an item."""
    for T, lengths in ((333, [(40, 10)]), (520, [(100, 50), (106, 1)]), (470, [(3, 1), (1, 2), (200, 133)])):
        for causal in (True, False):
            _junk_changes_nothing(T, heads, _padded(T, lengths, causal), junk, T, softcap, bias)


@pytest.mark.parametrize("heads", SPLIT + PAIRS)
def test_scattered_intervals(heads):
    """Rows of one tile that see keys far apart, in no order, whole tiles of unseen keys between."""
    T = 700
    g = torch.Generator().manual_seed(heads[2])
    rows = []
    for i in range(T):
        a = int(torch.randint(0, 3, (1,), generator=g)) * 300 + int(torch.randint(0, 40, (1,), generator=g))
        rows.append([(a, a + int(torch.randint(1, 50, (1,), generator=g))), (0, 0)][i % 7 == 3])
    spans = torch.tensor(rows, dtype=torch.int32, device="cuda")
    for junk in JUNK:
        _junk_changes_nothing(T, heads, spans, junk, 5)


@pytest.mark.parametrize("softcap,bias", [(0.0, False), *FORMS[:3]])
@pytest.mark.parametrize("heads", SPLIT + PAIRS)
def test_nan_in_a_seen_place_reaches_its_rows(heads, softcap, bias):
    """A row that sees a NaN has NaN as its result, not that of a row without
    keys; the other rows keep theirs."""
    HQ, HKV, D = heads
    T, key, row = 400, 150, 260
    q, k, v, _ = _inputs(T, HQ, HKV, D, 8)
    form = dict(softcap=softcap, slopes=torch.linspace(0.0, 0.4, HQ, device="cuda") if bias else None)
    spans = ops.attention_spans(torch.tensor([0, 70, 333], dtype=torch.int32, device="cuda"), T)
    want, want_lse = ops.attention(q, k, v, spans, **form)
    sees = torch.zeros(T, dtype=torch.bool, device="cuda")
    sees[key:333] = True                             # causal, one document from 70 to 333
    bad = k.clone()
    bad[key, :, D // 2] = math.nan
    o, lse = ops.attention(q, bad, v, spans, **form)
    assert torch.isnan(o[sees]).all() and torch.isnan(lse[:, sees]).all()
    assert torch.equal(o[~sees], want[~sees]) and torch.equal(lse[:, ~sees], want_lse[:, ~sees])
    sees[:] = False
    sees[row] = True
    bad = q.clone()
    bad[row, :, 3] = math.nan
    o, lse = ops.attention(bad, k, v, spans, **form)
    assert torch.isnan(o[row]).all() and torch.isnan(lse[:, row]).all()
    assert torch.equal(o[~sees], want[~sees]) and torch.equal(lse[:, ~sees], want_lse[:, ~sees])
    sees[key:333] = True
    bad = v.clone()
    bad[key, :, 5] = math.nan
    o, lse = ops.attention(q, k, bad, spans, **form)
    assert torch.isnan(o[key:333, :, 5]).all() and torch.equal(lse, want_lse)


@pytest.mark.parametrize("heads", SPLIT + PAIRS)
def test_a_product_that_overflows_is_not_an_empty_row(heads):
    HQ, HKV, D = heads
    T = 300
    q, k, v, _ = _inputs(T, HQ, HKV, D, 9)
    q[200], k[40] = 1e30, 1e30
    o, lse = ops.attention(q, k, v, ops.attention_spans(torch.tensor([0, T], dtype=torch.int32, device="cuda"), T))
    assert torch.isnan(o[200]).all() and torch.isnan(lse[:, 200]).all()
    # (the rows between see a score of 1e30, of which FP32 holds no digit that exp could use)
    assert torch.isfinite(o[:40]).all() and torch.isfinite(lse[:, :40]).all()
