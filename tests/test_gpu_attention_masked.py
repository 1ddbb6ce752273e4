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
