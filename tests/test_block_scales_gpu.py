"""Attention over an 8-bit cache whose scales, or whose queries' sizes, lie far apart: against the fp64 oracle, with the
bounds that test_block_attend_gpu.check derives."""
import numpy as np
import pytest

from tests.test_block_attend_gpu import case, check, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def far_keys(c, scale, every, seed=0):
    """The first block of every sequence, and one in `every` of the others, has K scale `scale` (zero codes where that would
    make scores of another size), the others 2^-7."""
    (k, ks), v = c["pools"]
    k, ks = k.copy(), np.full_like(ks, 2.0 ** -7)
    far = np.random.default_rng(seed).random(ks.shape) < 1 / every
    far[c["table"][:, 0], :, 0] = True
    ks[far] = scale
    if scale > 1:
        k = np.where(np.repeat(far, 16, -1)[..., None], 0, k).astype(k.dtype)
    return dict(c, pools=[(k, ks), v])


@pytest.mark.parametrize("rows", [1, 3, 60])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("exponent", [-126, -112, -64, 60, 100, 126])
def test_k_scales_far_from_the_first(rows, D, dtype, exponent):
    c = far_keys(case(41, [500, 900, 40], [rows, rows, 1], 4, 2, D, dtype, 16), 2.0 ** exponent, 20)
    check(c, *run(c))
    # the other way round: the far scale in every block but the first of each sequence and some others
    (k, ks), v = c["pools"]
    if exponent < 0:
        other = np.where(ks == 2.0 ** -7, np.float32(2.0 ** exponent), np.float32(2.0 ** -7))
        check(d := dict(c, pools=[(k, other), v]), *run(d))


@pytest.mark.parametrize("rows", [1, 40])
def test_k_scales_of_every_size(rows):
    """Blocks from 2^-126 to 2^-7 side by side, powers of two and not, over sequences that CTAs share."""
    c = case(42, [5000, 700], [rows, rows], 4, 2, 128, "bf16", 16)
    (k, ks), v = c["pools"]
    rng = np.random.default_rng(1)
    for x in (np.exp2(rng.integers(-126, -6, ks.shape)), np.exp2(rng.uniform(-126, -7, ks.shape)), np.exp2(rng.integers(-40, -6, ks.shape))):
        d = dict(c, pools=[(k, x.astype(np.float32)), v])
        check(d, *run(d))


@pytest.mark.parametrize("bad", [np.nan, 2.0 ** -64])
def test_a_nan_scale_reaches_the_rows_that_see_it(bad):
    """Beside a first block whose scale is far away, more than 32 packed rows."""
    c = far_keys(case(43, [300], [100], 2, 1, 128, "bf16", 16), 2.0 ** -112, 1000)
    c["pools"][0][1][c["table"][0, 17]] = bad  # tokens 272 .. 287, seen from row 72 on
    out, lse = run(c)
    if np.isnan(bad):
        assert torch.isnan(out[72:100].float()).all() and torch.isnan(lse[72:100]).all()
        assert torch.isfinite(out[:72].float()).all() and torch.isfinite(lse[:72]).all()
    else:
        check(c, out, lse)


@pytest.mark.parametrize("rows", [1, 3, 5, 8, 60])
@pytest.mark.parametrize("D", [64, 128])
def test_small_queries_over_large_keys(rows, D):
    """Queries near 2^-112 over K scales near 2^105: their products are of ordinary size."""
    c = case(44, [500, 900, 40], [rows, rows, 1], 4, 1, D, "bf16", 16)
    (k, ks), v = c["pools"]
    c["q"] = (c["q"].float() * 2.0 ** -112).to(torch.bfloat16)
    d = dict(c, pools=[(k, np.full_like(ks, 2.0 ** 105)), v])
    check(d, *run(d))
    first = np.full_like(ks, 2.0 ** 105)
    first[c["table"][:, 0]] = 2.0 ** 20
    d = dict(c, pools=[(k, first), v])
    check(d, *run(d))


@pytest.mark.parametrize("rows", [1, 3, 5, 8, 60])
@pytest.mark.parametrize("D", [64, 128])
def test_zero_codes_beside_large_scales_and_queries(rows, D):
    """Dims of 2^90 in the queries meet zero codes of blocks with a scale of 2^60, and the other way round: scores of 0."""
    c = case(45, [500, 900, 40], [rows, rows, 1], 4, 1, D, "bf16", 16)
    (k, ks), v = c["pools"]
    q = torch.zeros_like(c["q"])
    q[..., :8] = 2.0 ** 90
    c["q"] = q
    k = k.copy()
    k[..., :8] = 0
    for scales in (np.full_like(ks, 2.0 ** 60), np.where(np.arange(len(ks))[:, None, None] % 3, 2.0 ** 60, 2.0 ** -7)):
        d = dict(c, pools=[(k, scales.astype(np.float32)), v])
        ref = check(d, *run(d))
        assert np.all(ref["smax"] == 0)


@pytest.mark.parametrize("rows,keys", [(1, 9000), (16, 9000), (40, 700), (40, 9000), (300, 2000)])
@pytest.mark.parametrize("exponent", [-64, -30, 30, 90, 112])
def test_v_scales_of_every_size(rows, keys, exponent):
    """All of V near 2^exponent: outputs of pieces that CTAs share, up to bf16's range."""
    c = case(46, [keys, 40], [rows, min(rows, 40)], 2, 1, 128, "bf16", 16, levels=3.0)
    k, (v, vs) = c["pools"]
    base = 2.0 ** (exponent + 7)  # codes reach 448: scales lie near 2^-7
    d = dict(c, pools=[k, (v, (vs * base).astype(np.float32))])
    check(d, *run(d))
    # no powers of two
    rng = np.random.default_rng(2)
    odd = (vs * base * rng.uniform(1.0, 1.9, vs.shape)).astype(np.float32)
    check(d := dict(c, pools=[k, (v, odd)]), *run(d))


@pytest.mark.parametrize("rows", [1, 16, 40])
@pytest.mark.parametrize("low,high", [(-64, 16), (-20, 60), (20, 100)])
@pytest.mark.parametrize("first", [0, 1])
def test_v_scales_that_one_row_sees(rows, low, high, first):
    """Blocks 2^80 apart, side by side and in halves, the small ones first or last, over sequences that CTAs share."""
    c = case(47, [6000, 300], [rows, rows], 2, 1, 128, "bf16", 16)
    k, (v, vs) = c["pools"]
    pages = len(vs)
    order = np.zeros(pages, int)
    for row in c["table"]:
        order[row] = np.arange(len(row))
    half = order < 200
    for small in ((order + first) % 2 == 0, half if first else ~half):
        x = np.where(small, 2.0 ** low, 2.0 ** high).astype(np.float32)[:, None, None]
        d = dict(c, pools=[k, (v, np.broadcast_to(x, vs.shape).copy())])
        check(d, *run(d))
