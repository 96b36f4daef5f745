"""The 8-bit step without a GPU: the oracle against closed forms, and every refusal of the entry points (they return
before anything is enqueued)."""
import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import block_step as bs
from zero_copy_offloaded_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return dkv.lib()


# ---- the oracle -------------------------------------------------------------------------

def test_codes_and_scales():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    assert np.array_equal(bs.encode(bs.decode(codes)), codes)
    assert bs.decode(np.array([0x7E, 0xFE, 0x01, 0x08])).tolist() == [448, -448, 2.0 ** -9, 2.0 ** -6]
    # a tie goes to the even code: 17 lies between 16 (0x58) and 18 (0x59), 19 between 18 and 20 (0x5A)
    assert bs.encode(np.array([17.0, 19.0, -17.0])).tolist() == [0x58, 0x5A, 0xD8]
    assert np.isnan(bs.decode(bs.encode(np.array([np.inf, -np.inf, np.nan])))).all()
    assert bs.scale_for(np.array([448.0, 448.1, 3.5, 3.6, 0.0, 2.0 ** 127])).tolist() == [
        1.0, 2.0, 2.0 ** -7, 2.0 ** -6, 2.0 ** -64, 2.0 ** 119]


def test_append_grows_scales_without_loss():
    """Powers of two: a block that grew holds what one written at once holds, but for E4M3's subnormals."""
    rng = np.random.default_rng(0)
    y = (rng.standard_normal((16, 2, 64)) * np.exp2(rng.integers(-3, 4, (16, 1, 1)))).astype(np.float32)
    y = np.where(np.abs(y) < 0.1, 0.1, y).astype(np.float32)
    pool, scales = np.zeros((2, 2, 16, 64), np.uint8), np.full((2, 2, 1), 7.0, np.float32)
    at_once = bs.append(y, np.arange(16, 32), pool, scales)
    p, s = pool, scales
    for i in range(16):
        p, s, held = bs.append(y[i:i + 1], np.array([16 + i]), p, s)
        assert np.abs(held - y[i]).max() <= np.abs(y[i]).max() / 16
    assert np.array_equal(p, at_once[0]) and np.array_equal(s, at_once[1])
    assert (s[0] == 7).all()  # the other page's, untouched
    # cut back and appended to again: the scale stays
    p2, s2, _ = bs.append(y[3:4] * 2.0 ** -5, np.array([20]), p, s)
    assert np.array_equal(s2, s) and np.array_equal(p2[1, :, 5:], p[1, :, 5:])
    # from the first row on: it begins anew
    assert (bs.append(y[3:4] * 2.0 ** -5, np.array([16]), p, s)[1][1] < s[1]).all()


# ---- refusals ---------------------------------------------------------------------------

A = 4096
APPEND = dict(q=A, k=A, v=A, qs=512, ks=128, vs=128, qg=0, kg=0, cs=A, pos=A, slots=A, kp=A, vp=A, ksc=A, vsc=A,
              qo=A, ko=0, vo=0, rows=4, hq=8, hkv=2, d=64, dtype=0, rot=64, maxp=100, inter=0, pt=16, pages=8, eps=1e-6)


@pytest.mark.parametrize("change,status", [
    ({"k": 0}, 1), ({"v": 0}, 1), ({"kp": 0}, 1), ({"vp": 0}, 1), ({"ksc": 0}, 1), ({"vsc": 0}, 1), ({"slots": 0}, 1),
    ({"qo": 0}, 1), ({"rows": 0}, 1), ({"rows": (1 << 30) + 1}, 1), ({"dtype": 2}, 1), ({"d": 96}, 2), ({"hq": 0}, 1),
    ({"hkv": 0}, 1), ({"qs": 504}, 1), ({"ks": 132}, 1), ({"vs": 120}, 1), ({"q": A + 8}, 1), ({"kp": A + 8}, 1),
    ({"ksc": A + 2}, 1), ({"vsc": A + 1}, 1), ({"cs": A + 4}, 1), ({"pt": 8}, 1), ({"pt": 48}, 1), ({"pt": 8192}, 1),
    ({"pages": 0}, 1), ({"pages": 1 << 27}, 1), ({"pos": 0}, 1), ({"rot": 24}, 1), ({"rot": 80}, 1), ({"maxp": 0}, 1),
    ({"eps": -1.0}, 1), ({"eps": float("nan")}, 1)])
def test_append_refuses(L, change, status):
    assert L.dkv_block_append(dkv._BLOCK_APPEND.pack(*{**APPEND, **change}.values()), None) == status
    assert dkv.dkv_last_error()
    assert L.dkv_block_append(None, None) == 1


ATTEND = dict(q=A, qs=512, kp=A, vp=A, ksc=A, vsc=A, pt=A, kl=A, rs=A, out=A, lse=0, ws=A, size=1 << 30, batch=4, rows=9,
              max_rows=3, hq=8, hkv=2, d=64, dtype=0, page=16, pages=8, max_pages=4, scale=0.125)


@pytest.mark.parametrize("change,status", [
    ({"q": 0}, 1), ({"kp": 0}, 1), ({"vp": 0}, 1), ({"ksc": 0}, 1), ({"vsc": 0}, 1), ({"pt": 0}, 1), ({"kl": 0}, 1),
    ({"out": 0}, 1), ({"ws": 0}, 1), ({"batch": 0}, 1), ({"batch": 1025}, 1), ({"rows": 0}, 1), ({"max_rows": 0}, 1),
    ({"rs": 0}, 1), ({"dtype": 2}, 1), ({"d": 96}, 2), ({"hq": 7}, 1), ({"hkv": 0}, 1), ({"qs": 508}, 1), ({"qs": 256}, 1),
    ({"page": 8}, 1), ({"page": 24}, 1), ({"page": 8192}, 1), ({"pages": 0}, 1), ({"max_pages": 0}, 1),
    ({"max_pages": 1 << 27}, 1), ({"q": A + 8}, 1), ({"kp": A + 8}, 1), ({"ksc": A + 2}, 1), ({"out": A + 4}, 1), ({"ws": A + 64}, 1),
    ({"size": 1000}, 1), ({"scale": float("inf")}, 1), ({"scale": float("nan")}, 1)])
def test_attend_refuses(L, change, status):
    assert L.dkv_block_attend(dkv._BLOCK_ATTEND.pack(*{**ATTEND, **change}.values()), None) == status
    assert dkv.dkv_last_error()
    assert L.dkv_block_attend(None, None) == 1


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    k, pool, sc, i = z(4, 2, 64), z(8, 2, 16, 64, dt=torch.float8_e4m3fn), z(8, 2, 1, dt=torch.float32), z(4, dt=torch.int32)

    def call(k=k, v=k, pool=pool, other=pool, sc=sc):
        dkv.dkv_block_append(None, k, v, i, i, pool, other, sc, sc)
    with pytest.raises(ValueError, match="current CUDA device"):
        call()
    with pytest.raises(ValueError, match="neither queries nor keys"):
        call(k=None)
    with pytest.raises(ValueError, match="both are"):
        call(pool=z(8, 2, 16, 128, dt=torch.uint8))
    with pytest.raises(ValueError, match="neither float8"):
        call(pool=z(8, 2, 16, 64), other=z(8, 2, 16, 64))
    with pytest.raises(ValueError, match="float32"):
        call(sc=z(8, 2, 2, dt=torch.float32))
    with pytest.raises(ValueError, match="for 1 heads"):
        call(k=z(4, 1, 64), v=z(4, 1, 64))
    with pytest.raises(ValueError, match="contiguous"):
        call(pool=z(8, 2, 64, 16, dt=torch.uint8).transpose(2, 3), other=z(8, 2, 16, 64, dt=torch.uint8))
