"""The device-side step without a GPU: the numpy oracle against closed forms, and every
refusal of the three entry points (they return before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

import zero_copy_offloaded_gb300 as dkv
from oracle import paged_step as step
from zero_copy_offloaded_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return dkv.lib()


# ---- the oracle -------------------------------------------------------------------------

def test_formats_round_trip_and_ties():
    codes = np.arange(16, dtype=np.uint8)
    assert np.array_equal(step.to_e2m1(step.from_e2m1(codes)), codes)
    # midpoints go to the even code, just above and below them to the nearest
    mid = (step.E2M1[1:] + step.E2M1[:-1]) / 2
    even = [i if i % 2 == 0 else i + 1 for i in range(7)]
    assert step.to_e2m1(mid).tolist() == even
    assert step.to_e2m1(mid * (1 + 1e-9)).tolist() == list(range(1, 8))
    assert step.to_e2m1(mid * (1 - 1e-9)).tolist() == list(range(7))
    assert step.to_e2m1(np.array([1e9, -1e9])).tolist() == [7, 15]
    sc = np.arange(127, dtype=np.uint8)
    assert np.array_equal(step.to_e4m3(step.from_e4m3(sc)), sc)
    assert step.from_e4m3(np.array([0x7E]))[0] == 448 and np.isnan(step.from_e4m3(np.array([0x7F])))[0]
    assert step.to_e4m3(np.array([1e9]))[0] == 0x7E


def test_quantised_values_have_six_bits():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((50, 128)).astype(np.float32) * np.exp(rng.standard_normal((50, 1)) * 3)
    v = step.dequantise(*step.quantise(y.astype(np.float32)))
    assert np.array_equal(v, v.astype(np.float16).astype(np.float64))
    assert np.abs(v - y).max(-1).max() <= np.abs(y).max() * 0.2


def test_pool_layout_round_trip():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((3, 2, 16, 64)).astype(np.float32)
    pool = step.make_pool(v)
    assert pool.shape == (3, 2, 16 * 36)
    assert np.array_equal(step.read_pool(pool, 64), step.dequantise(*step.quantise(v)))


def test_rotation_keeps_lengths_and_relative_angles():
    torch = pytest.importorskip("torch")
    t = dkv.rope_table(300, 64, device="cpu")
    assert t.shape == (300, 64) and t.dtype == torch.float32
    t = t.numpy()
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 1, 64)).astype(np.float32)
    for inter in (False, True):
        rot = lambda v, p: step.turn(v[None, None], None, 0, t, np.array([p]), inter)[0][0, 0]  # noqa: E731
        a, b = x[0, 0], x[1, 0]
        assert np.allclose(np.linalg.norm(rot(a, 200)), np.linalg.norm(a), rtol=1e-6)
        assert np.allclose(rot(a, 250) @ rot(b, 210), rot(a, 140) @ rot(b, 100), rtol=1e-4, atol=1e-4)
        assert np.array_equal(rot(a, 0), a)


def test_plan_oracle_by_hand():
    table = np.array([[5, 9, -1, -1], [7, -1, -1, -1], [3, 4, -1, -1]], np.int32)
    free = np.array([1, 2, 8, -1, -1, -1, -1, -1, -1, -1], np.int32)
    r = step.plan(np.array([31, 0, 20]), np.array([3, 2, -1]), table, free, 3, 16, 8)
    # sequence 2's pages 3, 4 go on the stack and come off again: 4 to sequence 0, 3 to sequence 1
    assert r["table"].tolist() == [[5, 9, 4, -1], [3, -1, -1, -1], [3, 4, -1, -1]]
    assert r["free"].tolist()[:5] == [1, 2, 8, 3, 4] and r["free_left"] == 3
    assert r["row_start"].tolist() == [0, 3, 5, 5]
    assert r["pos"].tolist() == [31, 32, 33, 0, 1, 0, 0, 0]
    assert r["slot"].tolist() == [9 * 16 + 15, 64, 65, 48, 49, -1, -1, -1]
    assert r["kv_len"].tolist() == [34, 2, 0] and r["report"] == [0, 5, 2, 34]
    assert step.plan(np.array([31, 0, 20]), np.array([3, 2, 0]), table, free, 1, 16, 8)["report"][0] == 3


def test_attention_oracle_closed_forms():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 1, 16, 64)), rng.standard_normal((2, 1, 16, 64))
    table = np.array([[1, 0]])
    q = np.zeros((1, 2, 64))
    r = step.attend(q, k, v, table, [20], [0, 1], 0.125)
    rows = np.concatenate([v[1, 0], v[0, 0, :4]])
    assert np.allclose(r["out"][0], rows.mean(0)) and np.allclose(r["lse"], np.log(20))
    q = rng.standard_normal((1, 2, 64))
    assert np.allclose(step.attend(q, k, v, table, [1], [0, 1], 0.125)["out"][0], v[1, 0, 0])
    # two rows: the first does not see the second's key
    two = step.attend(np.repeat(q, 2, 0), k, v, table, [20], [0, 2], 0.125)
    assert np.allclose(two["out"][0], step.attend(q, k, v, table, [19], [0, 1], 0.125)["out"][0])
    assert step.attend(q, k, v, table, [0], [0, 1], 0.125)["lse"].max() == -np.inf


# ---- refusals ---------------------------------------------------------------------------

P16 = 1 << 20  # a 16-byte aligned address that no refused call touches


class AppendArgs(ctypes.Structure):
    """dkv_append_t of include/dkv.h, field by field."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v")]
                + [(n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "v_stride")]
                + [(n, ctypes.c_void_p) for n in (
                    "q_gamma", "k_gamma", "cos_sin", "positions", "slots", "k_pool", "v_pool",
                    "q_out", "k_out", "v_out")]
                + [(n, ctypes.c_int) for n in (
                    "rows", "n_q_heads", "n_kv_heads", "head_dim", "dtype", "rotary_dim",
                    "max_positions", "interleaved", "page_tokens", "num_pages")]
                + [(n, ctypes.c_float) for n in ("eps", "k_scale", "v_scale")])


class AttendArgs(ctypes.Structure):
    """dkv_attend_t."""
    _fields_ = ([("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in (
                    "k_pool", "v_pool", "page_table", "kv_len", "row_start", "out", "lse",
                    "workspace")]
                + [("workspace_bytes", ctypes.c_size_t)]
                + [(n, ctypes.c_int) for n in (
                    "batch", "rows", "max_rows", "n_q_heads", "n_kv_heads", "head_dim", "dtype",
                    "page_tokens", "num_pages", "max_pages")]
                + [(n, ctypes.c_float) for n in ("scale", "v_scale")])


def test_packed_arguments_match_the_structures():
    # the binding packs every field in order; numbers of their own find a field out of place
    for packer, cls in ((dkv._APPEND, AppendArgs), (dkv._ATTEND, AttendArgs)):
        names = [n for n, _ in cls._fields_]
        raw = packer.pack(*range(1, len(names) + 1))
        a = cls.from_buffer_copy(raw + bytes(ctypes.sizeof(cls) - len(raw)))
        assert [getattr(a, n) for n in names] == list(range(1, len(names) + 1))


def append_args(**over):
    a = AppendArgs(q=P16, k=P16, v=P16, q_stride=6144, k_stride=6144, v_stride=6144, positions=P16,
                   cos_sin=P16, slots=P16, k_pool=P16, v_pool=P16, q_out=P16, rows=4, n_q_heads=32,
                   n_kv_heads=8, head_dim=128, dtype=0, rotary_dim=128, max_positions=64,
                   page_tokens=16, num_pages=4, eps=1e-6, k_scale=1.0, v_scale=1.0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over", [
    dict(q=None, k=None, v=None), dict(v=None), dict(k=None), dict(q_out=None), dict(rows=0),
    dict(rows=-1), dict(dtype=2), dict(n_q_heads=0), dict(n_kv_heads=0), dict(q_stride=4095),
    dict(q_stride=4088), dict(k_stride=1020), dict(v_stride=1025), dict(q=P16 + 8), dict(k_pool=P16 + 4),
    dict(slots=None), dict(v_pool=None), dict(k_pool=None), dict(k_pool=None, v_pool=None),
    dict(k_pool=None, v_pool=None, slots=None), dict(k=None, v=None), dict(page_tokens=8),
    dict(page_tokens=24), dict(page_tokens=8192), dict(num_pages=0), dict(num_pages=1 << 27),
    dict(k_scale=0.0), dict(k_scale=float("nan")), dict(v_scale=float("inf")), dict(v_scale=-1.0),
    dict(k_scale=1e-45), dict(positions=None), dict(rotary_dim=8), dict(rotary_dim=0), dict(rotary_dim=144),
    dict(max_positions=0), dict(eps=-1.0), dict(eps=float("nan")),
])
def test_append_refuses(L, over):
    assert L.dkv_qkv_append(ctypes.byref(append_args(**over)), None) == 1, dkv.dkv_last_error()


def test_append_unsupported_head_dim(L):
    assert L.dkv_qkv_append(ctypes.byref(append_args(head_dim=96)), None) == 2
    assert L.dkv_qkv_append(None, None) == 1


def attend_args(**over):
    a = AttendArgs(q=P16, q_stride=4096, k_pool=P16, v_pool=P16, page_table=P16, kv_len=P16,
                   row_start=P16, out=P16, workspace=P16, workspace_bytes=1 << 30, batch=4, rows=8,
                   max_rows=2, n_q_heads=32, n_kv_heads=8, head_dim=128, dtype=0, page_tokens=16,
                   num_pages=64, max_pages=16, scale=0.1, v_scale=1.0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over", [
    dict(q=None), dict(k_pool=None), dict(v_pool=None), dict(page_table=None), dict(kv_len=None),
    dict(out=None), dict(workspace=None), dict(batch=0), dict(batch=1025), dict(rows=0),
    dict(rows=(1 << 30) + 1), dict(max_rows=0), dict(row_start=None), dict(row_start=None, rows=4),
    dict(dtype=5), dict(n_kv_heads=0), dict(n_q_heads=0), dict(n_q_heads=33), dict(q_stride=4088),
    dict(q_stride=4100), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=8192), dict(num_pages=0),
    dict(num_pages=1 << 27), dict(max_pages=0), dict(max_pages=1 << 27), dict(q=P16 + 2), dict(out=P16 + 8),
    dict(k_pool=P16 + 8), dict(workspace=P16 + 16), dict(workspace_bytes=1000), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(v_scale=float("nan")), dict(rows=1 << 30),
])
def test_attend_refuses(L, over):
    assert L.dkv_paged_attend(ctypes.byref(attend_args(**over)), None) == 1, dkv.dkv_last_error()


def test_attend_unsupported_head_dim(L):
    assert L.dkv_paged_attend(ctypes.byref(attend_args(head_dim=256, q_stride=1 << 20)), None) == 2
    assert L.dkv_paged_attend(None, None) == 1
    for bad in [(0, 8, 8, 128, 1), (1, 8, 3, 128, 1), (1, 8, 8, 96, 1), (1, 8, 8, 128, 0), (1, 0, 8, 128, 1)]:
        assert dkv.dkv_paged_attend_workspace(*bad) == 0
    assert dkv.dkv_paged_attend_workspace(4, 32, 8, 128, 2) > 0


PLAN = dict(lengths=P16, new=P16, table=P16, free=P16, count=P16, batch=4, max_pages=8, page=16,
            pages=64, rows=32, start=P16, pos=P16, slot=P16, kv=P16, left=P16, report=P16)


@pytest.mark.parametrize("over", [{k: None} for k, v in PLAN.items() if v == P16] + [
    dict(batch=0), dict(batch=1025), dict(max_pages=0), dict(max_pages=1 << 27), dict(page=0),
    dict(page=12), dict(page=8192), dict(pages=0), dict(pages=1 << 27), dict(rows=0), dict(rows=(1 << 30) + 1)])
def test_plan_refuses(L, over):
    assert L.dkv_step_plan(*{**PLAN, **over}.values(), None) == 1


def test_e2m1_caches_are_paged(L):
    for kw in (dict(max_tokens=64), dict(page_tokens=8, num_pages=4, max_pages_per_seq=4)):
        with pytest.raises(dkv.DkvError) as ei:
            dkv.dkv_cache_alloc_ex(1, 1, 128, kv_format="e2m1", **kw)
        assert ei.value.name == "DKV_ERR_UNSUPPORTED"


def test_binding_checks_tensors(L):
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, k = z(4, 8, 128), z(4, 2, 128)
    with pytest.raises(ValueError, match="current CUDA device"):  # host tensors
        dkv.dkv_qkv_append(q, k, k, q_out=z(4, 8, 128), k_out=k, v_out=k)
    with pytest.raises(ValueError, match="q_out has shape"):
        dkv.dkv_qkv_append(q, k, k, q_out=z(4, 7, 128), k_out=k, v_out=k)
    with pytest.raises(ValueError, match="contiguous"):
        dkv.dkv_qkv_append(z(4, 128, 8).transpose(1, 2), k, k, q_out=q, k_out=k, v_out=k)
    with pytest.raises(ValueError, match="neither bfloat16 nor float16"):
        dkv.dkv_qkv_append(q.float(), None, None, q_out=q.float())
    with pytest.raises(ValueError, match="neither queries nor keys"):
        dkv.dkv_qkv_append(None, None, None)
    with pytest.raises(ValueError, match="not torch.int32"):
        dkv.dkv_step_plan(i(2).long(), i(2), i(2, 4), i(8), i(1), 16, i(3), i(4), i(4), i(2), i(1), i(4))
    with pytest.raises(ValueError, match="row_start has shape"):
        dkv.dkv_step_plan(i(2), i(2), i(2, 4), i(8), i(1), 16, i(2), i(4), i(4), i(2), i(1), i(4))
    with pytest.raises(ValueError, match="current CUDA device"):
        dkv.dkv_paged_attend(q, z(4, 2, 1152, dt=torch.uint8), z(4, 2, 1152, dt=torch.uint8), i(4, 4), i(4), q)
