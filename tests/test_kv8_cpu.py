"""8-bit K/V cache without a GPU: the oracle against itself, and what the C ABI
and the Python entry points refuse (a refused call returns before any CUDA call)."""

import contextlib
import ctypes
import math

import numpy as np
import pytest
import torch

import looped_transformer_latent_b200 as L
from looped_transformer_latent_b200 import _abi
from oracle import kv8


# ------------------------------------------------------------------ oracle --
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("n,block", [(1, 16), (16, 16), (33, 16), (64, 64)])
def test_codes_are_within_half_a_step(code, n, block):
    rng = np.random.default_rng(n)
    x = rng.standard_normal((n, 48)).astype(np.float32)
    c, s = kv8.write(x, block, code)
    y = kv8.values(c, s, block)
    sc = s[np.arange(n) // block, None].astype(np.float64)
    # int8: half a step of the scale; e4m3: 2^-4 relative, or half the subnormal spacing; and the fp32 quotient
    half = 0.5 * sc if code == "i8" else np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
    assert np.all(np.abs(y - x) <= half * (1 + 2.0 ** -20) + sc * 448 * 2.0 ** -23)
    assert np.all(np.abs(c) <= kv8.TOP[code])


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_blocks_of_zeros_and_of_non_finite_values(code):
    x = np.zeros((4, 16), dtype=np.float32)
    c, s = kv8.quantise_block(x, code)
    assert s == 0 and not c.any()
    for bad in (np.inf, -np.inf, np.nan):
        x[1, 2] = bad
        c, s = kv8.quantise_block(x, code)
        assert math.isnan(s) and not c.any()


def test_attention_of_exact_rows_is_a_softmax():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((2, 1, 1, 8)), rng.standard_normal((1, 5, 8)), rng.standard_normal((1, 5, 8))
    wk, wv = rng.standard_normal((3, 1, 8)), rng.standard_normal((3, 1, 8))
    out, w = kv8.attn(q, k, v, wk, wv)
    kk, vv = np.concatenate([k[0], wk[:, 0]]), np.concatenate([v[0], wv[:, 0]])
    s = np.exp(kk @ q[1, 0, 0] / math.sqrt(8))
    assert np.allclose(out[1, 0, 0], (s[:, None] * vv).sum(0) / s.sum())
    s0 = np.exp(kk[:7] @ q[0, 0, 0] / math.sqrt(8))   # the first query does not see the last row
    assert np.allclose(out[0, 0, 0], (s0[:, None] * vv[:7]).sum(0) / s0.sum())
    assert np.allclose(w[0], s[:5] / s.sum() + s0[:5] / s0.sum())
    empty, w = kv8.attn(q, k[:, :0], v[:, :0], wk[:0], wv[:0])
    assert not empty.any() and w.shape == (1, 0)


def test_choice_keeps_ends_ties_go_to_the_lowest_and_nan_goes_first():
    w = np.zeros(10 * 4, dtype=np.float32)
    w[5 * 4] = 3.0
    w[7 * 4:8 * 4] = 1.0
    assert kv8.choose(w, 40, 4, 4, 1, 1) == [0, 5, 7, 9]
    assert kv8.choose(w, 40, 4, 5, 1, 1) == [0, 1, 5, 7, 9]     # of the zeros, the lowest
    w[5 * 4 + 1] = np.nan
    assert kv8.choose(w, 40, 4, 4, 1, 1) == [0, 1, 7, 9]
    assert kv8.choose(w, 38, 4, 10, 0, 1) == list(range(10))
    assert kv8.choose(w, 0, 4, 3, 0, 1) == []


# ---------------------------------------------------------------- refusals --
FAKE = 1 << 20   # a pointer that is never read: every call below is refused on the host


def _cache(**kw):
    c = dict(B=2, H=3, d=64, block=32, Ncap=128, code=_abi.LLA_KV8_I8, k=FAKE, v=FAKE + (1 << 16),
             stride_b=3 * 128 * 64, stride_h=128 * 64, k_scale=2 * FAKE, v_scale=2 * FAKE + 4096, scale_stride_b=12,
             scale_stride_h=4)
    c.update(kw)
    return _abi.Kv8Cache(**c)


def _i32(all=0, at=None):
    return _abi.I32(at, all)


def _write(cache=None, **kw):
    p = dict(cache=_cache(**(cache or {})), x_k=3 * FAKE, x_v=4 * FAKE, dtype=_abi.LLA_BF16, rows=64, ring=0,
             x_stride_b=64 * 3 * 64, x_stride_n=3 * 64, x_stride_h=64, max_n=64, n=_i32(64), src0=_i32(), row0=_i32(32))
    p.update(kw)
    return _abi.Kv8WriteParams(**p)


def _attn(cache=None, **kw):
    p = dict(cache=_cache(**(cache or {})), len=_i32(100), nq=1, G=2, q=3 * FAKE, out=4 * FAKE, dtype=_abi.LLA_BF16,
             q_stride_b=384, q_stride_n=384, out_stride_b=384, out_stride_n=384, win_k=5 * FAKE, win_v=6 * FAKE,
             win_dtype=_abi.LLA_BF16, Wcap=16, win_stride_b=16 * 192, win_stride_n=192, win_stride_h=64,
             ctx=_i32(110), tail=_i32(10), scale=0.0, weights=7 * FAKE, weights_stride_b=3 * 128, weights_stride_h=128)
    p.update(kw)
    return _abi.Kv8AttnParams(**p)


def _evict(src=None, dst=None, **kw):
    d = dict(k=8 * FAKE, v=9 * FAKE, k_scale=10 * FAKE, v_scale=11 * FAKE)
    d.update(dst or {})
    p = dict(src=_cache(**(src or {})), dst=_cache(**d), weights=7 * FAKE, weights_stride_b=384, weights_stride_h=128,
             dst_weights=12 * FAKE, dst_weights_stride_b=384, dst_weights_stride_h=128, len=13 * FAKE, dst_len=14 * FAKE,
             keep=3, first=1, last=1, kept=None)
    p.update(kw)
    return _abi.Kv8EvictParams(**p)


CACHE_FAULTS = [
    (dict(B=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(Ncap=-32), "SHAPE"), (dict(Ncap=100), "SHAPE"),
    (dict(code=2), "DTYPE"), (dict(d=8), "UNSUPPORTED"), (dict(d=72), "UNSUPPORTED"), (dict(d=272), "UNSUPPORTED"),
    (dict(block=8), "UNSUPPORTED"), (dict(block=48), "UNSUPPORTED"), (dict(block=512), "UNSUPPORTED"),
    (dict(B=40000), "UNSUPPORTED"), (dict(H=70000), "UNSUPPORTED"), (dict(Ncap=(1 << 30) + 32), "UNSUPPORTED"), (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(k_scale=None), "NULL"),
    (dict(v_scale=None), "NULL"), (dict(k=FAKE + 8), "ALIGN"), (dict(v=FAKE + 4), "ALIGN"),
    (dict(stride_b=3 * 128 * 64 + 8), "ALIGN"), (dict(stride_h=128 * 64 + 8), "ALIGN"),
    (dict(k_scale=2 * FAKE + 2), "ALIGN"), (dict(stride_b=-64), "SHAPE"), (dict(scale_stride_h=-1), "SHAPE"),
]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_every_entry_point_refuses_a_bad_cache(fault, status):
    lib, want = L.lib(), getattr(_abi, "LLA_ERR_" + status)
    assert lib.lla_kv8_write(ctypes.byref(_write(fault)), None) == want
    p = _attn(fault)
    assert lib.lla_kv8_attn_workspace_bytes(ctypes.byref(p)) == 0
    assert lib.lla_kv8_attn(ctypes.byref(p), None, 0, None) == want
    p = _evict(fault)
    assert lib.lla_kv8_evict_workspace_bytes(ctypes.byref(p)) == 0
    assert lib.lla_kv8_evict(ctypes.byref(p), None, 0, None) == want


@pytest.mark.parametrize("p,status", [
    (_write(dtype=2), "DTYPE"), (_write(rows=-1), "SHAPE"), (_write(max_n=-1), "SHAPE"), (_write(max_n=65), "SHAPE"),
    (_write(max_n=32), "SHAPE"), (_write(n=_i32(-1)), "SHAPE"), (_write(row0=_i32(33)), "SHAPE"),
    (_write(row0=_i32(96)), "SHAPE"), (_write(row0=_i32(-32)), "SHAPE"), (_write(src0=_i32(1)), "SHAPE"),
    (_write(src0=_i32(-1)), "SHAPE"), (_write(n=_i32(at=FAKE + 2)), "ALIGN"), (_write(x_k=None), "NULL"),
    (_write(x_v=None), "NULL"), (_write(x_k=3 * FAKE + 8), "ALIGN"), (_write(x_v=4 * FAKE + 2), "ALIGN"),
    (_write(x_stride_n=196), "ALIGN"), (_write(x_stride_h=-64), "SHAPE"),
    (_write(dict(stride_b=0)), "SHAPE"), (_write(dict(stride_h=64)), "SHAPE"), (_write(dict(scale_stride_b=0)), "SHAPE"),
])
def test_write_refuses(p, status):
    assert L.lib().lla_kv8_write(ctypes.byref(p), None) == getattr(_abi, "LLA_ERR_" + status)


@pytest.mark.parametrize("p,status", [
    (_attn(dtype=2), "DTYPE"), (_attn(win_dtype=7), "DTYPE"), (_attn(nq=-1), "SHAPE"), (_attn(G=0), "SHAPE"),
    (_attn(nq=40000), "UNSUPPORTED"), (_attn(len=_i32(129)), "SHAPE"), (_attn(len=_i32(-1)), "SHAPE"),
    (_attn(len=_i32(at=FAKE + 1)), "ALIGN"), (_attn(scale=-1.0), "SHAPE"), (_attn(scale=math.inf), "SHAPE"),
    (_attn(scale=math.nan), "SHAPE"), (_attn(q=None), "NULL"), (_attn(out=None), "NULL"), (_attn(win_v=None), "NULL"),
    (_attn(win_k=None), "NULL"), (_attn(q=3 * FAKE + 8), "ALIGN"), (_attn(out=4 * FAKE + 4), "ALIGN"),
    (_attn(q_stride_b=388), "ALIGN"), (_attn(out_stride_b=376), "SHAPE"), (_attn(nq=2, out_stride_n=376), "SHAPE"),
    (_attn(nq=2, out_stride_n=384, out_stride_b=384), "SHAPE"), (_attn(out=3 * FAKE), "UNSUPPORTED"),
    (_attn(Wcap=0), "SHAPE"), (_attn(tail=_i32(17)), "SHAPE"), (_attn(tail=_i32(-1)), "SHAPE"),
    (_attn(ctx=_i32(-1)), "SHAPE"), (_attn(ctx=_i32(at=3)), "ALIGN"), (_attn(win_k=5 * FAKE + 8), "ALIGN"),
    (_attn(win_v=6 * FAKE + 8), "ALIGN"), (_attn(win_stride_n=196), "ALIGN"), (_attn(win_stride_b=-192), "SHAPE"),
    (_attn(weights=7 * FAKE + 2), "ALIGN"), (_attn(weights_stride_h=127), "SHAPE"), (_attn(weights_stride_b=0), "SHAPE"),
])
def test_attn_refuses(p, status):
    assert L.lib().lla_kv8_attn(ctypes.byref(p), None, 0, None) == getattr(_abi, "LLA_ERR_" + status)


@pytest.mark.parametrize("p,status", [
    (_evict(first=-1), "SHAPE"), (_evict(last=0), "SHAPE"), (_evict(first=3), "SHAPE"), (_evict(keep=5), "SHAPE"),
    (_evict(keep=0, first=0), "SHAPE"), (_evict(dst=dict(Ncap=64)), "SHAPE"), (_evict(dst=dict(d=96)), "SHAPE"),
    (_evict(dst=dict(block=64)), "SHAPE"), (_evict(dst=dict(code=0)), "DTYPE"), (_evict(weights=None), "NULL"),
    (_evict(dst_weights=None), "NULL"), (_evict(len=None), "NULL"), (_evict(dst_len=None), "NULL"),
    (_evict(len=13 * FAKE + 1), "ALIGN"), (_evict(kept=3), "ALIGN"), (_evict(weights_stride_h=-1), "SHAPE"),
    (_evict(dst_weights_stride_h=127), "SHAPE"), (_evict(dst=dict(stride_h=64)), "SHAPE"),
    (_evict(dst_weights=7 * FAKE), "UNSUPPORTED"),                       # weights in place, codes not
    (_evict(dst=dict(k=FAKE)), "UNSUPPORTED"),                           # k in place, the rest not
    (_evict(src=dict(block=16, Ncap=16 * 8193, stride_h=16 * 8193 * 64, stride_b=3 * 16 * 8193 * 64,
                     scale_stride_h=8193, scale_stride_b=3 * 8193), dst=dict(block=16), weights_stride_h=16 * 8193),
     "UNSUPPORTED"),
])
def test_evict_refuses(p, status):
    assert L.lib().lla_kv8_evict(ctypes.byref(p), None, 0, None) == getattr(_abi, "LLA_ERR_" + status)


def test_workspace_is_checked():
    lib, p = L.lib(), _attn()
    need = lib.lla_kv8_attn_workspace_bytes(ctypes.byref(p))
    assert need > 0
    for ws, nb in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert lib.lla_kv8_attn(ctypes.byref(p), ws, nb, None) == _abi.LLA_ERR_WORKSPACE
    assert lib.lla_kv8_evict_workspace_bytes(ctypes.byref(_evict())) == 0        # few heads
    many = dict(B=200, stride_b=3 * 128 * 64, scale_stride_b=12)
    p = _evict(many, many)
    need = lib.lla_kv8_evict_workspace_bytes(ctypes.byref(p))
    assert need >= 200 * 3 * 3 * 4
    assert lib.lla_kv8_evict(ctypes.byref(p), None, need, None) == _abi.LLA_ERR_WORKSPACE
    assert lib.lla_kv8_evict(ctypes.byref(p), FAKE, need - 1, None) == _abi.LLA_ERR_WORKSPACE
    assert lib.lla_kv8_evict_workspace_bytes(ctypes.byref(_evict(many, many, kept=15 * FAKE))) == 0


def test_empty_calls_do_nothing():
    lib = L.lib()
    assert lib.lla_kv8_write(None, None) == _abi.LLA_ERR_NULL
    assert lib.lla_kv8_attn(None, None, 0, None) == _abi.LLA_ERR_NULL
    assert lib.lla_kv8_evict(None, None, 0, None) == _abi.LLA_ERR_NULL
    assert lib.lla_kv8_write(ctypes.byref(_write(dict(B=0))), None) == 0
    assert lib.lla_kv8_write(ctypes.byref(_write(max_n=0, n=_i32(0))), None) == 0
    assert lib.lla_kv8_attn(ctypes.byref(_attn(dict(B=0))), None, 0, None) == 0
    assert lib.lla_kv8_attn(ctypes.byref(_attn(nq=0)), None, 0, None) == 0
    assert lib.lla_kv8_evict(ctypes.byref(_evict(dict(B=0), dict(B=0))), None, 0, None) == 0


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(_abi.I32) == 16
    assert ctypes.sizeof(_abi.Kv8Cache) == 24 + 8 * 8
    assert _abi.Kv8WriteParams.n.offset % 8 == 0
    assert ctypes.sizeof(_abi.Kv8AttnParams) == _abi.Kv8AttnParams.weights_stride_h.offset + 8
    assert ctypes.sizeof(_abi.Kv8EvictParams) == _abi.Kv8EvictParams.kept.offset + 8


def test_python_entry_points_want_cuda_tensors():
    k8 = torch.zeros(1, 1, 32, 16, dtype=torch.int8)
    s = torch.zeros(1, 1, 1)
    x = torch.zeros(1, 32, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        L.lla_kv8_write(k=x, v=x, k8=k8, v8=k8, k_scale=s, v_scale=s)
    with pytest.raises(ValueError, match="CUDA"):
        L.lla_kv8_attn(q=x[:, :1], k8=k8, v8=k8, k_scale=s, v_scale=s, lens=32, out=x[:, 1:2])
    with pytest.raises(ValueError, match="CUDA"):
        L.lla_kv8_evict(k8=k8, v8=k8, k_scale=s, v_scale=s, weights=torch.zeros(1, 1, 32),
                        lens=torch.zeros(1, dtype=torch.int32), keep=1)


@pytest.mark.parametrize("change,error", [
    (dict(k8=torch.zeros(1, 2, 32, 16)), TypeError), (dict(k_scale=torch.zeros(1, 2, 2, dtype=torch.float64)), TypeError),
    (dict(v8=torch.zeros(1, 2, 32, 32, dtype=torch.int8)), ValueError), (dict(v_scale=torch.zeros(1, 2, 4)), ValueError),
    (dict(k_scale=torch.zeros(1, 2, 3), v_scale=torch.zeros(1, 2, 3)), ValueError),
    (dict(q=torch.zeros(1, 1, 3, 16)), ValueError), (dict(q=torch.zeros(1, 1, 2, 32)), ValueError),
    (dict(out=torch.zeros(1, 1, 2, 16, dtype=torch.bfloat16)), ValueError), (dict(lens=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(lens=torch.zeros(1, dtype=torch.int64)), ValueError), (dict(win_k=torch.zeros(1, 8, 2, 16)), ValueError),
    (dict(win_v=torch.zeros(1, 8, 2, 16)), ValueError), (dict(weights=torch.zeros(1, 2, 31)), ValueError),
    (dict(win_k=torch.zeros(1, 8, 2, 16), win_v=torch.zeros(1, 8, 2, 16)), ValueError),
])
def test_python_binding_checks_shapes_and_dtypes(change, error):
    args = dict(q=torch.zeros(1, 1, 2, 16), k8=torch.zeros(1, 2, 32, 16, dtype=torch.int8),
                v8=torch.zeros(1, 2, 32, 16, dtype=torch.int8), k_scale=torch.zeros(1, 2, 2), v_scale=torch.zeros(1, 2, 2),
                lens=32, out=torch.zeros(1, 1, 2, 16))
    L._kv8_attn_params(**args)
    with pytest.raises(error):
        L._kv8_attn_params(**{**args, **change})


class _Recorder:
    """Stands in for torch.cuda.stream, torch.cuda.device and torch.empty: notes what is current where memory is taken."""

    def __init__(self, monkeypatch):
        self.now, self.taken = {"stream": None, "device": 0}, []
        for what in ("stream", "device"):
            monkeypatch.setattr(torch.cuda, what, lambda v, what=what: self._with(what, v))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.now["device"])
        monkeypatch.setattr(torch, "empty", self._empty)

    @contextlib.contextmanager
    def _with(self, what, value):
        before, self.now[what] = self.now[what], value
        yield
        self.now[what] = before

    def _empty(self, n, dtype, device):
        self.taken.append((n, device, self.now["stream"]))
        return torch.zeros(n, dtype=dtype)


def test_scratch_is_taken_on_the_stream_that_runs_the_call(monkeypatch):
    rec, side = _Recorder(monkeypatch), object()
    for stream in (None, side):
        address, have, kept = L._kv8_workspace(lambda p: 512, None, 0, None, stream)
        assert rec.taken.pop() == (512, torch.device("cuda", 0), stream)
        assert address == kept.data_ptr() and have == 512
    assert L._kv8_workspace(lambda p: 0, None, 0, None, side) == (None, 0, None) and not rec.taken


def test_attn_refuses_more_query_heads_than_32_bits_number():
    """Head h * G + g is a 32-bit number in the kernels: past it rows would lie outside the caller's buffers."""
    for H, G, status in ((65535, 32768, 0), (65535, 32769, _abi.LLA_ERR_UNSUPPORTED)):
        cache = dict(B=0, H=H)          # an empty batch: a call that is not refused does nothing
        assert L.lib().lla_kv8_attn(ctypes.byref(_attn(cache, G=G)), None, 0, None) == status
    row = 65535 * 65535 * 64
    p = _attn(dict(H=65535, stride_b=65535 * 128 * 64, scale_stride_b=65535 * 4), G=65535, q_stride_b=row, q_stride_n=row,
              out_stride_b=row, out_stride_n=row, weights_stride_b=65535 * 128)
    assert L.lib().lla_kv8_attn_workspace_bytes(ctypes.byref(p)) == 0
    assert L.lib().lla_kv8_attn(ctypes.byref(p), None, 0, None) == _abi.LLA_ERR_UNSUPPORTED


def test_attn_refuses_rings_whose_slots_pass_32_bits():
    """Slot of the oldest token plus a token's number, both below Wcap, is summed in 32 bits."""
    lib = L.lib()
    for wcap, status in ((1 << 30, _abi.LLA_ERR_WORKSPACE), ((1 << 30) + 1, _abi.LLA_ERR_UNSUPPORTED),
                         ((1 << 31) - 1, _abi.LLA_ERR_UNSUPPORTED)):
        p = _attn(Wcap=wcap, win_stride_b=0, win_stride_n=0, tail=_i32(at=20 * FAKE))
        assert lib.lla_kv8_attn(ctypes.byref(p), None, 0, None) == status
        assert (lib.lla_kv8_attn_workspace_bytes(ctypes.byref(p)) > 0) == (status == _abi.LLA_ERR_WORKSPACE)


def test_workspace_sizes_are_those_of_the_tensors_device(monkeypatch):
    rec, asked = _Recorder(monkeypatch), []

    def size(p):
        asked.append(rec.now["device"])
        return 64

    monkeypatch.setattr(L, "lib", lambda: type("Lib", (), {"lla_kv8_attn_workspace_bytes": staticmethod(size),
                                                           "lla_kv8_evict_workspace_bytes": staticmethod(size)}))
    k8, s, w = torch.zeros(1, 2, 32, 16, dtype=torch.int8), torch.zeros(1, 2, 2), torch.zeros(1, 2, 32)
    q, lens = torch.zeros(1, 1, 2, 16), torch.zeros(1, dtype=torch.int32)
    for dev in (0, 3):
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t, dev=dev: dev)
        assert L.lla_kv8_attn_workspace_bytes(q=q, k8=k8, v8=k8, k_scale=s, v_scale=s, lens=32, out=q) == 64
        assert L.lla_kv8_evict_workspace_bytes(k8=k8, v8=k8, k_scale=s, v_scale=s, weights=w, lens=lens, keep=1) == 64
    assert asked == [0, 0, 3, 3] and rec.now["device"] == 0


def test_axes_of_one_element_may_carry_any_stride():
    """K from one buffer and V from another whose batch or head axis is longer: the same layout where it counts."""
    def pair(shape, dtype=torch.float32):
        long = torch.zeros(shape[0] * 3, *shape[1:], dtype=dtype)
        return torch.zeros(*shape, dtype=dtype), long.as_strided(shape, (7 * long.stride(0), *long.stride()[1:]))

    k8, v8 = pair((1, 2, 32, 16), torch.int8)
    ks, vs = pair((1, 2, 2))
    wk, wv = pair((1, 8, 2, 16))
    assert k8.stride() != v8.stride() and ks.stride() != vs.stride() and wk.stride() != wv.stride()
    q = torch.zeros(1, 1, 2, 16)
    args = dict(q=q, k8=k8, v8=v8, k_scale=ks, v_scale=vs, lens=32, out=q.clone(), win_k=wk, win_v=wv, ctx=3, tail=3)
    p = L._kv8_attn_params(**args)
    assert (p.cache.stride_h, p.win_stride_n, p.cache.scale_stride_h) == (32 * 16, 32, 2)
    with pytest.raises(ValueError):
        L._kv8_attn_params(**{**args, "v8": torch.zeros(1, 32, 2, 16, dtype=torch.int8).transpose(1, 2)})
    with pytest.raises(ValueError):
        L._kv8_attn_params(**{**args, "win_v": torch.zeros(1, 2, 8, 16).transpose(1, 2)})


def test_workspace_views_with_gaps_or_shared_bytes_are_refused(monkeypatch):
    """Their element count says nothing about the bytes behind their address."""
    rec = _Recorder(monkeypatch)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: rec.now["device"])
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(4096), torch.zeros(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            L._kv8_workspace(lambda p: 512, None, 0, ws, None)
        with pytest.raises(ValueError, match="contiguous"):
            L._workspace(512, torch.device("cuda", 0), ws, None)
    ws = torch.zeros(64, 64, dtype=torch.uint8)
    assert L._kv8_workspace(lambda p: 512, None, 0, ws, None)[:2] == (ws.data_ptr(), 4096)
    assert L._workspace(512, torch.device("cuda", 0), ws, None)[1] == 4096


@pytest.mark.parametrize("gap,status", [(4, "UNSUPPORTED"), (-4, "UNSUPPORTED"), (0, "SHAPE"), (8, "SHAPE"), (-8, "SHAPE")])
def test_evict_refuses_lengths_that_overlap_in_part(gap, status):
    # two sequences; the calls that this check lets pass are refused by a later one
    p = _evict(len=13 * FAKE, dst_len=13 * FAKE + gap, dst_weights_stride_h=127)
    assert L.lib().lla_kv8_evict(ctypes.byref(p), None, 0, None) == getattr(_abi, "LLA_ERR_" + status)
