"""Rotary positions and cache appends without a GPU: pins of the step oracle, the
frequencies of mla_rope_init against it, and the refusals of the C entries and of the
binding."""

import ctypes
import math

import numpy as np
import pytest

import deepseek_mla_decode_b200 as mla
from oracle import step_oracle as S


# ---- pins of the oracle ---------------------------------------------------------------
@pytest.mark.parametrize("half", [False, True])
def test_rotation_depends_on_the_distance_only(half):
    rng = np.random.default_rng(0)
    f = S.rope_freq_ref(10000.0)
    q, k = rng.standard_normal(64), rng.standard_normal(64)
    a = S.rotate_ref(q, 1000, f, half) @ S.rotate_ref(k, 990, f, half)
    b = S.rotate_ref(q, 10, f, half) @ S.rotate_ref(k, 0, f, half)
    assert abs(a - b) < 1e-10
    assert np.array_equal(S.rotate_ref(q, 0, f, half), q)
    assert abs(np.linalg.norm(S.rotate_ref(q, 77, f, half)) - np.linalg.norm(q)) < 1e-12


def test_rotation_by_hand():
    x = np.zeros(64)
    x[0], x[1] = 1.0, 0.0  # pair 0 turns one radian a position
    y = S.rotate_ref(x, 3, S.rope_freq_ref(10000.0), False)
    assert abs(y[0] - math.cos(3)) < 1e-15 and abs(y[1] - math.sin(3)) < 1e-15 and not y[2:].any()
    z = np.zeros(64)
    z[32] = 1.0  # second member of pair 0 in the half layout
    y = S.rotate_ref(z, 3, S.rope_freq_ref(10000.0), True)
    assert abs(y[0] + math.sin(3)) < 1e-15 and abs(y[32] - math.cos(3)) < 1e-15


def test_layouts_are_a_permutation_of_each_other():
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal(64), S.rope_freq_ref(500000.0)
    perm = np.arange(64).reshape(32, 2).T.reshape(-1)  # interleaved -> half
    assert np.allclose(S.rotate_ref(x, 55, f, False)[perm], S.rotate_ref(x[perm], 55, f, True), atol=1e-15)


def test_yarn_ends():
    plain, y = S.rope_freq_ref(10000.0), S.rope_freq_ref(10000.0, "yarn", factor=40.0)
    # the fastest pairs keep their frequency, the slowest are interpolated, none is outside
    assert np.array_equal(y[:8], plain[:8]) and np.allclose(y[-5:], plain[-5:] / 40, rtol=1e-14)
    assert np.all(y <= plain) and np.all(y >= plain / 40 * (1 - 1e-14))
    assert np.allclose(S.rope_freq_ref(10000.0, "yarn", factor=1.0), plain, rtol=1e-14)


def test_window_keys_by_hand():
    assert list(S.window_keys(9, 3, 2)) == [0, 1, 7, 8, 9]
    assert list(S.window_keys(2, 64, 0)) == [0, 1, 2]
    assert list(S.window_keys(4, 2, 4)) == [0, 1, 2, 3, 4]


def test_positions_by_hand():
    assert list(S.new_tokens([5, 1, 0], [2, 3, 1], 3)) == [(0, 0, 3), (0, 1, 4), (1, 2, 0)]


# ---- mla_rope_init --------------------------------------------------------------------
@pytest.mark.parametrize("kw", [
    dict(base=10000.0),
    dict(base=500000.0, scaling="linear", factor=8.0),
    dict(base=10000.0, scaling="yarn", factor=40.0),
    dict(base=10000.0, scaling="yarn", factor=4.0, original_len=32768.0, beta_fast=16.0, beta_slow=2.0),
    dict(base=10000.0, scaling="yarn", factor=40.0, original_len=5.0),   # every pair below beta_slow but the first
    dict(base=10000.0, scaling="yarn", factor=40.0, original_len=1e30),  # every pair above beta_fast
    dict(base=2.0, scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=1.0),
])
def test_frequencies(kw):
    r = mla.rope_params(layout="half", amplitude=1.25, **kw)
    # pow and log are within an ulp or two of each other across libraries
    assert np.allclose(np.array(r.freq), S.rope_freq_ref(**kw), rtol=1e-13, atol=0)
    assert r.amplitude == 1.25 and r.half_layout == 1


@pytest.mark.parametrize("kw", [
    dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(amplitude=float("inf")),
    dict(amplitude=1e39), dict(scaling="linear", factor=0.0), dict(scaling="linear", factor=float("nan")),
    dict(scaling="yarn", factor=-1.0), dict(scaling="yarn", factor=2.0, original_len=0.0),
    dict(scaling="yarn", factor=2.0, beta_slow=0.0), dict(scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0),
])
def test_bad_rotations_are_refused(kw):
    with pytest.raises(mla.MLAError) as e:
        mla.rope_params(**kw)
    assert e.value.code == 1


def test_bad_names_are_refused():
    with pytest.raises(ValueError):
        mla.rope_params(layout="neox")
    with pytest.raises(ValueError):
        mla.rope_params(scaling="dynamic")
    assert mla.load_library().mla_rope_init(None, 1e4, 0, 0, 1.0, 1.0, 1.0, 1.0, 1.0) == 1
    r = mla.Rope()
    assert mla.load_library().mla_rope_init(ctypes.byref(r), 1e4, 2, 0, 1.0, 1.0, 1.0, 1.0, 1.0) == 1
    assert mla.load_library().mla_rope_init(ctypes.byref(r), 1e4, 0, 3, 1.0, 1.0, 1.0, 1.0, 1.0) == 1


# ---- refusals before any device call --------------------------------------------------
P = 1 << 20  # a well-aligned address that nothing reads: every call below is refused


def rope_q_args(**kw):
    a = dict(q=P, stride=16 * 192, n=P, q_lens=None, B=2, s_q=3, H=16, rope=ctypes.byref(mla.rope_params()), heads=P,
             pe=P, status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(n=None), dict(rope=None), dict(heads=None), dict(pe=None), dict(B=0), dict(s_q=0), dict(H=0),
    dict(H=65536, stride=65536 * 192), dict(B=65536, s_q=32768), dict(stride=16 * 192 - 8), dict(stride=16 * 192 + 4),
    dict(q=P + 8), dict(heads=P + 2), dict(pe=P + 4), dict(n=P + 2), dict(q_lens=P + 1), dict(status=P + 2),
])
def test_rope_q_refusals(kw):
    assert mla.load_library().mla_rope_q(*rope_q_args(**kw)) == 1


def test_rope_with_unusable_frequencies_is_refused():
    L = mla.load_library()
    for change in (lambda r: r.freq.__setitem__(3, float("nan")), lambda r: r.freq.__setitem__(0, 1e7),
                   lambda r: setattr(r, "amplitude", float("nan")), lambda r: setattr(r, "half_layout", 2)):
        r = mla.rope_params()
        change(r)
        assert L.mla_rope_q(*rope_q_args(rope=ctypes.byref(r))) == 1
        a = rope_q_args(rope=ctypes.byref(r))
        assert L.mla_rope_inplace(*(a[:8] + a[10:])) == 1
        assert L.mla_append_kv(*append_args(rope=ctypes.byref(r))) == 1


def append_args(**kw):
    a = dict(kv_a=P, stride=576, weight=P, eps=1e-6, table=P, max_blocks=4, n=P, q_lens=None, B=2, s_q=3, rope=None,
             cache=P, num_blocks=8, status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(kv_a=None), dict(table=None), dict(n=None), dict(cache=None), dict(stride=568), dict(stride=580),
    dict(max_blocks=0), dict(num_blocks=0), dict(num_blocks=1 << 31), dict(B=0), dict(s_q=0), dict(B=65536, s_q=32768),
    dict(eps=-1.0), dict(eps=float("nan")), dict(kv_a=P + 8), dict(weight=P + 2), dict(cache=P + 8), dict(table=P + 2),
    dict(n=P + 1), dict(q_lens=P + 2), dict(status=P + 3),
])
def test_append_refusals(kw):
    for fn in ("mla_append_kv", "mla_append_kv_fp8"):
        assert getattr(mla.load_library(), fn)(*append_args(**kw)) == 1


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    rope = mla.rope_params()
    n = torch.ones(2, dtype=i32)
    with pytest.raises(ValueError):
        mla.rope_q(torch.zeros(2, 1, 4, 128, dtype=bf), n, rope)
    with pytest.raises(ValueError):
        mla.rope_q(torch.zeros(2, 1, 4, 192), n, rope)
    with pytest.raises(ValueError, match="CUDA"):
        mla.rope_q(torch.zeros(2, 1, 4, 192, dtype=bf), n, rope)
    with pytest.raises(ValueError, match="contiguous"):
        mla.rope_inplace(torch.zeros(2, 1, 192, 4, dtype=bf).transpose(2, 3), n, rope)
    with pytest.raises(ValueError, match="evenly"):
        mla.rope_inplace(torch.zeros(4, 3, 4, 192, dtype=bf)[:, :2], n, rope)
    cache, table = torch.zeros(3, 64, 576, dtype=bf), torch.zeros(2, 2, dtype=i32)
    with pytest.raises(ValueError):
        mla.append_kv(torch.zeros(2, 1, 512, dtype=bf), cache, table, n)
    with pytest.raises(ValueError):
        mla.append_kv(torch.zeros(2, 1, 576, dtype=bf), torch.zeros(3, 64, 656, dtype=torch.uint8), table, n)
    with pytest.raises(ValueError, match="CUDA"):
        mla.append_kv(torch.zeros(2, 1, 576, dtype=bf), cache, table, n)


# ---- windowed decode ------------------------------------------------------------------
def window_args(**kw):
    a = dict(q_nope=P, q_pe=P, cache=P, num_blocks=8, table=P, max_blocks=4, n=P, q_lens=None, B=2, s_q=2, H=16,
             scale=0.1, window=64, sinks=0, meta=P, meta_bytes=1 << 30, ws=P, ws_bytes=1 << 40, out=P, lse=P,
             status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("code,kw", [
    (1, dict(q_nope=None)), (1, dict(q_pe=None)), (1, dict(cache=None)), (1, dict(table=None)), (1, dict(n=None)),
    (1, dict(meta=None)), (1, dict(out=None)), (1, dict(lse=None)), (1, dict(sinks=-1)), (1, dict(max_blocks=0)),
    (1, dict(num_blocks=0)), (1, dict(scale=0.0)), (1, dict(scale=float("nan"))), (1, dict(q_lens=P + 2)),
    (1, dict(out=P + 8)), (1, dict(lse=P + 1)), (1, dict(status=P + 1)),
    (2, dict(window=63)), (2, dict(window=0)), (2, dict(window=-64)), (2, dict(H=48)), (2, dict(s_q=5)), (2, dict(B=0)),
    (2, dict(B=40000, s_q=2)), (4, dict(meta_bytes=100)),
])
def test_window_refusals(code, kw):
    for fn in ("mla_decode_window", "mla_decode_fp8_window"):
        assert getattr(mla.load_library(), fn)(*window_args(**kw)) == code


@pytest.mark.parametrize("code,kw", [
    (1, dict(n=None)), (1, dict(meta=None)), (1, dict(meta=P + 4)), (1, dict(n=P + 2)), (1, dict(q_lens=P + 2)),
    (1, dict(sinks=-1)), (2, dict(window=63)), (2, dict(s_q=5)), (2, dict(H=20)), (2, dict(B=65536, s_q=2)),
    (4, dict(meta_bytes=16)),
])
def test_window_metadata_refusals(code, kw):
    a = dict(n=P, q_lens=None, B=2, s_q=2, H=16, window=64, sinks=4, meta=P, meta_bytes=1 << 20, stream=None)
    a.update(kw)
    assert mla.load_library().mla_get_metadata_window(*a.values()) == code


@pytest.mark.parametrize("window,sinks", [(2**32 + 100, 4), (2**31, 0), (100, 2**32), (100, 2**31)])
def test_window_sizes_beyond_an_int_are_refused(window, sinks):
    """A C int would cut them: 2^32 + 100 keys to 100."""
    torch = pytest.importorskip("torch")
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        mla.get_metadata_window(n, None, 1, 16, window, sinks)
    q = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16)
    for call, cache in ((mla.decode_window, torch.zeros(1, 64, 576, dtype=torch.bfloat16)),
                        (mla.decode_fp8_window, torch.zeros(1, 64, 656, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="2\\^31"):
            call(q, q[..., :64].contiguous(), cache, torch.zeros(2, 1, dtype=torch.int32), n, None, 0.1, window, sinks, n)


@pytest.mark.parametrize("s_q,H,window,sinks", [
    (1, 16, -(2**32) + 100, 4), (1, 16, 100, -(2**32) + 4), (1, 16, -(2**31) - 1, 0), (1, 16, 100, -(2**40)),
    (2**32 + 1, 16, 100, 4), (1, 2**32 + 16, 100, 4), (-(2**32) + 1, 16, 100, 4), (1, -(2**32) + 16, 100, 4),
])
def test_window_sizes_below_an_int_and_shapes_beyond_one_are_refused(s_q, H, window, sinks):
    """A C int would cut them too: -2^32 + 100 keys to 100, 2^32 + 16 heads to 16."""
    torch = pytest.importorskip("torch")
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        mla.get_metadata_window(n, None, s_q, H, window, sinks)
    if (s_q, H) == (1, 16):
        q = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16)
        for call, cache in ((mla.decode_window, torch.zeros(1, 64, 576, dtype=torch.bfloat16)),
                            (mla.decode_fp8_window, torch.zeros(1, 64, 656, dtype=torch.uint8))):
            with pytest.raises(ValueError, match="2\\^31"):
                call(q, q[..., :64].contiguous(), cache, torch.zeros(2, 1, dtype=torch.int32), n, None, 0.1, window,
                     sinks, n)
