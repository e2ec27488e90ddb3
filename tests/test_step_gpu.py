"""GPU tests of rotary queries and cache appends against the float64 oracle.

Tolerances.  A result is rounded once, to half a step: bf16 2^-8, e4m3 2^-4 of its value
(below the e4m3 normal range half of 2^-9 in units of the scale).  Before that:
* rotation: the angle is off by at most pi 2^-24 = 2^-22.3 (the reduced fraction in fp32) and
  the fast cos / sin by 2^-21.2, together 2^-20.6 of each operand; with the fp32 multiplies
  and adds the sum of two products is off by less than 2^-20 (|a| + |b|) amplitude;
* norm: 512 squares in a tree 16 + 5 deep, rsqrt (2 ulp) and two multiplies: under 2^-19 of
  the value."""

import numpy as np
import pytest

from oracle import mla_fp8_oracle as F
from oracle import mla_oracle as O
from oracle import step_oracle as S
from deepseek_mla_decode_b200.workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import deepseek_mla_decode_b200 as mla  # noqa: E402

ROTATIONS = [dict(), dict(layout="half"), dict(scaling="yarn", factor=40.0, amplitude=1.25),
             dict(layout="half", scaling="linear", factor=8.0, base=500000.0)]


def bits(shape, seed, scale=1.0):
    return f32_to_bf16_bits((np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32))


def dev(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).cuda()


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def f64(t):
    return t.float().cpu().double().numpy()


def oracle_rotation(kw):
    kw = dict(kw)
    half, amp = kw.pop("layout", "interleaved") == "half", kw.pop("amplitude", 1.0)
    return dict(freq=S.rope_freq_ref(kw.pop("base", 10000.0), **kw), half=half, amplitude=amp)


def rope_slack(x, half, amp):
    """2^-20 (|a| + |b|) amplitude for both members of each pair of x [..., 64]."""
    a, b = S._members(half)
    y = np.empty_like(x)
    y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y * (abs(amp) * 2.0 ** -20)


def check_bf16(got, ref, slack, what):
    err = np.abs(got - ref)
    lim = 2.0 ** -8 * np.abs(ref) + slack * (1 + 2.0 ** -8)
    assert np.all(err <= lim), (what, float((err - lim).max()), float(err.max()))


# ---- queries --------------------------------------------------------------------------
@pytest.mark.parametrize("kw", ROTATIONS)
@pytest.mark.parametrize("s_q,H,lens,q_lens", [
    (1, 16, [130], None),
    (1, 128, [1, 64, 70000, 2**31 - 1], None),
    (3, 5, [9, 2, 0, 400], None),           # fewer cached tokens than new ones: no place
    (4, 33, [4, 100, 1000, 7], [4, 0, 2, 3]),
    (200, 1, [200, 131072], [200, 77]),
    (700, 40, [700, 5000, -1, 3, 900], [700, 3, 1, 5, 701]),  # padding and invalid counts past the GPU's warps
])
def test_rope_q(kw, s_q, H, lens, q_lens):
    q = bits((len(lens), s_q, H, 192), seed=H)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    heads, pe = mla.rope_q(dev(q), i32(lens), mla.rope_params(**kw), q_lens=None if q_lens is None else i32(q_lens),
                           status=status)
    x, rot = O.bf16_to_f64(q), oracle_rotation(kw)
    bad = [n < 0 or (q_lens is not None and not 0 <= q_lens[b] <= s_q) for b, n in enumerate(lens)]
    counts = None if q_lens is None else [0 if w else c for w, c in zip(bad, q_lens)]
    ref_heads, ref_pe = S.rope_q_ref(x, lens, counts, **rot)
    ref_heads[bad], ref_pe[bad] = np.nan, np.nan
    assert int(status.item()) == (mla.MLA_DEVICE_ERR_SEQLEN if any(bad) else 0)
    assert np.array_equal(f64(heads), ref_heads, equal_nan=True)
    assert np.array_equal(np.isnan(f64(pe)), np.isnan(ref_pe))
    ref_pe[bad], pe[bad] = 0, 0
    check_bf16(f64(pe), ref_pe, rope_slack(x[..., 128:], rot["half"], rot["amplitude"]) * (ref_pe != 0), "q_pe")


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_q_of_a_projection_slice_and_in_place(layout):
    """A strided q gives the bits of its contiguous copy, and so does the rotation in place,
    which leaves everything but the rotary parts as it was."""
    B, s_q, H = 3, 2, 7
    wide = dev(bits((B, s_q, H * 192 + 40), seed=5))
    q = wide[..., 16:16 + H * 192].unflatten(-1, (H, 192))
    lens, r = i32([5, 900, 3]), mla.rope_params(layout=layout)
    heads, pe = mla.rope_q(q, lens, r)
    heads2, pe2 = mla.rope_q(q.contiguous(), lens, r)
    assert torch.equal(heads, heads2) and torch.equal(pe, pe2)
    want = wide.clone()
    want[..., 16:16 + H * 192].unflatten(-1, (H, 192))[..., 128:] = pe
    mla.rope_inplace(q, lens, r)
    assert torch.equal(wide, want)


def test_rope_in_place_with_padding_past_the_gpus_warps():
    q = dev(bits((4, 700, 33, 192), seed=9))
    lens, q_lens, r = i32([700, 5000, -1, 3]), i32([700, 3, 1, 5]), mla.rope_params(layout="half")
    _, pe = mla.rope_q(q, lens, r, q_lens=q_lens)
    want = q.clone()
    want[..., 128:] = pe
    mla.rope_inplace(q, lens, r, q_lens=q_lens)
    assert torch.equal(torch.nan_to_num(q, 777.0), torch.nan_to_num(want, 777.0))


def test_rope_q_invalid_lengths_and_counts():
    q = dev(bits((4, 2, 3, 192), seed=6))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    heads, pe = mla.rope_q(q, i32([5, -1, 7, 9]), mla.rope_params(), q_lens=i32([2, 1, 3, -1]), status=status)
    assert int(status.item()) == mla.MLA_DEVICE_ERR_SEQLEN
    assert torch.isnan(heads[1:]).all() and torch.isnan(pe[1:]).all()
    good = mla.rope_q(q, i32([5, 5, 7, 9]), mla.rope_params())
    assert torch.equal(heads[0], good[0][0]) and torch.equal(pe[0], good[1][0])


def test_rope_q_on_another_stream_and_in_a_graph():
    B, H = 5, 16
    q, n, r = dev(bits((B, 1, H, 192), seed=8)), i32([1, 2, 300, 4, 5]), mla.rope_params()
    heads, pe = torch.empty(B, 1, H, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(
        B, 1, H, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mla.rope_q(q, n, r, q_heads=heads, q_pe=pe, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want = mla.rope_q(q, n, r)
    assert torch.equal(heads, want[0]) and torch.equal(pe, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.rope_q(q, n, r, q_heads=heads, q_pe=pe)
    n.add_(1000)
    g.replay()
    want = mla.rope_q(q, n, r)
    assert torch.equal(heads, want[0]) and torch.equal(pe, want[1])


# ---- appends --------------------------------------------------------------------------
def make_append(lens, s_q, seed, spare_cols=1):
    """kv_a bits, table, and the number of blocks; unused table entries point nowhere valid."""
    rng = np.random.default_rng(seed)
    nblk = [(n + 63) // 64 for n in lens]
    total = sum(nblk) + 2
    perm, cur = rng.permutation(total), 0
    table = np.full((len(lens), max(nblk) + spare_cols), 2**30, dtype=np.int32)
    for b, k in enumerate(nblk):
        table[b, :k] = perm[cur:cur + k]
        cur += k
    return bits((len(lens), s_q, 576), seed + 1), table, total


APPENDS = [
    (1, [130], None),
    (1, [1, 64, 65, 70000], None),
    (3, [9, 2, 0, 400], None),
    (4, [4, 100, 1000, 7], [4, 0, 2, 3]),
    (150, [150, 1000, 129], [150, 77, 129]),  # whole blocks and ragged ends
    (2500, [2500, 3000, 100], [2500, 17, 100]),  # more rows than the GPU holds warps, most of them padding
]


@pytest.mark.parametrize("kw", ROTATIONS + [None])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("s_q,lens,q_lens", APPENDS)
def test_append_bf16(kw, norm, s_q, lens, q_lens):
    kv_a, table, blocks = make_append(lens, s_q, seed=31)
    w = bits(512, 3) if norm else None
    cache = dev(bits((blocks, 64, 576), 4))
    before = f64(cache)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mla.append_kv(dev(kv_a), cache, i32(table), i32(lens), rope=mla.rope_params(**kw) if kw is not None else None,
                        norm_weight=dev(w) if norm else None, eps=1e-5,
                        q_lens=None if q_lens is None else i32(q_lens), status=status)
    assert got is cache and int(status.item()) == 0
    after = f64(cache)
    x = O.bf16_to_f64(kv_a)
    rot = oracle_rotation(kw) if kw is not None else {}
    rows = S.append_rows_ref(x, lens, q_lens, weight=O.bf16_to_f64(w) if norm else None, eps=1e-5, **rot)
    for (b, i, p), ref in rows.items():
        row = after[table[b, p // 64], p % 64]
        slack = np.abs(ref) * (2.0 ** -19 if norm else 0.0)
        slack[512:] = rope_slack(x[b, i, 512:], rot["half"], rot["amplitude"]) if kw is not None else 0.0
        check_bf16(row, ref, slack, (b, i, p))
        if not norm:
            assert np.array_equal(row[:512], x[b, i, :512])
        before[table[b, p // 64], p % 64] = row
    assert np.array_equal(before, after)  # nothing else was written


@pytest.mark.parametrize("kw", [ROTATIONS[1], ROTATIONS[2]])
@pytest.mark.parametrize("s_q,lens,q_lens", APPENDS)
def test_append_fp8(kw, s_q, lens, q_lens):
    kv_a, table, blocks = make_append(lens, s_q, seed=32)
    w = bits(512, 3)
    cache = torch.full((blocks, 64, 656), 0x55, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.append_kv_fp8(dev(kv_a), cache, i32(table), i32(lens), rope=mla.rope_params(**kw), norm_weight=dev(w), eps=1e-5,
                      q_lens=None if q_lens is None else i32(q_lens), status=status)
    assert int(status.item()) == 0
    after = cache.cpu().numpy()
    x, rot = O.bf16_to_f64(kv_a), oracle_rotation(kw)
    rows = S.append_rows_ref(x, lens, q_lens, weight=O.bf16_to_f64(w), eps=1e-5, **rot)
    rest = np.ones(after.shape[:2], bool)
    for (b, i, p), ref in rows.items():
        at = table[b, p // 64], p % 64
        rest[at] = False
        row = after[at]
        scale = float(row[640:644].view(np.float32)[0])
        slack = np.abs(ref) * 2.0 ** -19
        slack[512:] = rope_slack(x[b, i, 512:], rot["half"], rot["amplitude"])
        amax = np.abs(ref).max()
        assert abs(scale * 448 - amax) <= slack.max() + amax * 2.0 ** -22
        codes = F.e4m3_decode(row[:512])
        # the quotient by the computed scale, rounded once
        unit = ref / scale
        lim = np.maximum(2.0 ** -4 * np.abs(unit), 2.0 ** -10) + slack / scale * (1 + 2.0 ** -4) + np.abs(unit) * 2.0 ** -22
        assert np.all(np.abs(codes - unit[:512]) <= lim[:512])
        pe = O.bf16_to_f64(row[512:640].view(np.uint16))
        lim = 2.0 ** -8 * np.abs(unit) + slack / scale * (1 + 2.0 ** -8) + np.abs(unit) * 2.0 ** -22
        assert np.all(np.abs(pe - unit[512:]) <= lim[512:])
        assert not row[644:].any()
    assert np.all(after[rest] == 0x55)


def test_append_fp8_without_norm_and_rotation_is_the_quantiser():
    lens = [64, 200, 3]
    kv_a, table, blocks = make_append(lens, 200, seed=33)
    kv_a[0, 1] = 0                      # a row of zeros
    kv_a[0, 2, :] = bits(576, 9, 1e-38)  # the smallest scales
    kv_a[0, 3, 5] = 0x7F80              # an infinity
    cache = torch.zeros(blocks, 64, 656, dtype=torch.uint8, device="cuda")
    x = dev(kv_a)
    mla.append_kv_fp8(x, cache, i32(table), i32(lens), q_lens=i32(lens))
    packed = mla.quantize_kv_fp8(x)
    for b, n in enumerate(lens):
        rows = cache[torch.from_numpy(table[b, :(n + 63) // 64]).long().cuda()].view(-1, 656)[:n]
        assert torch.equal(rows, packed[b, :n])


def test_append_fp8_keeps_a_nan():
    kv_a, table, blocks = make_append([3], 3, seed=34)
    kv_a[0, 0, 9] = 0x7FC0
    kv_a[0, 1, :] = 0x7FC0
    cache = torch.zeros(blocks, 64, 656, dtype=torch.uint8, device="cuda")
    mla.append_kv_fp8(dev(kv_a), cache, i32(table), i32([3]))
    scale = cache[int(table[0, 0]), :3, 640:644].contiguous().view(torch.float32).flatten()
    assert torch.isnan(scale[:2]).all() and torch.isfinite(scale[2])


@pytest.mark.parametrize("fp8", [False, True])
def test_append_errors_leave_the_rest(fp8):
    lens = [100, 70, 5, 64, 8]
    kv_a, table, blocks = make_append(lens, 2, seed=35, spare_cols=0)
    x, good = dev(kv_a), table.copy()
    table[1, 1] = blocks        # one past the pool
    table[3, 0] = -1
    n = [100, 70, -5, 64, 10**6]  # and lengths below zero and past the table
    width, dtype = (656, torch.uint8) if fp8 else (576, torch.bfloat16)
    append = mla.append_kv_fp8 if fp8 else mla.append_kv
    cache = torch.zeros(blocks, 64, width, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    append(x, cache, i32(table), i32(n), rope=mla.rope_params(), status=status)
    assert int(status.item()) == mla.MLA_DEVICE_ERR_SEQLEN | mla.MLA_DEVICE_ERR_BLOCK_ID
    want = torch.zeros_like(cache)
    append(x, want, i32(good), i32(lens), rope=mla.rope_params(), q_lens=i32([2, 0, 0, 0, 0]))
    assert torch.equal(cache, want)
    # counts out of range write nothing
    cache.zero_()
    append(x, cache, i32(good), i32(lens), q_lens=i32([3, -1, 3, 5, 99]))
    assert not cache.any()


def test_append_of_a_slice_on_another_stream_and_in_a_graph():
    lens = [70, 3, 64]
    kv_a, table, blocks = make_append(lens, 3, seed=36)
    wide = torch.zeros(3, 3, 1536 + 576 + 8, dtype=torch.bfloat16, device="cuda")
    x = wide[..., 1536:1536 + 576]
    x.copy_(dev(kv_a))
    t, n, w, r = i32(table), i32(lens), dev(bits(512, 3)), mla.rope_params()
    cache = torch.zeros(blocks, 64, 576, dtype=torch.bfloat16, device="cuda")
    want = mla.append_kv(x.contiguous(), cache.clone(), t, n, rope=r, norm_weight=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mla.append_kv(x, cache, t, n, rope=r, norm_weight=w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(cache, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.append_kv(x, cache, t, n, rope=r, norm_weight=w)
    cache.zero_()
    n.sub_(2)
    g.replay()
    want = mla.append_kv(x, torch.zeros_like(cache), t, n, rope=r, norm_weight=w)
    assert torch.equal(cache, want)


def test_append_past_32_bits_of_bytes():
    """A block whose rows lie beyond 2^32 bytes of the pool (and 2^31 elements)."""
    blocks = 60000  # 4.42e9 bytes
    cache = torch.empty(blocks, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache[-1].zero_()
    kv_a = bits((1, 2, 576), 40)
    mla.append_kv(dev(kv_a), cache, i32([[blocks - 1]]), i32([64]))
    assert torch.equal(cache[-1, 62:], dev(kv_a)[0]) and not cache[-1, :62].any()
