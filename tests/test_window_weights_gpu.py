"""GPU tests of the windowed decode where one key takes most of the weight, as the first keys that
stay visible do: the thousands of small weights that share the rest must arrive, for the values
they carry may be all there is to see.

What is allowed.  Over the FP8 cache the kernel holds the weight of a key, times the key's scale (P = w s), in two
terms whose unit follows the largest P of its tile of 256 keys.  A weight is off by at most half
a step of bf16's eight bits, 2^-8 P (the four bits of e4m3 and the three and a sign of e5m2), or
2^-20 of the tile's largest where that is more (e5m2's half step 2^-14 below 2^-10, the largest
kept at 2^6 or above), and never by more than P itself.  Added up over the keys this bounds an
output, with the bf16 rounding of the result (2^-8) and 2^-14 of sum |w c| for what fp32 scores,
exponentials and sums of a few dozen bits' range leave.  Over the bf16 cache a weight is off by
2^-8 of itself, and so is their sum, which is of the rounded ones.  Neither bound grows with the
number of keys."""

import numpy as np
import pytest

from oracle import mla_fp8_oracle as F
from oracle import mla_oracle as O
from oracle import step_oracle as S
from deepseek_mla_decode_b200.workloads import SCALE_192, f32_to_bf16_bits
from mla_testlib import compare

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import deepseek_mla_decode_b200 as mla  # noqa: E402

TILE = 256


def dev(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).cuda()


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class OneKeyAhead:
    """n keys whose values share the mean 0.5 and one at position `at` of mean -0.5 in the first
    256 dims and zeros in the others, ahead of them by 8 to 13 nats from the first head to the
    last (and some heads by 0, 5, 16 and 20).  All sequences read the same blocks; sequence b
    has the queries of set b % sets."""

    def __init__(self, n, at, H=16, sets=2, spread=0.0, value=1.0, seed=0, fp8=True):
        rng = np.random.default_rng(seed)
        self.n, self.at, self.H, self.sets, self.fp8 = n, at, H, sets, fp8
        blocks = (n + 63) // 64
        rows = np.zeros((blocks * 64, 576), dtype=np.float32)
        rows[:n, :512] = 0.5 + 0.5 * rng.standard_normal((n, 512), dtype=np.float32)
        rows[:n, 514:] = rng.standard_normal((n, 62), dtype=np.float32)
        rows[at, :256] = value * (-0.5 + 0.5 * rng.standard_normal(256, dtype=np.float32))
        rows[at, 256:] = 0
        rows[at, 512] = 4.0
        order = rng.permutation(blocks)
        self.table = np.argsort(order)
        self.kv = f32_to_bf16_bits(rows).reshape(blocks, 64, 576)[order]
        if fp8:
            self.packed = F.pack_cache(self.kv)
            self.scales = F.unpack_cache(self.packed)[2][self.table].reshape(-1)[:n].astype(np.float64)
        store = F.dequantize_cache(self.packed) if fp8 else O.bf16_to_f64(self.kv)
        self.rows = store[self.table].reshape(-1, 576)[:n]
        lead = np.linspace(8, 13, H)
        lead[[1, 3, H // 2, H - 2]] = 0, 5, 16, 20
        q_pe = np.zeros((sets, 1, H, 64), dtype=np.float32)
        q_pe[..., 0] = lead / (SCALE_192 * 4.0)
        q_pe[..., 2:] = spread / (SCALE_192 * np.sqrt(62)) * rng.standard_normal((sets, 1, H, 62))
        self.q_pe = f32_to_bf16_bits(q_pe)
        self.q_nope = f32_to_bf16_bits(np.zeros((sets, 1, H, 512), dtype=np.float32))

    def run(self, B, window, sinks, tokens=False):
        n = i32([self.n] * B)
        pick = np.arange(B) % self.sets
        args = (dev(self.q_nope[pick]), dev(self.q_pe[pick]), torch.from_numpy(self.packed).cuda() if self.fp8 else dev(self.kv),
                i32(np.tile(self.table, (B, 1))), n, None, SCALE_192)
        if tokens:
            out, lse = mla.decode_fp8_tokens(*args, True, mla.get_metadata_tokens(n, None, 1, self.H, True))
            splits = None
        else:
            meta = mla.get_metadata_window(n, None, 1, self.H, window, sinks)
            splits = meta.cpu().numpy()[16 + 4 * 256 + 2 * B:][:B]
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            fn = mla.decode_fp8_window if self.fp8 else mla.decode_window
            out, lse = fn(*args, window, sinks, meta, status=status)
            assert int(status.item()) == 0
        return out.float().cpu().double().numpy(), lse.cpu().double().numpy(), splits

    def reference(self, window, sinks, whole):
        """out, lse and the bound of every output; whole: a sequence's keys are one piece."""
        q = np.concatenate([O.bf16_to_f64(self.q_nope), O.bf16_to_f64(self.q_pe)], -1)[:, 0]
        ref = S.window_decode_ref(O.bf16_to_f64(self.q_nope), O.bf16_to_f64(self.q_pe), lambda b, t: self.rows[t],
                                  [self.n] * self.sets, None, SCALE_192, window, sinks)
        t = S.window_keys(self.n - 1, window, sinks)
        w = np.exp(SCALE_192 * (q @ self.rows[t].T) - ref[1][:, 0][..., None])  # [sets, H, keys]
        c = np.abs(self.rows[t, :512])
        rounding = (2.0 ** -14 * (w @ c))[:, None] + 2.0 ** -8 * np.abs(ref[0])
        if not self.fp8:
            return ref[0], ref[1], rounding + 2.0 ** -8 * ((w @ c)[:, None] + np.abs(ref[0]))
        P = w * self.scales[t]
        if whole:
            # tiles of four blocks in the order of visible blocks; a block that first keys and
            # window share counts for each, unless nothing is hidden between them
            near = (t >= self.n - window) | (self.n - window <= sinks)
            first = np.unique(t[~near] // 64)
            block = np.where(near, len(first) + t // 64 - t[near][0] // 64, np.searchsorted(first, t // 64))
            tile = block // 4
            top = np.stack([P[..., tile == k].max(-1) for k in range(tile[-1] + 1)], -1)[..., tile]
        else:  # pieces may begin at any block: the largest of the keys within a tile's reach
            top = P.copy()
            for d in range(1, TILE):
                top[..., d:] = np.maximum(top[..., d:], P[..., :-d])
                top[..., :-d] = np.maximum(top[..., :-d], P[..., d:])
        err = np.minimum(P, np.maximum(2.0 ** -8 * P, 2.0 ** -20 * top)) / self.scales[t]
        return ref[0], ref[1], (err @ c)[:, None] + rounding

    def check(self, B, window, sinks, bars=True):
        out, lse, splits = self.run(B, window, sinks)
        ref, ref_lse, lim = self.reference(window, sinks, whole=splits.max() == 1)
        pick = np.arange(B) % self.sets
        over = np.abs(out - ref[pick]) / lim[pick]
        assert over.max() <= 1.0, f"error over its bound: {over.max()}"
        if bars:
            compare(out, lse, ref[pick], ref_lse[pick], what=f"{self.n} keys, {self.at} ahead")
        else:
            assert np.abs(lse - ref_lse[pick]).max() <= 1e-3
        return splits


def whole_batch():
    """Sequences of one length that the schedule leaves in one piece each: two a partition."""
    return 2 * (mla.device_sm_count() // 2)


@pytest.mark.parametrize("spread", [0.0, 1.0], ids=["equal", "normal"])
@pytest.mark.parametrize("n,window,sinks", [(4099, 4096, 3), (4096, 1 << 20, 0), (32800, 32768, 32), (32768, 1 << 20, 0)])
def test_first_key_ahead_of_a_long_window(n, window, sinks, spread):
    p = OneKeyAhead(n, 0, spread=spread, seed=n)
    assert p.check(whole_batch(), window, sinks).max() == 1


@pytest.mark.parametrize("n,window,sinks", [(4099, 4096, 3), (32800, 32768, 32)])
def test_first_key_ahead_of_a_long_window_bf16(n, window, sinks):
    p = OneKeyAhead(n, 0, spread=1.0, seed=n, fp8=False)
    p.check(whole_batch(), window, sinks)
    p.check(5, window, sinks)


@pytest.mark.parametrize("at", [4098, 2000, 3], ids=["last", "middle", "window_start"])
def test_the_key_ahead_anywhere(at):
    p = OneKeyAhead(4099, at, spread=1.0, seed=at)
    assert p.check(whole_batch(), 4096, 3).max() == 1


@pytest.mark.parametrize("B", [3, 100])
def test_the_key_ahead_in_split_sequences(B):
    p = OneKeyAhead(8200, 1, spread=0.5, seed=B)
    assert p.check(B, 8192, 4).max() > 1


def test_the_key_ahead_with_a_larger_scale():
    """Its row 2^7 times the others': its own values are rounded coarsely, but where they are
    zero the others are what is seen."""
    p = OneKeyAhead(4099, 0, spread=1.0, value=128.0, seed=5)
    p.check(whole_batch(), 4096, 3, bars=False)


def test_all_heads_of_a_tile():
    p = OneKeyAhead(4200, 0, H=128, sets=1, spread=2.0, seed=6)
    p.check(whole_batch(), 4096, 16)


@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_a_window_beyond_the_lengths_is_the_plain_decode(spread):
    """decode_fp8_tokens holds its weights in bf16 whatever their size: each of the two is
    within its bound of the exact result (the plain one's is the smaller)."""
    p = OneKeyAhead(6000, 0, spread=spread, seed=7)
    B = whole_batch()
    out, lse, _ = p.run(B, 6000, 0)
    plain, plain_lse, _ = p.run(B, 0, 0, tokens=True)
    lim = p.reference(6000, 0, whole=True)[2][np.arange(B) % p.sets]
    assert np.all(np.abs(out - plain) <= 2 * lim)
    assert np.abs(lse - plain_lse).max() <= 1e-3


def test_units_that_fall_and_rise():
    """Tiles of very different weight in any order: 60 bits between the smallest and the
    largest, and the sum of many small tiles after and before a large one."""
    p = OneKeyAhead(2048 + 40, 700, spread=6.0, seed=8)
    p.check(whole_batch(), 2048, 40)
    p = OneKeyAhead(2048 + 40, 1300, spread=14.0, seed=9)
    p.check(whole_batch(), 2048, 40)


# ---- query and rotary terms ------------------------------------------------------------
@pytest.mark.parametrize("outlier", [2.0 ** 10, 2.0 ** 11])
def test_a_query_channel_far_above_the_others(outlier):
    """A channel that meets only zeros in the cache sets the power of two of a query row and adds
    nothing; the others are 2^-10 and 2^-11 of it, 2^-3 and 2^-4 in units where it is 2^7.  The
    terms of a bf16 value are exact from 2^-6 up and off by at most 2^-14 below, 2^-21 of the
    outlier: 2^-10 at most here, on the smaller values of a row.  A score of 575 such products is
    then off by SCALE_192 sqrt(575) 2^-10 / sqrt(3) = 1e-3 at most (one standard deviation), and
    the lse, a weighted mean of a few dozen keys' errors, by 2e-4: inside the usual bars, which
    terms with steps of 2^-9 in these units miss by a factor of ten."""
    n, B, H = 700, 4, 16
    rng = np.random.default_rng(int(np.log2(outlier)))
    rows = rng.standard_normal((11 * 64, 576), dtype=np.float32)
    rows[:, 7] = 0
    packed = F.pack_cache(f32_to_bf16_bits(rows).reshape(11, 64, 576))
    store = F.dequantize_cache(packed).reshape(-1, 576)
    q = rng.standard_normal((B, 1, H, 576), dtype=np.float32)
    q[..., 7] = outlier
    qn, qp = f32_to_bf16_bits(q[..., :512]), f32_to_bf16_bits(q[..., 512:])
    nt = i32([n] * B)
    meta = mla.get_metadata_window(nt, None, 1, H, 512, 100)
    out, lse = mla.decode_fp8_window(dev(qn), dev(qp), torch.from_numpy(packed).cuda(),
                                     i32(np.tile(np.arange(11), (B, 1))), nt, None, SCALE_192, 512, 100, meta)
    ref, ref_lse = S.window_decode_ref(O.bf16_to_f64(qn), O.bf16_to_f64(qp), lambda b, t: store[t], [n] * B, None,
                                       SCALE_192, 512, 100)
    compare(out.float().cpu().double().numpy(), lse.cpu().double().numpy(), ref, ref_lse, what=f"outlier {outlier}")
