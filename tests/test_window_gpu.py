"""GPU tests of the windowed decode (mla_get_metadata_window with mla_decode_window /
mla_decode_fp8_window) against the float64 oracle.  In every case the rows that no token
sees hold NaN and the table entries of blocks without a visible key point outside the pool.
Tolerances as in test_decode_gpu.py (the arithmetic is that decode's)."""

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

NOWHERE = 2**30


def bits(rng, shape):
    return f32_to_bf16_bits(rng.standard_normal(shape, dtype=np.float32))


def dev(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).cuda()


def i32(x):
    return None if x is None else torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class Problem:
    """Only blocks with a visible key exist; rows hidden from every token are NaN."""

    def __init__(self, lens, s_q, H, window, sinks, q_lens=None, seed=0):
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.lens, self.q_lens, self.window, self.sinks, self.H, self.s_q = lens, q_lens, window, sinks, H, s_q
        self.table = np.full((B, max((max(lens) + 63) // 64, 1) + 1), NOWHERE, dtype=np.int64)
        seen = [np.zeros(max(n, 0), bool) for n in lens]
        for b, i, p in S.new_tokens(lens, q_lens, s_q):
            seen[b][S.window_keys(p, window, sinks)] = True
        used = [np.unique(np.nonzero(v)[0] // 64) for v in seen]
        blocks = sum(len(u) for u in used) + 1
        perm, cur = rng.permutation(blocks), 0
        self.kv = np.full((blocks, 64, 576), f32_to_bf16_bits(np.array([np.nan], np.float32))[0])
        for b, u in enumerate(used):
            self.table[b, u] = perm[cur:cur + len(u)]
            cur += len(u)
            t = np.nonzero(seen[b])[0]
            self.kv[self.table[b, t // 64], t % 64] = bits(rng, (len(t), 576))
        self.q_nope, self.q_pe = bits(rng, (B, s_q, H, 512)), bits(rng, (B, s_q, H, 64))

    def packed(self):
        """The FP8 cache, with NaN codes, keys and scales in the hidden rows."""
        hidden = np.isnan(O.bf16_to_f64(self.kv[..., 0]))
        kv = self.kv.copy()
        kv[hidden] = 0
        packed = F.pack_cache(kv)
        packed[hidden] = 0x7F  # e4m3 NaN; as bf16 and fp32 bytes 0x7F7F.. finite, so set those
        packed[hidden, 512:640] = np.tile(np.array([0xC0, 0x7F], np.uint8), 64)
        packed[hidden, 640:644] = np.array([0, 0, 0xC0, 0x7F], np.uint8)
        return packed

    def rows_of(self, fp8):
        store = F.dequantize_cache(self.packed()) if fp8 else O.bf16_to_f64(self.kv)
        return lambda b, t: store[self.table[b, t // 64], t % 64]

    def reference(self, fp8=False):
        return S.window_decode_ref(O.bf16_to_f64(self.q_nope), O.bf16_to_f64(self.q_pe), self.rows_of(fp8), self.lens,
                                   self.q_lens, SCALE_192, self.window, self.sinks)

    def run(self, fp8=False, status=None, **kw):
        n, ql = i32(self.lens), i32(self.q_lens)
        meta = mla.get_metadata_window(n, ql, self.s_q, self.H, self.window, self.sinks)
        cache = torch.from_numpy(self.packed()).cuda() if fp8 else dev(self.kv)
        fn = mla.decode_fp8_window if fp8 else mla.decode_window
        return fn(dev(self.q_nope), dev(self.q_pe), cache, i32(self.table), n, ql, SCALE_192, self.window, self.sinks,
                  meta, status=status, **kw)

    def check(self, fp8=False):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = self.run(fp8, status)
        assert int(status.item()) == 0
        compare(out.float().cpu().double().numpy(), lse.cpu().double().numpy(), *self.reference(fp8),
                what=f"window {self.window} sinks {self.sinks} fp8={fp8}")


CASES = [
    # lens, s_q, H, window, sinks, q_lens
    ([1, 63, 64, 65, 0, 130], 1, 16, 64, 0, None),           # nothing hidden up to one key hidden
    ([1000], 1, 16, 128, 4, None),
    ([127, 128, 129, 191, 192, 193, 255, 256, 257], 1, 32, 64, 1, None),
    ([300, 301, 302, 303], 1, 64, 100, 63, None),            # odd and even first rows
    ([300, 364, 429, 1001], 1, 128, 77, 64, None),           # a whole block of first keys
    ([500, 170, 169, 171], 1, 128, 65, 105, None),           # first keys end in the block the window starts in
    ([70, 90, 128, 100], 1, 16, 64, 3, None),                # first keys and window share block 0
    ([5000, 2500, 77], 1, 128, 2048, 300, None),             # pieces
    ([40000], 1, 128, 20000, 4, None),                       # one sequence over many partitions
    ([100000, 33], 1, 16, 64, 128, None),                    # few keys far out
    ([500, 3, 2, 700], 4, 128, 64, 5, None),                 # fewer keys than tokens
    ([900, 1030, 64, 500, 130], 4, 64, 96, 70, [4, 1, 2, 0, 3]),
    ([259, 260, 261], 3, 16, 256, 0, [3, 2, 1]),
    ([320, 2000], 2, 32, 1 << 30, 0, None),                  # a window wider than everything
    ([320, 2000], 2, 32, 64, 2**31 - 1, None),               # first keys that cover everything
    ([1500] * 130, 1, 128, 192, 4, None),                    # more sequences than partitions
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,s_q,H,window,sinks,q_lens", CASES)
def test_window_matches_oracle(lens, s_q, H, window, sinks, q_lens, fp8):
    Problem(lens, s_q, H, window, sinks, q_lens, seed=window % 1000 + sinks % 1000 + len(lens)).check(fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_every_first_row_and_every_tail(fp8):
    """All 64 offsets of a window's first row and of the last key, in one batch."""
    Problem([256 + k for k in range(64)], 1, 16, 128, 4, seed=3).check(fp8)
    Problem([512 + 7 * k for k in range(64)], 1, 16, 64 + 37, 66, seed=4).check(fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_random_windows(fp8):
    rng = np.random.default_rng(77)
    for k in range(12):
        B, s_q = int(rng.integers(1, 9)), int(rng.integers(1, 5))
        lens = [int(x) for x in rng.integers(0, rng.choice([100, 600, 3000]), size=B)]
        q_lens = [int(x) for x in rng.integers(0, s_q + 1, size=B)] if k % 2 else None
        if q_lens is not None and not any(min(a, b) for a, b in zip(lens, q_lens)):
            q_lens = None
        Problem(lens, s_q, int(rng.choice([16, 32, 64, 128])), int(rng.integers(64, 700)), int(rng.integers(0, 200)),
                q_lens, seed=100 + k).check(fp8)


def test_a_key_reaches_only_the_tokens_that_see_it():
    """The window's first key of token 0 is hidden from token 1: NaN there leaves token 1
    exact; so does a NaN in token 1's own key for token 0."""
    p = Problem([500], 2, 16, 100, 2, seed=5)
    out, lse = (x.clone() for x in p.run())
    for t, hit in ((499 - 100, 0), (499, 1)):
        q = Problem([500], 2, 16, 100, 2, seed=5)
        q.kv[q.table[0, t // 64], t % 64] = 0x7FC0
        o, l = q.run()
        assert torch.isnan(o[0, hit]).all() and torch.isnan(l[0, hit]).all()
        assert torch.equal(o[0, 1 - hit], out[0, 1 - hit]) and torch.equal(l[0, 1 - hit], lse[0, 1 - hit])


@pytest.mark.parametrize("units", [(60, 4, 16), (300, 3, 128), (500, 3, 128)])  # one pass of the scheduler, and several
@pytest.mark.parametrize("window,sinks", [(64, 0), (500, 70), (1 << 20, 0)])
def test_window_schedule_matches_oracle(window, sinks, units):
    rng = np.random.default_rng(9)
    B, s_q, H = units
    lens, q_lens = rng.integers(-1, 6000, size=B), rng.integers(-1, s_q + 2, size=B)
    meta = mla.get_metadata_window(i32(lens), i32(q_lens), s_q, H, window, sinks).cpu().numpy()
    keys = np.zeros(B * s_q, dtype=np.int64)  # 64 keys for each visible block
    ok = np.where((q_lens >= 0) & (q_lens <= s_q) & (lens >= 0), q_lens, 0)
    for b, i, p in S.new_tokens(lens, ok, s_q):
        t = S.window_keys(p, window, sinks)
        far = t[t > p - window]
        near = t[t <= p - window]
        # a block that first keys and window share is counted for each, unless all is visible
        whole = len(t) == p + 1
        keys[b * s_q + i] = 64 * (len(np.unique(t // 64)) if whole else len(np.unique(near // 64)) + len(np.unique(far // 64)))
    workers = min(mla.device_sm_count() // 2, 256)
    sc = O.schedule_ref(keys, 1, H, workers)
    Bt, P = B * s_q, sc["num_parts"]
    assert list(meta[1:14]) == [Bt, 1, H, P, sc["num_tiles"], sc["cap"], sc["total_slots"], workers,
                                O.SCHED_OVERHEAD_TILES, s_q, 1, window, sinks]
    assert np.array_equal(meta[16:528].reshape(256, 2)[:P], sc["part_start"])
    assert np.array_equal(meta[528:1040].reshape(256, 2)[:P], sc["part_end"])
    for i, key in enumerate(["nblk", "first_part", "num_splits", "split_prefix"]):
        assert np.array_equal(meta[1040 + i * Bt:1040 + (i + 1) * Bt], sc[key]), key


def test_window_errors():
    p = Problem([500, 300, 400, 200, 260], 2, 16, 100, 4, seed=6)
    good, good_lse = (x.clone() for x in p.run())
    # a block id out of range among the visible ones, an invalid count and lengths
    p.table[0, 499 // 64] = len(p.kv)
    p.q_lens, p.lens = [2, 3, 2, 2, 2], [500, 300, -3, 10**7, 260]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = p.run(status=status)
    assert int(status.item()) == mla.MLA_DEVICE_ERR_BLOCK_ID | mla.MLA_DEVICE_ERR_SEQLEN
    assert torch.isnan(out[:4]).all() and torch.isnan(lse[:4]).all()
    assert torch.equal(out[4], good[4]) and torch.equal(lse[4], good_lse[4])


def test_another_schedule_is_refused_on_the_device():
    p = Problem([500, 300], 2, 16, 100, 4, seed=7)
    n = i32(p.lens)
    args = dev(p.q_nope), dev(p.q_pe), dev(p.kv), i32(p.table), n, None, SCALE_192
    for meta in (mla.get_metadata_window(n, None, 2, 16, 101, 4), mla.get_metadata_window(n, None, 2, 16, 100, 5),
                 mla.get_metadata_tokens(n, None, 2, 16, True)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((2, 2, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        mla.decode_window(*args, 100, 4, meta, out=out, status=status)
        assert int(status.item()) & mla.MLA_DEVICE_ERR_METADATA and (out == 7).all()
    # and a windowed schedule by the plain decode
    status.zero_()
    mla.decode_tokens(*args, True, mla.get_metadata_window(n, None, 2, 16, 100, 4), out=out, status=status)
    assert int(status.item()) & mla.MLA_DEVICE_ERR_METADATA and (out == 7).all()
    # lengths that moved since the schedule was made, by a block for sequence 0 only
    meta = mla.get_metadata_window(n, None, 2, 16, 100, 4)
    n2 = i32([512 + 65, 300])
    p2 = Problem([512 + 65, 300], 2, 16, 100, 4, seed=7)
    ref = S.window_decode_ref(O.bf16_to_f64(p2.q_nope), O.bf16_to_f64(p2.q_pe), p2.rows_of(False), p2.lens, None,
                              SCALE_192, 100, 4)
    status.zero_()
    out, lse = mla.decode_window(dev(p2.q_nope), dev(p2.q_pe), dev(p2.kv), i32(p2.table), n2, None, SCALE_192, 100, 4,
                                 meta, status=status)
    got, got_lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    for b in range(2):
        for i in range(2):
            stale = np.isnan(got[b, i]).all()
            assert stale or np.abs(got[b, i] - ref[0][b, i]).max() <= 2e-2
            assert not (b == 1 and stale)
    assert (int(status.item()) & mla.MLA_DEVICE_ERR_METADATA != 0) == bool(np.isnan(got).any())


@pytest.mark.parametrize("fp8", [False, True])
def test_window_deterministic_and_on_another_stream(fp8):
    p = Problem([9000, 10, 777, 5000, 1, 2048], 4, 128, 1500, 100, [4, 1, 3, 2, 1, 4], seed=8)
    a, al = p.run(fp8)
    s = torch.cuda.Stream()
    n, ql = i32(p.lens), i32(p.q_lens)
    cache = torch.from_numpy(p.packed()).cuda() if fp8 else dev(p.kv)
    qn, qp, table = dev(p.q_nope), dev(p.q_pe), i32(p.table)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        meta = mla.get_metadata_window(n, ql, 4, 128, 1500, 100)
        fn = mla.decode_fp8_window if fp8 else mla.decode_window
        b, bl = fn(qn, qp, cache, table, n, ql, SCALE_192, 1500, 100, meta)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(al, bl)


def test_window_step_in_a_graph_follows_the_lengths():
    p = Problem([3000, 17, 700, 5000], 1, 128, 512, 64, seed=10)
    n, table, cache = i32(p.lens), i32(p.table), dev(np.where(O.bf16_to_f64(p.kv) == O.bf16_to_f64(p.kv), p.kv, 0))
    table.clamp_(max=0)  # entries that another length may reach: any block of the pool
    table.copy_(torch.where(i32(p.table) == NOWHERE, table, i32(p.table)))
    qn, qp = dev(p.q_nope), dev(p.q_pe)
    meta = mla.get_metadata_window(n, None, 1, 128, 512, 64)
    ws = torch.empty(mla.workspace_size(4, 1, 128), dtype=torch.uint8, device="cuda")
    out, lse = mla.decode_window(qn, qp, cache, table, n, None, SCALE_192, 512, 64, meta, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.get_metadata_window(n, None, 1, 128, 512, 64, metadata=meta)
        mla.decode_window(qn, qp, cache, table, n, None, SCALE_192, 512, 64, meta, workspace=ws, out=out, lse=lse)
    for lens in ([3000, 17, 700, 5000], [2999, 577, 70, 4000], [1, 0, 512, 576]):
        n.copy_(i32(lens))
        out.zero_()
        g.replay()
        want = mla.decode_window(qn, qp, cache, table, n, None, SCALE_192, 512, 64,
                                 mla.get_metadata_window(n, None, 1, 128, 512, 64))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_steps_together(fp8):
    """A prompt's rows appended, then three draft-verification steps of up to two tokens:
    rope_q -> absorb_q, append, windowed decode, absorb_out, against the same chain in
    float64 (from the rounded outputs of each stage, so each is held to its own bound)."""
    B, H, window, sinks, prompt = 3, 16, 128, 4, [150, 1, 64]
    rng = np.random.default_rng(12)
    rope = mla.rope_params(scaling="yarn", factor=40.0, amplitude=1.1)
    rot = dict(freq=np.array(rope.freq), half=False, amplitude=float(rope.amplitude))
    w = f32_to_bf16_bits(1 + 0.1 * rng.standard_normal(512).astype(np.float32))
    w_uk, w_uv = (f32_to_bf16_bits(0.05 * rng.standard_normal((H, 128, 512)).astype(np.float32)) for _ in range(2))
    table = np.arange(B * 5).reshape(B, 5)
    cache = torch.zeros(B * 5, 64, 656 if fp8 else 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    append, decode = (mla.append_kv_fp8, mla.decode_fp8_window) if fp8 else (mla.append_kv, mla.decode_window)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = np.array(prompt)
    append(dev(bits(rng, (B, 150, 576))), cache, i32(table), i32(n), rope=rope, norm_weight=dev(w), q_lens=i32(n),
           status=status)
    for q_lens in ([1, 2, 2], [2, 0, 1], None):
        n = n + (np.array(q_lens) if q_lens is not None else 2)
        kv_a, q = bits(rng, (B, 2, 576)), bits(rng, (B, 2, H, 192))
        nt, qt, tt = i32(n), i32(q_lens), i32(table)
        append(dev(kv_a), cache, tt, nt, rope=rope, norm_weight=dev(w), q_lens=qt, status=status)
        heads, q_pe = mla.rope_q(dev(q), nt, rope, q_lens=qt, status=status)
        q_nope = mla.absorb_q(heads, dev(w_uk))
        meta = mla.get_metadata_window(nt, qt, 2, H, window, sinks)
        out, lse = decode(q_nope, q_pe, cache, tt, nt, qt, SCALE_192, window, sinks, meta, status=status)
        y = mla.absorb_out(out, dev(w_uv))
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        f64 = lambda t: t.float().cpu().double().numpy()  # noqa: E731
        store = F.dequantize_cache(cache.cpu().numpy()) if fp8 else f64(cache)
        x = O.bf16_to_f64(kv_a)
        for (b, i, p), row in S.append_rows_ref(x, n, q_lens, weight=O.bf16_to_f64(w), **rot).items():
            got = store[table[b, p // 64], p % 64]
            # bf16 half a step; e4m3 half a step of the value or of the smallest code, keys bf16
            lim = 2.0 ** -8 * np.abs(row) + 2.0 ** -18 * np.abs(row).max()
            if fp8:
                lim[:512] = np.maximum(2.0 ** -4 * np.abs(row[:512]), 2.0 ** -10 * np.abs(row).max() / 448) * 1.001 + \
                    2.0 ** -18 * np.abs(row).max()
            assert np.all(np.abs(got - row) <= lim)
        ref, ref_lse = S.window_decode_ref(f64(q_nope), f64(q_pe), lambda b, t: store[table[b, t // 64], t % 64], n,
                                           q_lens, SCALE_192, window, sinks)
        compare(f64(out), lse.cpu().double().numpy(), ref, ref_lse, what="step")
        ref_y = O.absorb_out_ref(f64(out), O.bf16_to_f64(w_uv))
        assert np.all(np.abs(f64(y) - ref_y) <= 2.0 ** -8 * np.abs(ref_y) + 1e-4)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_nan_or_infinite_query_row_stays_alone(fp8):
    p = Problem([500, 300, 70], 2, 64, 100, 70, seed=14)
    good, good_lse = (x.clone() for x in p.run(fp8))
    p.q_nope[0, 1, 5, 17], p.q_pe[2, 0, 63, 3], p.q_nope[1, 0, 9, 0] = 0x7FC0, 0x7FFF, 0x7F80
    out, lse = p.run(fp8)
    hit = torch.zeros(3, 2, 64, dtype=torch.bool, device="cuda")
    hit[0, 1, 5] = hit[2, 0, 63] = hit[1, 0, 9] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1.0])
def test_softmax_scales(fp8, scale):
    """From equal weights (the mean of the visible rows) to one key taking nearly all."""
    p = Problem([700, 130], 1, 16, 200, 3, seed=15)
    meta = mla.get_metadata_window(i32(p.lens), None, 1, 16, 200, 3)
    cache = torch.from_numpy(p.packed()).cuda() if fp8 else dev(p.kv)
    fn = mla.decode_fp8_window if fp8 else mla.decode_window
    out, lse = fn(dev(p.q_nope), dev(p.q_pe), cache, i32(p.table), i32(p.lens), None, scale, 200, 3, meta)
    ref, ref_lse = S.window_decode_ref(O.bf16_to_f64(p.q_nope), O.bf16_to_f64(p.q_pe), p.rows_of(fp8), p.lens, None,
                                       scale, 200, 3)
    compare(out.float().cpu().double().numpy(), lse.cpu().double().numpy(), ref, ref_lse, what=f"scale {scale}")


def test_fp8_rows_of_very_different_scales():
    """Rows 2^-60 to 2^6 of the others' size, rows of zeros, and zero queries: each row's scale
    rides with its weight.  Weights are held to 2^-8 or 2^-14 of the largest s 2^x, so each
    output is held to 2^-7 sum_t w_t |c_t| / sum_t w_t and what 1e-3 of the largest row adds."""
    p = Problem([600, 90], 1, 16, 300, 64, seed=16)
    rng = np.random.default_rng(17)
    exp = rng.choice([-60, -20, -6, 0, 0, 0, 3, 6], size=p.kv.shape[:2])
    values = O.bf16_to_f64(p.kv) * np.exp2(exp)[..., None]
    values[rng.random(p.kv.shape[:2]) < 0.1] = 0
    p.kv = np.where(np.isnan(values), p.kv, f32_to_bf16_bits(values.astype(np.float32)))
    p.q_nope[0, 0, 3], p.q_pe[0, 0, 3] = 0, 0
    out, lse = p.run(True)
    got, got_lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    ref, ref_lse = p.reference(True)
    rows = p.rows_of(True)
    for b, i, pos in S.new_tokens(p.lens, None, 1):
        r = rows(b, S.window_keys(pos, 300, 64))
        q = np.concatenate([O.bf16_to_f64(p.q_nope[b, i]), O.bf16_to_f64(p.q_pe[b, i])], -1)
        w = np.exp(SCALE_192 * (q @ r.T) - ref_lse[b, i][:, None])
        contrib = w[:, :, None] * np.abs(r[None, :, :512])
        lim = 2.0 ** -7 * contrib.sum(1) + 1e-3 * contrib.max((1, 2))[:, None] + 2.0 ** -8 * np.abs(ref[b, i])
        assert np.all(np.abs(got[b, i] - ref[b, i]) <= lim)
    assert np.abs(got_lse - ref_lse).max() <= 1e-3


@pytest.mark.parametrize("fp8", [False, True])
def test_window_wait_timeout_sets_status_and_returns(fp8):
    """The MMA warp waits on a barrier nothing completes (a test hook), bounded by 1 ms; every
    role stops at its next bounded wait, the pair drains and returns, and the next call is
    exact."""
    p = Problem([3000, 700, 5000], 2, 128, 1024, 100, seed=18)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        mla.set_wait_timeout_ns(1_000_000)
        mla.set_stall_injection(True)
        p.run(fp8, status)
        torch.cuda.synchronize()
    finally:
        mla.set_stall_injection(False)
        mla.set_wait_timeout_ns(0)
    assert int(status.item()) & mla.MLA_DEVICE_ERR_TIMEOUT
    p.check(fp8)


def test_window_with_the_callers_buffers_and_stream_argument():
    """Every tensor given, on a stream given; and nothing given but the stream."""
    p = Problem([900, 64, 300], 2, 32, 128, 4, [2, 1, 2], seed=19)
    want, want_lse = p.run()
    n, ql, table, cache = i32(p.lens), i32(p.q_lens), i32(p.table), dev(p.kv)
    qn, qp = dev(p.q_nope), dev(p.q_pe)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    meta = torch.empty(mla.metadata_size(6, 1, 32) // 4, dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.workspace_size(6, 1, 32), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    s.wait_stream(torch.cuda.current_stream())
    mla.get_metadata_window(n, ql, 2, 32, 128, 4, metadata=meta, stream=s)
    got = mla.decode_window(qn, qp, cache, table, n, ql, SCALE_192, 128, 4, meta, workspace=ws, out=out, lse=lse, stream=s)
    assert got[0] is out and got[1] is lse
    m2 = mla.get_metadata_window(n, ql, 2, 32, 128, 4, stream=s)
    out2, lse2 = mla.decode_window(qn, qp, cache, table, n, ql, SCALE_192, 128, 4, m2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.equal(out2, want) and torch.equal(lse2, want_lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[9000, 7000], [900 + 37 * i for i in range(100)]], ids=["wide", "by_partition"])
def test_split_sequences_of_another_schedule_are_left(lens, fp8):
    """Sequences in several pieces: the merge must not touch them either."""
    p = Problem(lens, 1, 128, 8000, 4, seed=31)
    n = i32(p.lens)
    kv = torch.from_numpy(p.packed()).cuda() if fp8 else dev(p.kv)
    args = dev(p.q_nope), dev(p.q_pe), kv, i32(p.table), n, None, SCALE_192
    call = mla.decode_fp8_window if fp8 else mla.decode_window
    B = len(lens)
    splits = mla.get_metadata_window(n, None, 1, 128, 8000, 4).cpu().numpy()[16 + 4 * 256 + 2 * B:][:B]
    assert splits.max() > 1
    for meta in (mla.get_metadata_window(n, None, 1, 128, 8001, 4), mla.get_metadata_window(n, None, 1, 128, 8000, 5)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((B, 1, 128, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, 1, 128), 7.0, device="cuda")
        call(*args, 8000, 4, meta, out=out, lse=lse, status=status)
        assert int(status.item()) == mla.MLA_DEVICE_ERR_METADATA
        assert (out == 7).all() and (lse == 7).all()
