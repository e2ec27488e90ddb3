"""Cases of the serving step's operators around the paged latent cache: rotary positions of the queries, appending new
tokens' rows to the bf16 or FP8 cache, and decode attention with a sliding window and first tokens that stay visible.

Every sequence b has n_b cached tokens, its q_b <= s_q new ones counted; new token i has position n_b - q_b + i.  A
sequence's lengths are drawn from the case's range with the other inputs; work() counts their expectation.
"""
import math

import numpy as np
import torch

own = False

BLOCK, LATENT, ROPE, NOPE, ROW, ROW8 = 64, 512, 64, 128, 576, 656
SCALE = 1.0 / math.sqrt(192.0)


def listed():
    serving = dict(B=256, s_q=1, H=128, ragged=False, n_lo=1812, n_hi=2790)
    return [
        # queries of one decode step of the serving mix: 256 sequences, all 128 heads
        dict(name="rope_q_decode_b256", op="rope_q", layout="interleaved", scaling="yarn", **serving),
        # one sequence, one token, one GPU's share of 16 heads: latency
        dict(name="rope_q_one_token", op="rope_q", B=1, s_q=1, H=16, ragged=False, n_lo=130, n_hi=130, layout="half", scaling="none"),
        # queries of an 8K prompt chunk far into a long context
        dict(name="rope_q_prompt_8k", op="rope_q", B=1, s_q=8192, H=128, ragged=False, n_lo=65536, n_hi=131072, layout="half", scaling="linear"),
        # new rows of one decode step of the serving mix
        dict(name="append_decode_b256", op="append", layout="interleaved", scaling="yarn", norm=True, **serving),
        # the rows of a whole 64K prompt
        dict(name="append_prompt_64k", op="append", B=1, s_q=65536, H=1, ragged=False, n_lo=65536, n_hi=65536, layout="interleaved", scaling="yarn", norm=True),
        # draft verification, 1 to 4 new tokens a sequence, FP8 cache
        dict(name="append_fp8_mtp_b128", op="append_fp8", B=128, s_q=4, H=1, ragged=True, n_lo=1024, n_hi=8192, layout="half", scaling="none", norm=True),
        # prompt chunks of odd and unequal lengths, FP8 cache
        dict(name="append_fp8_prompt_b4", op="append_fp8", B=4, s_q=8191, H=1, ragged=True, n_lo=8191, n_hi=32768, layout="interleaved", scaling="yarn", norm=True),
        # the serving mix with a window of 1024
        dict(name="window_serving_b256", op="window", window=1024, sinks=4, **serving),
        # one short sequence, one token, 16 heads: latency
        dict(name="window_one_token", op="window", B=1, s_q=1, H=16, ragged=False, n_lo=1000, n_hi=1000, window=128, sinks=4),
        # draft verification under a short window, sinks over more than one block
        dict(name="window_mtp_b128", op="window", B=128, s_q=4, H=128, ragged=True, n_lo=1024, n_hi=8192, window=512, sinks=100),
        # few long sequences over the FP8 cache
        dict(name="window_fp8_long_b4", op="window_fp8", B=4, s_q=1, H=128, ragged=False, n_lo=8192, n_hi=65536, window=4096, sinks=64),
        # many sequences, a wide window, FP8 cache
        dict(name="window_fp8_b192", op="window_fp8", B=192, s_q=1, H=128, ragged=False, n_lo=4500, n_hi=8192, window=4096, sinks=4),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["rope_q", "append", "append_fp8", "window", "window_fp8"])
    c = dict(op=op)
    if op.startswith("window"):
        c["H"] = rng.choice([16, 32, 64, 128])
        c["s_q"] = rng.choice([1, 1, 1, 2, 3, 4])
        c["window"] = spread(64, 4096)
        c["sinks"] = rng.choice([0, rng.randint(1, 16), rng.randint(1, 300)])
        c["B"] = spread(1, max(1, min(256, 192 * 4096 // (c["s_q"] * (c["window"] + c["sinks"])))))
        c["n_lo"] = spread(1, 65536)
    else:
        rows = 8192 * 128 if op == "rope_q" else 65536
        c["H"] = rng.choice([16, 32, 64, 128, rng.randint(1, 128)]) if op == "rope_q" else 1
        c["s_q"] = rng.choice([rng.randint(1, 4), spread(1, 8192)])
        c["B"] = spread(1, max(1, min(512, rows // (c["s_q"] * c["H"]))))
        c["n_lo"] = spread(c["s_q"], 131072)
        c["layout"] = rng.choice(["interleaved", "half"])
        c["scaling"] = rng.choice(["none", "linear", "yarn"])
        if op != "rope_q":
            c["norm"] = rng.random() < 0.75
    c["n_hi"] = c["n_lo"] + rng.randint(0, c["n_lo"])
    c["ragged"] = rng.random() < 0.5
    return c


def _rope_spec(case):
    """The arguments of the rotation that the model's configuration fixes."""
    spec = dict(base=10000.0, layout=case["layout"], scaling=case["scaling"])
    if case["scaling"] == "linear":
        spec.update(factor=8.0)
    elif case["scaling"] == "yarn":
        spec.update(factor=40.0, original_len=4096, beta_fast=32.0, beta_slow=1.0, amplitude=1.1)
    return spec


def _frequencies(spec):
    """Radians per position of the 32 pairs, from the definition, on the host."""
    freq = [spec["base"] ** (-2.0 * i / ROPE) for i in range(ROPE // 2)]
    s = spec.get("factor", 1.0)
    if spec["scaling"] == "linear":
        return [f / s for f in freq]
    if spec["scaling"] == "yarn":
        def dim(turns):
            return ROPE * math.log(spec["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(spec["base"]))

        lo, hi = max(math.floor(dim(spec["beta_fast"])), 0), min(math.ceil(dim(spec["beta_slow"])), ROPE - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(ROPE // 2)]
        return [f * (1 - r) + f / s * r for f, r in zip(freq, ramp)]
    return freq


def _first_window_key(case, n, q):
    """The first key in the window of a sequence's first new token."""
    return (n - q + 1 - case["window"]).clamp(min=0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, s_q, H, op = case["B"], case["s_q"], case["H"], case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def whole(lo, hi, shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)

    n = whole(case["n_lo"], case["n_hi"], (B,))
    q_lens = torch.minimum(whole(1, s_q, (B,)), n) if case["ragged"] else None
    st = dict(case=case, n=n, q_lens=q_lens)
    q = q_lens if q_lens is not None else torch.full_like(n, s_q)
    if not op.startswith("window"):
        st["rope"] = _rope_spec(case)
        st["freq"] = torch.tensor(_frequencies(st["rope"]), dtype=torch.float64, device="cuda")
    if op == "rope_q":
        st["q"] = normal(B, s_q, H, NOPE + ROPE)
        return st
    # The paged pool: blocks that hold appended or visible tokens, in a random order.  Blocks of tokens that are out of
    # everyone's sight were given back: their table entries point at the spare block.
    max_blocks = (case["n_hi"] + BLOCK - 1) // BLOCK + 1
    first = torch.arange(max_blocks, device="cuda")[None, :] * BLOCK
    last = n[:, None]
    if op.startswith("window"):
        lo = _first_window_key(case, n, q)[:, None]
        used = (first < last) & ((first + BLOCK > lo) | (first < case["sinks"]))
    else:
        used = (first < last) & (first + BLOCK > (n - q).clamp(min=0)[:, None])
    rank = torch.cumsum(used.reshape(-1).to(torch.int64), 0).reshape(used.shape) - 1
    if op.startswith("window"):
        blocks = int(rank[-1, -1]) + 2
    else:  # as many for each sequence as its new tokens can reach, and the spare one
        blocks = B * min(max_blocks, (s_q + BLOCK - 2) // BLOCK + 1) + 1
    order = torch.randperm(blocks - 1, generator=g, device="cuda").to(torch.int32)
    st["table"] = torch.where(used, order[rank.clamp(min=0)], torch.full_like(order[:1], blocks - 1)).contiguous()
    if op.startswith("append"):
        # the fused down-projection's output: 1536 columns of the query side, then the 576 of this one
        st["kv_a"] = normal(B, s_q, 1536 + ROW)[..., 1536:]
        st["norm"] = (1 + 0.1 * torch.randn(LATENT, generator=g, device="cuda")).bfloat16() if case["norm"] else None
        if op == "append_fp8":
            st["cache"] = torch.zeros(blocks, BLOCK, ROW8, dtype=torch.uint8, device="cuda")
        else:
            st["cache"] = torch.zeros(blocks, BLOCK, ROW, dtype=torch.bfloat16, device="cuda")
        return st
    st["q_nope"], st["q_pe"] = normal(B, s_q, H, LATENT), normal(B, s_q, H, ROPE)
    if op == "window_fp8":
        cache = torch.zeros(blocks, BLOCK, ROW8, dtype=torch.uint8, device="cuda")
        for k in range(0, blocks, 4096):
            part = normal(min(4096, blocks - k), BLOCK, ROW).float()
            scale = part.abs().amax(-1, keepdim=True) / 448
            cache[k : k + 4096, :, :LATENT] = (part[..., :LATENT] / scale).to(torch.float8_e4m3fn).view(torch.uint8)
            cache[k : k + 4096, :, LATENT : LATENT + 2 * ROPE] = (part[..., LATENT:] / scale).bfloat16().view(torch.uint8)
            cache[k : k + 4096, :, 640:644] = scale.view(torch.uint8)
        st["cache"] = cache
    else:
        st["cache"] = normal(blocks, BLOCK, ROW)
    return st


def _positions(st):
    """Positions [B, s_q] of the new tokens and which of them are real."""
    s_q = st["case"]["s_q"]
    q = st["q_lens"] if st["q_lens"] is not None else torch.full_like(st["n"], s_q)
    i = torch.arange(s_q, device="cuda")
    pos = st["n"][:, None].long() - q[:, None] + i
    return pos, (i < q[:, None]) & (pos >= 0)


def _rotate(x, pos, st):
    """x [..., 64] in 32 bits, pos broadcast against its leading sizes; angles in 64 bits."""
    angle = pos[..., None].double() * st["freq"]
    amp = st["rope"].get("amplitude", 1.0)
    cos, sin = (torch.cos(angle) * amp).float(), (torch.sin(angle) * amp).float()
    if st["rope"]["layout"] == "half":
        a, b = x[..., : ROPE // 2], x[..., ROPE // 2 :]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _plain_rope_q(st):
    pos, real = _positions(st)
    keep = real[:, :, None, None]
    pe = _rotate(st["q"][..., NOPE:].float(), pos[:, :, None], st)
    zero = torch.zeros((), device="cuda")
    return torch.where(keep, st["q"][..., :NOPE], zero.bfloat16()), torch.where(keep, pe, zero).bfloat16()


def _plain_append(st):
    pos, real = _positions(st)
    x = st["kv_a"].float()
    c, k = x[..., :LATENT], _rotate(x[..., LATENT:], pos, st)
    if st["norm"] is not None:
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6) * st["norm"].float()
    cache = st["cache"]
    place = torch.where(real, pos, torch.zeros_like(pos))
    block = torch.gather(st["table"].long(), 1, place // BLOCK)
    # tokens that are padding write zeros into the spare block, which holds zeros
    slot = torch.where(real, block * BLOCK + place % BLOCK, (cache.shape[0] - 1) * BLOCK).reshape(-1)
    keep = real[..., None]
    if st["case"]["op"] == "append":
        row = torch.where(keep, torch.cat([c, k], -1), torch.zeros((), device="cuda")).bfloat16()
        cache.view(-1, ROW)[slot] = row.reshape(-1, ROW)
        return cache
    scale = torch.maximum(c.abs().amax(-1, keepdim=True), k.abs().amax(-1, keepdim=True)) / 448
    inv = torch.where(scale > 0, scale, torch.ones_like(scale))
    row = torch.zeros(*pos.shape, ROW8, dtype=torch.uint8, device="cuda")
    row[..., :LATENT] = (c / inv).to(torch.float8_e4m3fn).view(torch.uint8)
    row[..., LATENT:640] = (k / inv).bfloat16().view(torch.uint8)
    row[..., 640:644] = scale.view(torch.uint8)
    row = torch.where(keep, row, torch.zeros_like(row))
    cache.view(-1, ROW8)[slot] = row.reshape(-1, ROW8)
    return cache


def _values8(cache):
    """What a packed cache holds: the codes' values, the scaled rotary keys and the rows' scales."""
    return [cache[..., :LATENT].view(torch.float8_e4m3fn), cache[..., LATENT:640].view(torch.bfloat16), cache[..., 640:644].view(torch.float32)]


def _plain_window(st):
    case = st["case"]
    W, S, H = case["window"], case["sinks"], case["H"]
    pos, real = _positions(st)
    n = torch.where(real, pos + 1, torch.zeros_like(pos))  # visible prefix of each token
    t = torch.cat([torch.arange(S, device="cuda").expand(*n.shape, S), n[..., None] - W + torch.arange(W, device="cuda")], -1)
    lo = (n - W).clamp(min=0)[..., None]
    seen = (t >= 0) & torch.cat([(t[..., :S] < lo) & (t[..., :S] < n[..., None]), t[..., S:] < n[..., None]], -1)
    t = torch.where(seen, t, torch.zeros_like(t))
    block = torch.gather(st["table"].long()[:, None, :].expand(-1, n.shape[1], -1), 2, t // BLOCK)
    slot = block * BLOCK + t % BLOCK
    if case["op"] == "window":
        rows = st["cache"].view(-1, ROW)[slot].float()
    else:
        packed = st["cache"].view(-1, ROW8)[slot]
        code = packed[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float()
        pe = packed[..., LATENT:640].contiguous().view(torch.bfloat16).float()
        rows = torch.cat([code, pe], -1) * packed[..., 640:644].contiguous().view(torch.float32)
    rows = rows.flatten(0, 1)
    q = torch.cat([st["q_nope"], st["q_pe"]], -1).float().flatten(0, 1)
    s = torch.bmm(q, rows.transpose(1, 2)) * SCALE
    s = torch.where(seen.flatten(0, 1)[:, None, :], s, torch.full((), -math.inf, device="cuda"))
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    out = torch.bmm(e, rows[..., :LATENT]) / torch.where(z > 0, z, torch.ones_like(z))
    shape = (*n.shape, H)
    return out.bfloat16().view(*shape, LATENT), (m + torch.log(z)).view(shape)


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        import deepseek_mla_decode_b200 as mla

        if op == "rope_q":
            return mla.rope_q(st["q"], st["n"], mla.rope_params(**st["rope"]), q_lens=st["q_lens"])
        if op == "append":
            return mla.append_kv(st["kv_a"], st["cache"], st["table"], st["n"], rope=mla.rope_params(**st["rope"]), norm_weight=st["norm"], eps=1e-6, q_lens=st["q_lens"])
        if op == "append_fp8":
            return _values8(mla.append_kv_fp8(st["kv_a"], st["cache"], st["table"], st["n"], rope=mla.rope_params(**st["rope"]), norm_weight=st["norm"], eps=1e-6, q_lens=st["q_lens"]))
        W, S = case["window"], case["sinks"]
        meta = mla.get_metadata_window(st["n"], st["q_lens"], case["s_q"], case["H"], W, S)
        decode = mla.decode_window if op == "window" else mla.decode_fp8_window
        return decode(st["q_nope"], st["q_pe"], st["cache"], st["table"], st["n"], st["q_lens"], SCALE, W, S, meta)
    if op == "rope_q":
        return _plain_rope_q(st)
    if op == "append":
        return _plain_append(st)
    if op == "append_fp8":
        return _values8(_plain_append(st))
    return _plain_window(st)


def _mean(lo, hi, f):
    """The mean of f over the whole numbers lo .. hi, from at most 4096 of them."""
    n = hi - lo + 1
    at = range(lo, hi + 1) if n <= 4096 else [lo + (2 * k + 1) * n // 8192 for k in range(4096)]
    return sum(f(x) for x in at) / len(at)


def work(case):
    B, s_q, H, op = case["B"], case["s_q"], case["H"], case["op"]
    counts = list(range(1, s_q + 1)) if case["ragged"] else [s_q]
    mean_n = (case["n_lo"] + case["n_hi"]) / 2
    tokens = B * sum(min(c, mean_n) for c in counts) / len(counts)
    if op == "rope_q":
        # heads of real tokens read; every head of both outputs written
        return dict(bytes=384.0 * H * (tokens + B * s_q), flops=6.0 * (ROPE // 2) * H * tokens)
    if op == "append":
        return dict(bytes=2.0 * 2 * ROW * tokens, flops=(4.0 * LATENT + 6 * (ROPE // 2)) * tokens)
    if op == "append_fp8":
        return dict(bytes=(2.0 * ROW + ROW8) * tokens, flops=(6.0 * LATENT + 8 * (ROPE // 2)) * tokens)
    W, S = case["window"], case["sinks"]
    seen = _mean(case["n_lo"], case["n_hi"], lambda n: min(n, W + min(S, max(0, n - W))))  # keys of one token
    q = tokens / B
    rows = B * _mean(case["n_lo"], case["n_hi"], lambda n: min(n, W + q - 1 + min(S, max(0, n - W - q + 1))))  # distinct keys
    width = 2.0 * ROW if op == "window" else 644.0
    bytes_ = rows * width + tokens * H * 2.0 * ROW + B * s_q * H * (2.0 * LATENT + 4)
    return dict(bytes=bytes_, flops=2.0 * (ROW + LATENT) * H * tokens * seen)


def exact(case, seed):
    """The definitions in 64 bits, token by token or sequence by sequence."""
    st = prepare(case, seed)
    B, s_q, H, op = case["B"], case["s_q"], case["H"], case["op"]
    n = st["n"].tolist()
    q = st["q_lens"].tolist() if st["q_lens"] is not None else [s_q] * B
    if not op.startswith("window"):
        spec = st["rope"]
        i = np.arange(ROPE // 2, dtype=np.float64)
        theta = np.power(spec["base"], -i / (ROPE // 2))
        if spec["scaling"] == "linear":
            theta = theta / spec["factor"]
        if spec["scaling"] == "yarn":
            edge = [(ROPE / 2) * np.log(spec["original_len"] / (2 * np.pi * b)) / np.log(spec["base"]) for b in (spec["beta_fast"], spec["beta_slow"])]
            lo, hi = max(0.0, np.floor(edge[0])), min(ROPE - 1.0, np.ceil(edge[1]))
            theta = theta * (1 - np.clip((i - lo) / (hi - lo), 0, 1) * (1 - 1 / spec["factor"]))
        # a rotation is a product with a unit complex number
        first, second = (slice(0, 32), slice(32, 64)) if spec["layout"] == "half" else (slice(0, None, 2), slice(1, None, 2))

        def turned(x, position):  # x [tokens, ..., 64], position [tokens]
            w = torch.polar(torch.full((1,), float(spec.get("amplitude", 1.0)), dtype=torch.float64, device="cuda"),
                            torch.outer(position.double(), torch.from_numpy(theta).cuda()))
            z = torch.complex(x[..., first], x[..., second]) * w.view(len(position), *([1] * (x.dim() - 2)), 32)
            y = torch.empty_like(x)
            y[..., first], y[..., second] = z.real, z.imag
            return y

    if op == "rope_q":
        if B * s_q * H > 300000:
            pe = torch.zeros(B, s_q, H, ROPE, dtype=torch.float64, device="cuda")
        else:
            pe = torch.zeros(B, s_q, H, ROPE, dtype=torch.float64)
        heads = torch.zeros(B, s_q, H, NOPE, dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            skip = max(0, q[b] - n[b])
            position = torch.arange(n[b] - q[b] + skip, n[b], device="cuda")
            heads[b, skip : q[b]] = st["q"][b, skip : q[b], :, :NOPE]
            pe[b, skip : q[b]] = turned(st["q"][b, skip : q[b], :, NOPE:].double(), position).to(pe.device)
        return heads.double(), pe
    if op.startswith("append"):
        wide = op == "append"
        cache = torch.zeros(*st["cache"].shape[:2], ROW, dtype=torch.float64, device="cuda")
        for b in range(B):
            skip = max(0, q[b] - n[b])
            position = torch.arange(n[b] - q[b] + skip, n[b], device="cuda")
            x = st["kv_a"][b, skip : q[b]].double()
            c = x[:, :LATENT]
            if st["norm"] is not None:
                c = c * torch.rsqrt(c.pow(2).sum(-1, keepdim=True) / LATENT + 1e-6) * st["norm"].double()
            cache[st["table"][b][position // BLOCK].long(), position % BLOCK] = torch.cat([c, turned(x[:, LATENT:], position)], -1)
        if wide:
            return cache
        scale = cache.abs().amax(-1, keepdim=True) / 448
        units = cache / torch.where(scale > 0, scale, torch.ones_like(scale))
        return [units[..., :LATENT], units[..., LATENT:], scale]
    if op == "window":
        store = st["cache"].double().view(-1, ROW)
    else:
        p = st["cache"].view(-1, ROW8)
        store = torch.empty(p.shape[0], ROW, dtype=torch.float32, device="cuda")
        for k in range(0, p.shape[0], 1 << 18):
            part = p[k : k + (1 << 18)]
            store[k : k + len(part), :LATENT] = part[:, :LATENT].contiguous().view(torch.float8_e4m3fn).float()
            store[k : k + len(part), LATENT:] = part[:, LATENT:640].contiguous().view(torch.bfloat16).float()
        row_scale = p[:, 640:644].contiguous().view(torch.float32).double()
    out = torch.zeros(B, s_q, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, s_q, H), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        for i in range(q[b]):
            p_i = n[b] - q[b] + i
            if p_i < 0:
                continue
            t = torch.arange(p_i + 1, device="cuda")
            t = t[(t > p_i - case["window"]) | (t < case["sinks"])]
            at = st["table"][b][t // BLOCK].long() * BLOCK + t % BLOCK
            keys = store[at].double()
            if op == "window_fp8":
                keys = keys * row_scale[at]
            s = SCALE * (st["q_nope"][b, i].double() @ keys[:, :LATENT].T + st["q_pe"][b, i].double() @ keys[:, LATENT:].T)
            lse[b, i] = torch.logsumexp(s, -1)
            out[b, i] = torch.softmax(s, -1) @ keys[:, :LATENT]
    return out, lse
