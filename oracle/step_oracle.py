"""Plain float64 CPU oracle of what surrounds the decode attention in a serving step:
rotary positions, the rows appended to the paged latent cache, and decode attention with a
sliding window and first tokens that stay visible.

TEST INFRASTRUCTURE ONLY (see mla_oracle.py): nothing on the product path imports it, and
it shares no code with the CUDA library.

Definitions.  Sequence b has n_b cached tokens, the q_b <= s_q new ones counted; new token
i (i < q_b) has position p = n_b - q_b + i, and has none when that is negative.

* rotation of the 64-wide rotary part: pair i, (x[2i], x[2i+1]) or (x[i], x[i+32]), is
  multiplied as a complex number by amplitude * exp(1j * p * freq[i]);
* frequencies: base^(-2i/64), divided by a factor, or mixed by YaRN's ramp (Peng et al.
  2023, "NTK-by-parts");
* appended row: [c * w / sqrt(mean(c^2) + eps) | rotated k];
* window: token at position p sees t <= p with t > p - window or t < sinks.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK_SIZE, D_LATENT, D_ROPE, D_QK = 64, 512, 64, 576


def rope_freq_ref(base, scaling="none", factor=1.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0):
    out = []
    for i in range(D_ROPE // 2):
        f = base ** (-2.0 * i / D_ROPE)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            # the pair index at which a wave turns r times within the original length
            def d(r):
                return D_ROPE / 2 * math.log(original_len / (r * 2 * math.pi), base)

            lo, hi = max(0, math.floor(d(beta_fast))), min(D_ROPE - 1, math.ceil(d(beta_slow)))
            g = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = (1 - g) * f + g * f / factor
        out.append(f)
    return np.array(out)


def _members(half):
    return (slice(0, 32), slice(32, 64)) if half else (slice(0, 64, 2), slice(1, 64, 2))


def rotate_ref(x, pos, freq, half, amplitude=1.0):
    """x [..., 64] float64 rotated at position pos (scalar)."""
    a, b = _members(half)
    z = (x[..., a] + 1j * x[..., b]) * (amplitude * np.exp(1j * np.float64(pos) * freq))
    y = np.empty_like(x)
    y[..., a], y[..., b] = z.real, z.imag
    return y


def new_tokens(cache_seqlens, q_lens, s_q):
    """(b, i, p) of every new token that has a place."""
    for b, n in enumerate(cache_seqlens):
        q = s_q if q_lens is None else int(q_lens[b])
        for i in range(q):
            if int(n) - q + i >= 0:
                yield b, i, int(n) - q + i


def rope_q_ref(q, cache_seqlens, q_lens, freq, half, amplitude=1.0):
    """q [B, s_q, H, 192] -> (q_heads, q_pe); tokens without a place give zeros."""
    heads, pe = np.zeros(q.shape[:3] + (128,)), np.zeros(q.shape[:3] + (64,))
    for b, i, p in new_tokens(cache_seqlens, q_lens, q.shape[1]):
        heads[b, i] = q[b, i, :, :128]
        pe[b, i] = rotate_ref(q[b, i, :, 128:], p, freq, half, amplitude)
    return heads, pe


def append_rows_ref(kv_a, cache_seqlens, q_lens, freq=None, half=False, amplitude=1.0, weight=None, eps=1e-6):
    """{(b, i, p): row [576]} of the new tokens, unrounded."""
    rows = {}
    for b, i, p in new_tokens(cache_seqlens, q_lens, kv_a.shape[1]):
        c, k = kv_a[b, i, :D_LATENT], kv_a[b, i, D_LATENT:]
        if weight is not None:
            c = c * weight / np.sqrt(np.mean(c * c) + eps)
        if freq is not None:
            k = rotate_ref(k, p, freq, half, amplitude)
        rows[b, i, p] = np.concatenate([c, k])
    return rows


def window_keys(p, window, sinks):
    """Positions that the token at position p sees."""
    t = np.arange(p + 1)
    return t[(t > p - window) | (t < sinks)]


def window_decode_ref(q_nope, q_pe, rows_of, cache_seqlens, q_lens, scale, window, sinks):
    """rows_of(b, t) -> float64 cache rows [len(t), 576].  Returns out, lse (0 and -inf for
    tokens without a place)."""
    B, s_q, H, _ = q_nope.shape
    out, lse = np.zeros((B, s_q, H, D_LATENT)), np.full((B, s_q, H), -np.inf)
    for b, i, p in new_tokens(cache_seqlens, q_lens, s_q):
        rows = rows_of(b, window_keys(p, window, sinks))
        s = scale * (np.concatenate([q_nope[b, i], q_pe[b, i]], -1) @ rows.T)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(-1, keepdims=True)
        out[b, i] = (e @ rows[:, :D_LATENT]) / z
        lse[b, i] = (m + np.log(z))[:, 0]
    return out, lse
