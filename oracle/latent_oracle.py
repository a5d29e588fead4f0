"""CPU oracle of the dense latent attention (absorbed and expanded forms) and of the 4-bit
latent rows -- TEST INFRASTRUCTURE.

Only tests/ and __graft_entry__.smoke() may import or run this module; it shares no code with
the CUDA library.  Everything is float64.

Readings ('Latent attention (MLA)' row: 512-dim latent plus a 64-dim shared key slot):
  * dense: query t at position p attends to rows 0..p of its own sequence; p = -1 to nothing
    (o = 0, lse = -inf); score = scale * (q . row) over the 576 cached values, value = latent;
  * expanded: a head's key is the bf16 up-projection of the latent (128 values) followed by the
    row's 64 rope values, its value the bf16 up-projection (128 values); the library keeps both
    in fp16 instead, and bounds that use this form allow a step of bf16 a value (rounded=False
    leaves both in float64);
  * 4-bit rows: blocks of 16 latent values share the scale e4m3(min(amax / 6, 448)); codes are
    e2m1, nearest, ties to even, saturating; the rope key stays bf16.
"""

from __future__ import annotations

import numpy as np

from .indexer_oracle import bf16_round, e4m3_round

FP4_GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FP4_ROW_BYTES = 416


def attend(x, v):
    """Scores x [H, n] and values v [n, D] (or [H, n, D]): o [H, D], lse [H], and the mean
    magnitude sum_j w_j |v_j| [H, D] that error bounds need."""
    H = x.shape[0]
    D = v.shape[-1]
    if x.shape[1] == 0:
        return np.zeros((H, D)), np.full(H, -np.inf), np.zeros((H, D))
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - m)
    z = e.sum(axis=1, keepdims=True)
    w = e / z
    if v.ndim == 2:
        return w @ v, (m + np.log(z))[:, 0], w @ np.abs(v)
    return np.einsum("hn,hnd->hd", w, v), (m + np.log(z))[:, 0], np.einsum("hn,hnd->hd", w, np.abs(v))


def sequence_rows(t, q_seq_offsets, cache_offsets):
    b = int(np.searchsorted(np.asarray(q_seq_offsets), t, side="right") - 1)
    return int(cache_offsets[b]), int(cache_offsets[b + 1])


def latent_attention(q, kv, positions, q_seq_offsets, cache_offsets, scale, idx=None):
    """q [T, H, 576], kv [rows, 576]; dense, or over idx [T, k].  Returns o [T, H, 512],
    lse [T, H] and sum_j w_j |v_j| [T, H, 512]; rows of tokens in no sequence are NaN."""
    T, H, _ = q.shape
    o = np.full((T, H, 512), np.nan)
    lse = np.full((T, H), np.nan)
    mag = np.full((T, H, 512), np.nan)
    for t in range(int(q_seq_offsets[0]), int(q_seq_offsets[-1])):
        r0, r1 = sequence_rows(t, q_seq_offsets, cache_offsets)
        if idx is None:
            rows = kv[r0:r0 + int(positions[t]) + 1]
        else:
            sel = np.asarray(idx[t], np.int64)
            rows = kv[r0 + sel[(sel >= 0) & (sel < r1 - r0)]]
        o[t], lse[t], mag[t] = attend(scale * (q[t] @ rows.T), rows[:, :512])
    return o, lse, mag


def expand(kv, W_ukv, rounded=True):
    """Keys [rows, H, 192] and values [rows, H, 128] of latent rows, rounded to bf16 or not."""
    H = W_ukv.shape[0]
    up = np.einsum("sc,hdc->shd", kv[:, :512], W_ukv)
    if rounded:
        up = bf16_round(up)
    rope = np.broadcast_to(kv[:, None, 512:], (kv.shape[0], H, 64))
    return np.concatenate((up[:, :, :128], rope), axis=2), up[:, :, 128:]


def latent_attention_expanded(q, kv, W_ukv, positions, q_seq_offsets, cache_offsets, scale, rounded=True):
    """q [T, H, 192]; returns o [T, H, 128] and sum_j w_j |v_j|."""
    T, H, _ = q.shape
    k, v = expand(kv, W_ukv, rounded)
    o = np.full((T, H, 128), np.nan)
    mag = np.full((T, H, 128), np.nan)
    for t in range(int(q_seq_offsets[0]), int(q_seq_offsets[-1])):
        r0, _ = sequence_rows(t, q_seq_offsets, cache_offsets)
        s = slice(r0, r0 + int(positions[t]) + 1)
        x = scale * np.einsum("hd,nhd->hn", q[t], k[s])
        o[t], _, mag[t] = attend(x, v[s].transpose(1, 0, 2))
    return o, mag


def quantize_latent_fp4(x):
    """Rows [n, 576] (bf16 values): block scales [n, 32], codes [n, 512] (sign in bit 3) and the
    values they stand for [n, 576]."""
    n = x.shape[0]
    v = x[:, :512].reshape(n, 32, 16)
    s = e4m3_round(np.minimum(np.abs(v).max(axis=2) / 6.0, 448.0))
    codes = np.zeros(v.shape, np.int64)
    for i, j, k in np.ndindex(*v.shape):
        if s[i, j] == 0:
            continue
        d = np.abs(abs(v[i, j, k]) - FP4_GRID * s[i, j])       # exact in float64
        best = np.flatnonzero(d == d.min())
        c = int(best[0]) if best.size == 1 else int(best[best % 2 == 0][0])
        codes[i, j, k] = c | (8 if np.signbit(v[i, j, k]) else 0)
    val = FP4_GRID[codes & 7] * s[..., None] * np.where(codes & 8, -1.0, 1.0)
    return s, codes.reshape(n, 512), np.concatenate((val.reshape(n, 512), x[:, 512:]), axis=1)
