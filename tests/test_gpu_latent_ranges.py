"""Latent-cache operators where their number formats and work lists could give way: values far
outside fp16's range, rows that only some queries see, many short sequences, many heads, and the
expanded form against the definition without any rounding of keys and values.

Tolerances (U = 2^-8 and F = 2^-11, the unit roundoffs of bf16 and fp16; all bounds per value).
  * expanded: keys, values and weights are fp16 roundings (F each; queries are scaled by powers of
    two, which rounds nothing).  A key's roundings move a score by at most e_k = F scale
    sum_d |q_d k_d|; values and weights move the output by F mag each, mag = sum_j w_j |v_j|; out
    is rounded once (U |o|).  fp32 sums: e_s = 6 sqrt(192) 2^-24 scale |q| max|k| for a score and,
    for its scaling, shift and exponential, 4 * 2^-24 max|x| + 2^-20.  With e = e_k + e_s:
    |o - o_ref| <= 1.01 U |o_ref| + (2.1 F + 2 expm1(e)) (mag + |o_ref|) + 2^-19 max|v|, the last
    term for weights below 2^-21 of the largest, which fp16 holds to 2^-32 of it, 8,192 of them.
  * 4-bit: values are exact in fp16, weights fp16 roundings: the same with e_k = 0 and F once."""

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from _parity import f64
from test_gpu_latent import DEV, SCALE, U, Batch, _check, _quantized, _weights

pytestmark = pytest.mark.gpu

F = 2.0 ** -11


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dsa_lightning_indexer_03_b200 import build
    build.build()
    import dsa_lightning_indexer_03_b200 as d
    return d


@pytest.fixture(scope="module")
def ix(dsa):
    wts = W.make_weights(41, hidden_dim=128, q_latent_dim=64)
    return dsa.Indexer(*(t.to(DEV).contiguous() for t in (wts.W_q, wts.W_k, wts.W_w, wts.gamma, wts.beta)),
                       max_tokens=4096)


def _expanded(ix, b, w, scale=SCALE, **kw):
    return f64(ix.latent_attention_expanded(*b.dev("q", "kv"), w.to(DEV), *b.dev("pos", "qo", "co"), scale, **kw))


def _check_exact(o, b, w, scale=SCALE, tokens=None):
    """o against softmax attention over unrounded keys and values (heads one by one)."""
    q, kv, wd = f64(b.q), f64(b.kv), f64(w)
    pos, qo, co = b.pos.numpy(), b.qo.numpy(), b.co.numpy()
    for s in range(len(qo) - 1):
        t0, t1, r0, r1 = int(qo[s]), int(qo[s + 1]), int(co[s]), int(co[s + 1])
        ts = [t for t in range(t0, t1) if tokens is None or t in tokens]
        n = max([int(pos[t]) + 1 for t in ts], default=0)
        if not ts:
            continue
        c = kv[r0:r0 + n]
        for h in range(q.shape[1]):
            k = np.concatenate((c[:, :512] @ wd[h, :128].T, c[:, 512:]), axis=1)
            v = c[:, :512] @ wd[h, 128:].T
            x = scale * (q[ts, h] @ k.T)
            mask = np.arange(n)[None] > pos[ts, None]
            x[mask] = -np.inf
            live = pos[ts] >= 0
            m = np.where(live, x.max(1, initial=-np.inf), 0.0)
            wt = np.exp(x - m[:, None])
            wt[mask] = 0.0
            z = np.where(live, wt.sum(1), 1.0)[:, None]
            ref, mag = wt @ v / z, wt @ np.abs(v) / z
            ax = np.where(mask, 0.0, np.abs(np.where(mask, 0.0, x)))
            e = F * scale * np.where(mask, 0.0, np.abs(q[ts, h]) @ np.abs(k).T).max(1, initial=0.0)
            e += 6 * np.sqrt(192) * 2.0 ** -24 * scale * np.linalg.norm(q[ts, h], axis=1) * np.linalg.norm(k, axis=1).max(initial=0.0)
            e += 4 * 2.0 ** -24 * ax.max(1, initial=0.0) + 2.0 ** -20
            tol = 1.01 * U * np.abs(ref) + (2.1 * F + 2 * np.expm1(e)[:, None]) * (mag + np.abs(ref))
            tol += 2.0 ** -19 * np.abs(v).max(initial=0.0)
            err = np.abs(o[ts, h] - ref)
            assert np.all(err <= tol), (s, h, err.max(), (err / tol).max())


@pytest.mark.parametrize("lens,nq,H", [([1], [1], 1), ([129, 127, 1], [129, 127, 1], 3), ([700, 90], [100, 90], 2),
                                       ([1030], [3], 16), ([600], [600], 7),
                                       ([300, 290, 280], [300, 290, 280], 450)])   # the last: whole items, by a counter
def test_expanded_against_unrounded_keys_and_values(dsa, ix, lens, nq, H):
    b, w = Batch(60 + H, lens, nq, H, dim=192), _weights(H + 1, H)
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_exact(o, b, w)


@pytest.mark.parametrize("q_exp,kv_exp", [(-30, 30), (30, -30), (-100, 100), (60, -60)])
def test_expanded_values_outside_the_range_of_fp16(dsa, ix, q_exp, kv_exp):
    # scores stay ordinary, queries and latents are far outside fp16's range
    b, w = Batch(70, [300], [150], 3, dim=192), _weights(20, 3)
    b.q = (b.q.float() * 2.0 ** q_exp).to(torch.bfloat16)
    b.kv = (b.kv.float() * 2.0 ** kv_exp).to(torch.bfloat16)
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK and np.all(np.isfinite(o))
    _check_exact(o, b, w)


def test_expanded_tiles_of_very_different_magnitude(dsa, ix):
    # 128-token tiles of a head carry scales of their own: the values of one are 2^25 times those
    # of the next, and every query sees both
    b, w = Batch(71, [384], [384], 2, dim=192), _weights(21, 2)
    b.kv[:128] = (b.kv[:128].float() * 2.0 ** -8).to(torch.bfloat16)
    b.kv[256:, :512] = (b.kv[256:, :512].float() * 2.0 ** 17).to(torch.bfloat16)
    b.q[:, :, :128] = (b.q[:, :, :128].float() * 2.0 ** -17).to(torch.bfloat16)
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_exact(o, b, w)


@pytest.mark.parametrize("v", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H", [3, 300])      # shares of steps; whole items
def test_expanded_a_row_that_only_later_queries_see(dsa, ix, v, H):
    b, w = Batch(72, [400, 390, 380], [400, 390, 380], H, dim=192), _weights(22, H)
    b.kv[150, 7] = v
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    assert not np.any(np.isfinite(o[150:400]).all(axis=2))
    keep = b.kv.clone()
    b.kv = torch.nan_to_num(b.kv, 0, 0, 0)
    _check_exact(o, b, w, tokens=set(range(0, 150, 9)) | {149} | set(range(400, 1170, 111)))
    b.kv = keep


def test_expanded_out_of_any_alignment_and_padding(dsa, ix):
    # out 16-byte but not 32-byte aligned; tokens of no sequence before the first and behind the last
    b, w = Batch(73, [260, 140], [130, 140], 5, dim=192), _weights(23, 5)
    b.qo = torch.tensor([2, 130, 265], dtype=torch.int32)
    b.pos = torch.cat((torch.tensor([-9, 1 << 20]), torch.arange(132, 260), torch.arange(0, 135), torch.full((5,), 77777))).int()
    buf = torch.full((270 * 5 * 128 + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8:].view(270, 5, 128)
    o = _expanded(ix, b, w, out=out)
    assert ix.device_error() == dsa.DSA_OK
    assert np.all(o[:2] == 7) and np.all(o[265:] == 7) and bool((buf[:8] == 7).all())
    _check_exact(o, b, w)


def test_many_short_sequences(dsa, ix):
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(0, 7, 1500)]
    nq = [min(n, int(x)) for n, x in zip(lens, r.integers(0, 3, 1500))]
    b = Batch(74, lens, nq, 4)
    o, lse = ix.latent_attention(*b.dev("q", "kv", "pos", "qo", "co"), SCALE)
    assert ix.device_error() == dsa.DSA_OK
    _check(f64(o), f64(lse), f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())
    b, w = Batch(75, lens, nq, 4, dim=192), _weights(24, 4)
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_exact(o, b, w)


@pytest.mark.parametrize("H", [97, 1024])
def test_more_heads_than_a_group(dsa, ix, H):
    b = Batch(76, [150, 20], [2, 1], H)
    kv4, val = _quantized(b.kv)
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    o, lse = ix.latent_attention(q, kv, pos, qo, co, SCALE)
    _check(f64(o), f64(lse), f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())
    idx = torch.full((3, 40), -1, dtype=torch.int32)
    for t, p in enumerate(b.pos.tolist()):
        idx[t, 3:3 + min(30, p + 1)] = torch.randperm(p + 1)[:30].to(torch.int32)
    o, lse = ix.latent_attention_fp4(q, kv4.to(DEV), None, qo, co, SCALE, idx=idx.to(DEV))
    assert ix.device_error() == dsa.DSA_OK
    _check(f64(o), f64(lse), f64(b.q), val, None, b.qo.numpy(), b.co.numpy(), idx=idx.numpy())


@pytest.mark.parametrize("q_exp", [-100, -40, 40, 100])
def test_4bit_queries_outside_the_range_of_fp16(dsa, ix, q_exp):
    # the scale undoes the queries' power of two: the same outputs bit for bit, since no rounding
    # step depends on it
    b = Batch(77, [700], [2], 24)
    kv4 = _quantized(b.kv)[0].to(DEV)
    q, pos, qo, co = b.dev("q", "pos", "qo", "co")
    want = ix.latent_attention_fp4(q, kv4, pos, qo, co, 0.0625)
    far = (q.float() * 2.0 ** q_exp).to(torch.bfloat16)
    got = ix.latent_attention_fp4(far, kv4, pos, qo, co, 0.0625 * 2.0 ** -q_exp)
    assert ix.device_error() == dsa.DSA_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_4bit_error_is_that_of_fp16_weights(dsa, ix):
    b = Batch(78, [900, 300], [2, 1], 96)
    kv4, val = _quantized(b.kv)
    q, pos, qo, co = b.dev("q", "pos", "qo", "co")
    o, lse = (f64(x) for x in ix.latent_attention_fp4(q, kv4.to(DEV), pos, qo, co, SCALE))
    ref, lref, mag = oracle.latent_attention(f64(b.q), val, b.pos.numpy(), b.qo.numpy(), b.co.numpy(), SCALE)
    qn = np.linalg.norm(f64(b.q), axis=2)
    e = 6 * np.sqrt(576) * 2.0 ** -24 * SCALE * qn * np.linalg.norm(val, axis=1).max() + 4 * 2.0 ** -24 * 60 + 2.0 ** -20
    tol = 1.01 * U * np.abs(ref) + (1.05 * F + 2 * np.expm1(e)[..., None]) * (mag + np.abs(ref)) + 2.0 ** -19 * np.abs(val).max()
    assert np.all(np.abs(o - ref) <= tol)
    assert np.all(np.abs(lse - lref) <= e + 2.0 ** -22 * (np.abs(lref) + 8) + 1e-6)


@pytest.mark.parametrize("lens,nq,H", [([2500], [300], 3), ([1900, 1700], [1, 260], 5), ([5000], [5], 2),
                                       ([3000], [129], 1)])
def test_expanded_few_long_items_in_equal_shares(dsa, ix, lens, nq, H):
    b, w = Batch(80 + H, lens, nq, H, dim=192), _weights(30 + H, H)
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_exact(o, b, w)
    assert np.array_equal(o, _expanded(ix, b, w))


def test_expanded_equal_shares_beside_a_nan_and_without_tokens(dsa, ix):
    b, w = Batch(81, [2200], [400], 3, dim=192), _weights(31, 3)
    b.kv[2000, 11] = float("nan")
    b.pos[7], b.pos[8] = -1, 3
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    assert np.all(o[7] == 0) and not np.any(np.isfinite(o[200:]).all(axis=2))
    b.kv = torch.nan_to_num(b.kv, 0)
    _check_exact(o, b, w, tokens={0, 5, 7, 8, 100, 199})
    b.co = torch.tensor([0, 2201], dtype=torch.int64)
    assert np.all(_expanded(ix, b, w) == 0) and ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS


def test_prompt_then_decode_through_one_cache(dsa, ix):
    # a prompt in the expanded form, its latents into the 4-bit cache, then tokens in the absorbed
    # form over both caches: the absorbed form over the values the 4-bit rows stand for is the same
    # operator over another cache, so its two results differ by the weights' types alone
    H, n = 16, 700
    b, w = Batch(82, [n], [n], H, dim=192), _weights(32, H)
    _check_exact(_expanded(ix, b, w), b, w, tokens=set(range(0, n, 37)))
    kv = b.kv.to(DEV)
    cache4 = torch.zeros((n + 3, 416), dtype=torch.uint8, device=DEV)
    ix.quantize_latent_fp4(kv, out=cache4, rows=torch.arange(3, n + 3, device=DEV))
    back = ix.dequantize_latent_fp4(cache4, rows=torch.arange(3, n + 3, device=DEV))
    d = Batch(83, [n], [4], H)
    q, pos = d.q.to(DEV), d.pos.to(DEV)
    qo = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    co4 = torch.tensor([3, n + 3], dtype=torch.int64, device=DEV)
    co = torch.tensor([0, n], dtype=torch.int64, device=DEV)
    o4, l4 = (f64(x) for x in ix.latent_attention_fp4(q, cache4, pos, qo, co4, SCALE))
    o, lse = (f64(x) for x in ix.latent_attention(q, back, pos, qo, co, SCALE))
    assert ix.device_error() == dsa.DSA_OK
    ref, lref, mag = oracle.latent_attention(f64(d.q), f64(back), d.pos.numpy(), [0, 4], [0, n], SCALE)
    assert np.all(np.abs(o4 - o) <= 2.02 * U * np.abs(ref) + (1.01 * U + 1.1 * F + 1e-4) * (mag + np.abs(ref)) + 1e-5)
    assert np.all(np.abs(l4 - lse) <= 1e-4) and np.all(np.abs(lse - lref) <= 1e-4)


def test_a_workspace_at_any_16_bytes(dsa, ix):
    import ctypes
    from dsa_lightning_indexer_03_b200 import _lib
    lib = _lib.load()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for n, nq, H in ((300, 140, 4), (2500, 300, 3)):
        b, w = Batch(90, [n], [nq], H, dim=192), _weights(33, H).to(DEV)
        q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
        want = ix.latent_attention_expanded(q, kv, w, pos, qo, co, SCALE)
        need = lib.dsa_indexer_latent_expanded_workspace(ix._h, nq, 1, H, n)
        ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
        for off in (16, 48, 240):
            out = torch.zeros_like(want)
            torch.cuda.synchronize()
            st = lib.dsa_indexer_latent_attention_expanded(ix._h, nq, p(q), H, p(kv), n, p(w), p(pos), p(qo), 1, p(co), SCALE,
                                                           p(out), ctypes.c_void_p(ws.data_ptr() + off), need, None)
            torch.cuda.synchronize()
            assert st == dsa.DSA_OK and ix.device_error() == dsa.DSA_OK and torch.equal(out, want)
        d = Batch(91, [n], [2], H)
        q, kv, pos, qo, co = d.dev("q", "kv", "pos", "qo", "co")
        want, lse = ix.latent_attention(q, kv, pos, qo, co, SCALE)
        need = lib.dsa_indexer_latent_attention_workspace(ix._h, 2, 1, H)
        out, l2 = torch.zeros_like(want), torch.zeros_like(lse)
        ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        st = lib.dsa_indexer_latent_attention(ix._h, 2, p(q), H, p(kv), n, p(pos), p(qo), 1, p(co), SCALE, p(out), p(l2),
                                              ctypes.c_void_p(ws.data_ptr() + 48), need, None)
        torch.cuda.synchronize()
        assert st == dsa.DSA_OK and torch.equal(out, want) and torch.equal(l2, lse)
