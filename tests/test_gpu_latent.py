"""Latent-cache operators against the fp64 oracle, through the public binding: dense attention
in the absorbed form (bf16 and 4-bit cache, and over a selection of a 4-bit cache), the 4-bit
rows, and the expanded form.

Tolerances, from the arithmetic (U = 2^-8, bf16's unit roundoff; all bounds per value).
  * scores: fp32 sums of D exact bf16 products, allowed e_s = 6 sqrt(D) 2^-24 scale |q| max|row|
    (a six-sigma random walk of the rounding), plus 4 * 2^-24 max|x| for the score's own scaling
    and shift before the exponential, plus 2^-21 for the exponential.
  * weights enter P.V as bf16 (<= U each, the normaliser is their unrounded sum) and out is
    rounded once (<= U |o|):  |o - o_ref| <= 1.01 U (mag + |o_ref|) + 2 e (mag + |o_ref|) + 1e-6
    with mag = sum_j w_j |v_j| and e the score allowance.
  * lse, from the unrounded sum: |lse - lse_ref| <= e + 2^-22 (|lse_ref| + 8) + 1e-6.
  * expanded: keys and values are bf16 roundings of fp32 sums of 512 products.  A sum that lies
    near a rounding border may round to the other side: at most 4 of a key's 128 values are
    allowed to (the chance for one is about 2^-24 sqrt(512) / U ~ 1e-3), each worth one step
    2 U max|k|: e_k = 8 U scale max|q| max|k|; and a value by one step: 2 U mag is added once."""

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from _parity import f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
SCALE = 192 ** -0.5
DEV = "cuda"


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


class Batch:
    """Sequences of lens[b] cached rows whose last nq[b] positions are queried."""

    def __init__(self, seed, lens, nq, H, dim=576, q_std=1.0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
        self.q = (r(sum(nq), H, dim).float() * q_std).to(torch.bfloat16)
        self.kv = r(max(1, sum(lens)), 576)
        self.pos = torch.tensor([p for n, m in zip(lens, nq) for p in range(n - m, n)], dtype=torch.int32)
        self.qo = torch.tensor(np.concatenate(([0], np.cumsum(nq))), dtype=torch.int32)
        self.co = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int64)

    def dev(self, *names):
        return [getattr(self, n).to(DEV) for n in names]


def _quantized(kv):
    """4-bit rows packed from the oracle's codes, and the values they stand for."""
    s, codes, val = oracle.quantize_latent_fp4(f64(kv))
    out = np.zeros((kv.shape[0], oracle.FP4_ROW_BYTES), np.uint8)
    out[:, :256] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    out[:, 256:288] = torch.from_numpy(s).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    out[:, 288:] = kv[:, 512:].contiguous().view(torch.uint8).numpy()
    return torch.from_numpy(out), val


def _allow(q_t, rows, scale, D):
    """Score allowance of each head of one query."""
    if rows.shape[0] == 0:
        return np.zeros(q_t.shape[0])
    x = np.abs(scale * (q_t @ rows.T)).max(1) if rows.ndim == 2 else np.abs(scale * np.einsum("hd,nhd->hn", q_t, rows)).max(1)
    rn = np.linalg.norm(rows, axis=-1).max()
    return 6 * np.sqrt(D) * 2.0 ** -24 * scale * np.linalg.norm(q_t, axis=1) * rn + 4 * 2.0 ** -24 * x + 2.0 ** -21


def _check(o, lse, q, kv, pos, qo, co, idx=None, scale=SCALE, rows=None):
    """o and lse of the tokens `rows` (all by default) against the oracle."""
    o_ref, lse_ref, mag = oracle.latent_attention(q, kv, pos, qo, co, scale, idx=idx)
    for t in (range(int(qo[0]), int(qo[-1])) if rows is None else rows):
        r0, r1 = oracle.latent_oracle.sequence_rows(t, qo, co)
        if idx is None:
            sel = kv[r0:r0 + int(pos[t]) + 1]
        else:
            i = np.asarray(idx[t], np.int64)
            sel = kv[r0 + i[(i >= 0) & (i < r1 - r0)]]
        e = _allow(q[t], sel, scale, 576)
        assert np.array_equal(np.isneginf(lse[t]), np.isneginf(lse_ref[t])), t
        fin = np.isfinite(lse_ref[t])
        dl = np.abs(lse[t][fin] - lse_ref[t][fin])
        assert np.all(dl <= (e + 2.0 ** -22 * (np.abs(lse_ref[t]) + 8) + 1e-6)[fin]), (t, dl.max())
        tol = (1.01 * U + 2 * e[:, None]) * (mag[t] + np.abs(o_ref[t])) + 1e-6
        err = np.abs(o[t] - o_ref[t])
        assert np.all(err <= tol), (t, err.max(), (err / tol).max())


def _run(dsa, ix, b, expect=None, **kw):
    o, lse = ix.latent_attention(*b.dev("q", "kv", "pos", "qo", "co"), SCALE, **kw)
    torch.cuda.synchronize()
    assert ix.device_error() == (dsa.DSA_OK if expect is None else expect)
    return f64(o), f64(lse)


SHAPES = [
    ([1], [1], 1),                       # one token, one head
    ([37], [1], 96),
    ([127, 128, 129], [1, 1, 1], 16),    # around a tile of 128 tokens
    ([256, 257, 15, 16, 17], [1, 2, 3, 1, 1], 8),
    ([500, 2], [5, 2], 96),              # several queries a sequence, ragged causal limits
    ([260], [260], 3),                   # a whole prompt
    ([300, 40], [3, 1], 128),            # more heads than one group of rows holds
    ([700], [3], 24),
    ([90, 0, 33], [2, 0, 1], 12),        # a sequence without queries or rows
    ([3000, 1700, 911], [1, 1, 2], 48),
    ([5000], [1], 6),                    # a long prefix split over many thread blocks
]


@pytest.mark.parametrize("lens,nq,H", SHAPES)
def test_dense(dsa, ix, lens, nq, H):
    b = Batch(len(lens) * 1000 + H, lens, nq, H)
    o, lse = _run(dsa, ix, b)
    _check(o, lse, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())


@pytest.mark.parametrize("lens,nq,H", SHAPES)
def test_dense_4bit(dsa, ix, lens, nq, H):
    b = Batch(len(lens) * 1000 + H + 1, lens, nq, H)
    kv4, val = _quantized(b.kv)
    q, pos, qo, co = b.dev("q", "pos", "qo", "co")
    o, lse = ix.latent_attention_fp4(q, kv4.to(DEV), pos, qo, co, SCALE)
    assert ix.device_error() == dsa.DSA_OK
    _check(f64(o), f64(lse), f64(b.q), val, b.pos.numpy(), b.qo.numpy(), b.co.numpy())


@pytest.mark.parametrize("lens,nq,H,k", [([200, 90], [3, 2], 96, 100), ([1], [1], 4, 1), ([400], [4], 16, 2048),
                                         ([1500, 700], [1, 2], 128, 257), ([2500], [2], 24, 2048), ([300], [2], 8, 128)])
def test_selected_4bit(dsa, ix, lens, nq, H, k):
    b = Batch(77 + k, lens, nq, H)
    kv4, val = _quantized(b.kv)
    g = torch.Generator().manual_seed(k)
    idx = torch.full((sum(nq), k), -1, dtype=torch.int32)
    for t, p in enumerate(b.pos.tolist()):
        n = min(k, p + 1)
        idx[t, torch.randperm(k, generator=g)[:n]] = torch.randperm(p + 1, generator=g)[:n].to(torch.int32)
    if k > 100:
        idx[0, 5:9] = idx[0, 60]          # the same index several times
    q, qo, co = b.dev("q", "qo", "co")
    o, lse = ix.latent_attention_fp4(q, kv4.to(DEV), None, qo, co, SCALE, idx=idx.to(DEV))
    assert ix.device_error() == dsa.DSA_OK
    _check(f64(o), f64(lse), f64(b.q), val, None, b.qo.numpy(), b.co.numpy(), idx=idx.numpy())


@pytest.mark.parametrize("q_std,H", [(4.0, 96), (12.0, 40)])
def test_scores_that_keep_rising(dsa, ix, q_std, H):
    # spreads of tens of units: the running maximum has to be raised again and again
    b = Batch(int(q_std), [1300, 600], [2, 1], H, q_std=q_std)
    o, lse = _run(dsa, ix, b)
    _check(o, lse, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())
    # rows along q whose scores climb with the position, for every head alike
    b = Batch(5, [1000], [1], 32)
    b.q[:] = b.q[:1, :1]
    b.kv[:] = (b.kv[:1].float() * 0 + b.q[0, 0].float() * torch.linspace(-2, 2, 1000)[:, None]).to(torch.bfloat16)
    o, lse = _run(dsa, ix, b)
    _check(o, lse, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())


def test_scores_far_below_zero_and_equal_weights(dsa, ix):
    # every score near -10,000 (no weight may underflow against a fixed reference) ...
    b = Batch(6, [300], [1], 16)
    b.q[:] = 64.0
    b.kv[:] = (-4.0 + b.kv.float() * 0.01).to(torch.bfloat16)
    o, lse = _run(dsa, ix, b)
    _check(o, lse, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())
    # ... and q = 0: the mean of the latents, ln n
    b = Batch(7, [900, 130], [2, 1], 24)
    b.q.zero_()
    o, lse = _run(dsa, ix, b)
    n = b.pos.numpy() + 1
    np.testing.assert_allclose(lse, np.broadcast_to(np.log(n)[:, None], lse.shape), rtol=0, atol=1e-5)
    _check(o, lse, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())


def test_positions_in_any_order_and_empty_queries(dsa, ix):
    b = Batch(8, [400, 150], [5, 4], 24)
    b.pos = torch.tensor([399, -1, 0, 130, 17, -1, -1, 149, 3], dtype=torch.int32)
    o, lse = _run(dsa, ix, b)
    _check(o, lse, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())
    assert np.all(o[1] == 0) and np.all(np.isneginf(lse[1]))
    # one token: its latent, bit for bit
    np.testing.assert_array_equal(o[2], np.broadcast_to(f64(b.kv[0, :512]), (24, 512)))


def test_what_lies_behind_the_prefix_is_never_used(dsa, ix):
    # rows past the queried positions and past the last sequence hold NaN and infinities, as
    # memory that nothing has written may
    b = Batch(9, [140, 77, 200], [1, 1, 1], 16)
    b.pos = torch.tensor([99, 60, 130], dtype=torch.int32)
    want = _run(dsa, ix, b)
    for v in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        for r0, p, r1 in ((0, 99, 140), (140, 60, 217), (217, 130, 417)):
            b.kv[r0 + p + 1:r1] = v
        got = _run(dsa, ix, b)
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])


@pytest.mark.parametrize("v", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,H", [(200, 40), (3000, 6)])     # in one block's share; split over many
def test_a_row_that_only_later_queries_see_may_hold_anything(dsa, ix, v, n, H):
    b = Batch(15, [n], [3], H)
    b.pos = torch.tensor([n - 60, n - 20, n - 2], dtype=torch.int32)
    want = _run(dsa, ix, b)
    b.kv[n - 30, 5] = v
    b.kv[n - 10] = v
    o, lse = _run(dsa, ix, b)
    np.testing.assert_array_equal(lse[0], want[1][0])
    keep = Batch(15, [n], [1], H)
    keep.q, keep.kv, keep.pos = b.q[:1], torch.nan_to_num(b.kv, 0, 0, 0), b.pos[:1]
    _check(o[:1], lse[:1], f64(keep.q), f64(keep.kv), keep.pos.numpy(), keep.qo.numpy(), keep.co.numpy())
    assert not np.any(np.isfinite(o[1:, :, 5]))       # they attend to it


def test_padded_batch_leaves_its_rows_as_they_were(dsa, ix):
    b = Batch(10, [300, 100], [3, 2], 32)
    b.qo = torch.tensor([0, 2, 3], dtype=torch.int32)            # tokens 3 and 4 belong to no sequence
    b.pos = torch.tensor([298, 299, 99, 1 << 20, -7], dtype=torch.int32)
    out = torch.full((5, 32, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((5, 32), 7.0, device=DEV)
    o, l = _run(dsa, ix, b, out=out, lse=lse)
    _check(o, l, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())
    assert np.all(o[3:] == 7) and np.all(l[3:] == 7)


def test_bad_positions_and_offsets_are_reported(dsa, ix):
    b = Batch(11, [200, 150], [2, 2], 8)
    good = b.pos.clone()
    b.pos[1], b.pos[3] = 200, -2                                  # past the sequence; below -1
    o, lse = _run(dsa, ix, b, expect=dsa.DSA_ERR_DEVICE_BOUNDS)
    b.pos = torch.tensor([good[0], -1, good[2], -1], dtype=torch.int32)
    _check(o, lse, f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())
    for qo, co in (([0, 3, 2], [0, 200, 350]), ([0, 2, 4], [0, 200, 351]), ([0, 2, 4], [0, 200, 100]),
                   ([0, 2, 5], [0, 200, 350]), ([-1, 2, 4], [0, 200, 350]), ([0, 2, 4], [-1, 200, 350])):
        b.qo, b.co = torch.tensor(qo, dtype=torch.int32), torch.tensor(co, dtype=torch.int64)
        o, lse = _run(dsa, ix, b, expect=dsa.DSA_ERR_DEVICE_BOUNDS)
        assert np.all(o == 0) and np.all(np.isneginf(lse))
    # an entry past its sequence's rows is skipped and reported
    b = Batch(12, [60, 50], [1, 1], 4)
    kv4, val = _quantized(b.kv)
    idx = torch.tensor([[3, 59, 60, -1], [49, -1, 1 << 30, 0]], dtype=torch.int32)
    q, qo, co = b.dev("q", "qo", "co")
    o, lse = ix.latent_attention_fp4(q, kv4.to(DEV), None, qo, co, SCALE, idx=idx.to(DEV))
    assert ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS
    _check(f64(o), f64(lse), f64(b.q), val, None, b.qo.numpy(), b.co.numpy(), idx=idx.numpy())
    # k_sel = 0: no token
    o, lse = ix.latent_attention_fp4(q, kv4.to(DEV), None, qo, co, SCALE,
                                     idx=torch.empty((2, 0), dtype=torch.int32, device=DEV))
    assert ix.device_error() == dsa.DSA_OK and bool((o == 0).all()) and bool(torch.isneginf(lse).all())


def test_a_cache_past_32_bit_offsets(dsa, ix):
    # the last sequence lies past 2^31 values of the cache (and past 2^32 bytes)
    rows, n = (1 << 31) // 576 + 5000, 700
    kv = torch.empty((rows, 576), dtype=torch.bfloat16, device=DEV)
    b = Batch(13, [n], [2], 96)
    kv[rows - n:] = b.kv.to(DEV)
    co = torch.tensor([0, rows - n, rows], dtype=torch.int64, device=DEV)
    qo = torch.tensor([0, 0, 2], dtype=torch.int32, device=DEV)
    o, lse = ix.latent_attention(b.q.to(DEV), kv, b.pos.to(DEV), qo, co, SCALE)
    assert ix.device_error() == dsa.DSA_OK
    _check(f64(o), f64(lse), f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy())


def test_repeatable_on_streams_and_in_graphs(dsa, ix):
    b = Batch(14, [4000, 900, 2500], [1, 3, 1], 64)
    kv4 = ix.quantize_latent_fp4(b.kv.to(DEV))
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    calls = [lambda **k: ix.latent_attention(q, kv, pos, qo, co, SCALE, **k),
             lambda **k: ix.latent_attention_fp4(q, kv4, pos, qo, co, SCALE, **k)]
    for call in calls:
        want = call()
        again = call()
        assert all(torch.equal(x, y) for x, y in zip(want, again))
        # two calls at once on two streams, each with its own workspace
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        outs = [call(stream=s) for s in (s1, s2, s1, s2)]
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(x, y) for x, y in zip(want, got))
        # two graphs, replayed in turn with new inputs, against eager calls
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                res = call()
            graphs.append((g, res))
        keep = q.clone()
        for k in range(4):
            q.copy_(torch.roll(keep, k, 0))
            g, res = graphs[k & 1]
            g.replay()
            eager = call()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(res, eager))
        q.copy_(keep)
    assert ix.device_error() == dsa.DSA_OK


# ------------------------------------------------------------------------------ 4-bit rows

@pytest.mark.parametrize("n", [1, 7, 64, 301])
def test_quantize_matches_the_oracle_bit_for_bit(dsa, ix, n):
    r = np.random.default_rng(n)
    x = oracle.bf16_round(r.standard_normal((n, 576)) * 10.0 ** r.integers(-4, 4, (n, 1)))
    x[0, :16] = oracle.bf16_round(np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.3, -2.4, 0, 5.5, -6]) * 0.40625)
    x[0, 16:32] = 0
    x[0, 32:48] = 2.0 ** -20                       # below the smallest scale
    x[0, 48:64] = 1e6                              # beyond the largest
    x[n // 2, 512:] *= 100
    kv = torch.from_numpy(x).to(torch.bfloat16)
    want, val = _quantized(kv)
    got = ix.quantize_latent_fp4(kv.to(DEV))
    np.testing.assert_array_equal(got.cpu().numpy(), want.numpy())
    np.testing.assert_array_equal(f64(ix.dequantize_latent_fp4(got)), val)
    # scattered into a cache and read back; the other rows stay as they were
    cache = torch.full((3 * n, 416), 9, dtype=torch.uint8, device=DEV)
    rows = torch.from_numpy(r.permutation(3 * n)[:n].astype(np.int64)).to(DEV)
    assert ix.quantize_latent_fp4(kv.to(DEV), out=cache, rows=rows) is cache
    ref = torch.full((3 * n, 416), 9, dtype=torch.uint8)
    ref[rows.cpu()] = want
    assert torch.equal(cache.cpu(), ref)
    np.testing.assert_array_equal(f64(ix.dequantize_latent_fp4(cache, rows=rows)), val)
    assert ix.device_error() == dsa.DSA_OK


def test_every_tie_of_every_scale_goes_to_the_even_code(dsa, ix):
    # blocks whose largest value is 6 s for each of the 119 scales s from 2^-6 up, holding
    # every midpoint mid * s that bf16 can hold, its two bf16 neighbours and both signs
    codes = torch.arange(8, 127, dtype=torch.uint8)
    s = codes.view(torch.float8_e4m3fn).float()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    blocks = []
    for d in (-1, 0, 1):
        blk = torch.zeros((s.numel(), 16))
        blk[:, 0] = 6 * s
        m = (mids[None] * s[:, None]).to(torch.bfloat16)
        m = (m.view(torch.int16) + d).view(torch.bfloat16).float()
        blk[:, 1:8], blk[:, 8:15] = m, -m
        blocks.append(blk)
    flat = torch.cat(blocks).to(torch.bfloat16)
    lat = torch.zeros((12 * 32, 16), dtype=torch.bfloat16)
    lat[:flat.shape[0]] = flat
    rows = torch.cat((lat.view(12, 512), torch.ones((12, 64), dtype=torch.bfloat16)), dim=1)
    want, _ = _quantized(rows)
    np.testing.assert_array_equal(ix.quantize_latent_fp4(rows.to(DEV)).cpu().numpy(), want.numpy())


def test_bad_rows_are_skipped_and_reported(dsa, ix):
    kv = torch.randn((4, 576)).to(torch.bfloat16).to(DEV)
    cache = torch.full((6, 416), 5, dtype=torch.uint8, device=DEV)
    rows = torch.tensor([1, 6, -1, 4], dtype=torch.int64, device=DEV)
    ix.quantize_latent_fp4(kv, out=cache, rows=rows)
    assert ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS
    one = ix.quantize_latent_fp4(kv)
    assert torch.equal(cache[1], one[0]) and torch.equal(cache[4], one[3])
    assert bool((cache[[0, 2, 3, 5]] == 5).all())
    back = ix.dequantize_latent_fp4(cache, rows=rows)
    assert ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS
    assert bool((back[1:3] == 0).all()) and torch.equal(back[0], ix.dequantize_latent_fp4(one)[0])


# ------------------------------------------------------------------------------ expanded form

def _weights(seed, H):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((H, 256, 512), generator=g) * 512 ** -0.5).to(torch.bfloat16)


def _check_expanded(o, b, w, rows=None):
    q, kv, pos, qo, co = f64(b.q), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy()
    o_ref, mag = oracle.latent_attention_expanded(q, kv, f64(w), pos, qo, co, SCALE)
    k, _ = oracle.latent_oracle.expand(kv, f64(w))
    for t in range(int(qo[0]), int(qo[-1])):
        r0, _ = oracle.latent_oracle.sequence_rows(t, qo, co)
        sel = k[r0:r0 + int(pos[t]) + 1]
        e = _allow(q[t], sel, SCALE, 192)
        if sel.shape[0]:
            e = e + 8 * U * SCALE * np.abs(q[t]).max(1) * np.abs(sel[:, :, :128]).max()
        tol = (1.01 * U + 2 * e[:, None]) * (mag[t] + np.abs(o_ref[t])) + 2 * U * mag[t] + 1e-6
        err = np.abs(o[t] - o_ref[t])
        assert np.all(err <= tol), (t, err.max(), (err / tol).max())


@pytest.mark.parametrize("lens,nq,H", [([1], [1], 1), ([128], [128], 2), ([129, 127, 1], [129, 127, 1], 3),
                                       ([300], [300], 5), ([700, 90], [100, 90], 2), ([513, 0, 40], [257, 0, 1], 4),
                                       ([1030], [3], 16)])
def test_expanded(dsa, ix, lens, nq, H):
    b, w = Batch(30 + H, lens, nq, H, dim=192), _weights(H, H)
    o = ix.latent_attention_expanded(*b.dev("q", "kv"), w.to(DEV), *b.dev("pos", "qo", "co"), SCALE)
    assert ix.device_error() == dsa.DSA_OK
    _check_expanded(f64(o), b, w)


def test_expanded_peaked_scores(dsa, ix):
    b, w = Batch(31, [600], [200], 2, dim=192, q_std=8.0), _weights(9, 2)
    o = ix.latent_attention_expanded(*b.dev("q", "kv"), w.to(DEV), *b.dev("pos", "qo", "co"), SCALE)
    assert ix.device_error() == dsa.DSA_OK
    _check_expanded(f64(o), b, w)


def test_expanded_positions_padding_and_errors(dsa, ix):
    b, w = Batch(32, [300, 100], [4, 3], 3, dim=192), _weights(10, 3)
    b.pos = torch.tensor([299, -1, 0, 150, 99, 12, 1 << 20], dtype=torch.int32)
    b.qo = torch.tensor([0, 4, 6], dtype=torch.int32)
    # unused rows hold NaN: past the last queried position, and of a sequence nobody asks for
    b.kv[200:300] = float("nan")
    b.pos[0] = 199
    out = torch.full((7, 3, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    args = lambda: [*b.dev("q", "kv"), w.to(DEV), *b.dev("pos", "qo", "co"), SCALE]  # noqa: E731
    o = f64(ix.latent_attention_expanded(*args(), out=out))
    assert ix.device_error() == dsa.DSA_OK
    assert np.all(o[6] == 7) and np.all(o[1] == 0) and np.all(np.isfinite(o))
    keep = b.kv.clone()
    b.kv = torch.nan_to_num(b.kv)
    _check_expanded(o, b, w)
    b.kv = keep
    b.pos[1] = 300
    o = f64(ix.latent_attention_expanded(*args(), out=out))
    assert ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS and np.all(o[1] == 0)
    b.co = torch.tensor([0, 300, 401], dtype=torch.int64)
    o = f64(ix.latent_attention_expanded(*args()))
    assert ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS and np.all(o == 0)


def test_expanded_streams_and_graphs(dsa, ix):
    b, w = Batch(33, [500, 260], [300, 260], 4, dim=192), _weights(11, 4).to(DEV)
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    want = ix.latent_attention_expanded(q, kv, w, pos, qo, co, SCALE)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [ix.latent_attention_expanded(q, kv, w, pos, qo, co, SCALE, stream=s) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(want, x) for x in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = ix.latent_attention_expanded(q, kv, w, pos, qo, co, SCALE)
    q.copy_(torch.roll(q, 1, 0))
    g.replay()
    eager = ix.latent_attention_expanded(q, kv, w, pos, qo, co, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(res, eager) and not torch.equal(res, want)


# ------------------------------------------------------------------------------ together

def test_the_expanded_and_absorbed_forms_agree(dsa, ix):
    # absorbing W_uk into the query and applying W_uv to the absorbed output gives the expanded
    # form up to the bf16 roundings of either path: keys, values, the absorbed query, its output
    # and the weights, each at most U of a term; 6 of them on a sum of magnitudes bound it
    H, n = 4, 400
    b, w = Batch(34, [n], [60], H, dim=192), _weights(12, H)
    o = f64(ix.latent_attention_expanded(*b.dev("q", "kv"), w.to(DEV), *b.dev("pos", "qo", "co"), SCALE))
    wd, q = f64(w), f64(b.q)
    qa = torch.from_numpy(np.concatenate((np.einsum("thd,hdc->thc", q[:, :, :128], wd[:, :128]), q[:, :, 128:]), axis=2))
    oa, _ = ix.latent_attention(qa.to(torch.bfloat16).to(DEV), *b.dev("kv", "pos", "qo", "co"), SCALE)
    got = np.einsum("thc,hdc->thd", f64(oa), wd[:, 128:])
    _, mag = oracle.latent_attention_expanded(q, f64(b.kv), wd, b.pos.numpy(), b.qo.numpy(), b.co.numpy(), SCALE)
    # a score moves by at most U * scale * sum_d |q_d k_d| for the keys and as much for the query
    k = np.abs(oracle.latent_oracle.expand(f64(b.kv), wd)[0])[:, :, :128].max(0)
    e = 2 * U * SCALE * np.einsum("thd,hd->th", np.abs(q[:, :, :128]), k)
    _, _, mag_lat = oracle.latent_attention(f64(qa.to(torch.bfloat16)), f64(b.kv), b.pos.numpy(), b.qo.numpy(), b.co.numpy(), SCALE)
    out_round = U * np.einsum("thc,hdc->thd", mag_lat, np.abs(wd[:, 128:]))
    assert np.all(np.abs(o - got) <= (4 * U + np.expm1(2 * e)[..., None]) * 2 * mag + 2 * out_round + 1e-6)


def test_project_select_and_attend_over_the_4bit_cache(dsa, ix):
    # a decode step as a serving loop runs it: the indexer projects and selects, the latent row
    # of the new token enters the 4-bit cache, and the attention reads the selection
    lens = [2600, 2100]
    dec = W.make_decode(50, lengths=lens, hidden_dim=128, q_latent_dim=64)
    mla = W.make_mla(51, lens, [1, 1], n_heads=96, k_sel=1)
    pos, qo, co = dec.positions.to(DEV), dec.q_seq_offsets.to(DEV), dec.cache_offsets.to(DEV)
    keys = ix.key_norm(dec.raw_keys.to(DEV))
    kv = mla.kv.to(DEV)
    last = (co[1:] - 1).contiguous()
    cache4 = ix.quantize_latent_fp4(kv)
    cache4[last] = 0
    q, w = ix.project(dec.hidden.to(DEV), dec.q_latent.to(DEV), pos, qo, keys, co)
    idx, _ = ix.topk(q, w, pos, qo, keys, co)
    ix.quantize_latent_fp4(kv[last].contiguous(), out=cache4, rows=last)
    o, lse = ix.latent_attention_fp4(mla.q.to(DEV), cache4, None, qo, co, SCALE, idx=idx)
    assert ix.device_error() == dsa.DSA_OK
    val = f64(ix.dequantize_latent_fp4(cache4))
    _check(f64(o), f64(lse), f64(mla.q), val, None, qo.cpu().numpy(), co.cpu().numpy(), idx=idx.cpu().numpy())
    # the same selection through the bf16 cache of the values stood for: bf16 weights in both,
    # one with the rounded and one with the unrounded normaliser
    o2, lse2 = ix.sparse_mla(mla.q.to(DEV), ix.dequantize_latent_fp4(cache4), co, qo, idx, SCALE)
    mag = np.abs(val[:, :512]).max(0)
    assert np.all(np.abs(f64(o) - f64(o2)) <= 1.01 * 4 * U * mag + 1e-5)
    assert np.all(np.abs(f64(lse) - f64(lse2)) <= 1.01 * U + 1e-4)
    # a selection of every row is the dense form
    full = torch.arange(2600, dtype=torch.int32, device=DEV).repeat(2, 1)
    full[1, 2100:] = -1
    a, la = ix.latent_attention_fp4(mla.q.to(DEV), cache4, None, qo, co, SCALE, idx=full)
    d, ld = ix.latent_attention_fp4(mla.q.to(DEV), cache4, pos, qo, co, SCALE)
    assert torch.equal(a, d) and torch.equal(la, ld)


def test_refusals(dsa, ix):
    b = Batch(40, [50], [2], 4)
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    kv4 = ix.quantize_latent_fp4(kv)
    ok = lambda **k: ix.latent_attention(*[{**dict(q=q, kv=kv, pos=pos, qo=qo, co=co), **k}[n]  # noqa: E731
                                           for n in ("q", "kv", "pos", "qo", "co")], k.get("scale", SCALE))
    ok()
    for bad in (dict(q=q.float()), dict(q=q[:, :, :512].contiguous()), dict(q=q.transpose(0, 1)), dict(q=q.cpu()),
                dict(kv=kv4), dict(kv=kv[:, ::2]), dict(pos=pos.long()), dict(pos=pos[:1]), dict(qo=qo.long()),
                dict(qo=qo[:1]), dict(co=co.int()), dict(co=co[:1])):
        with pytest.raises((TypeError, ValueError)):
            ok(**bad)
    for s in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(dsa.DSAError):
            ok(scale=s)
    with pytest.raises(dsa.DSAError):          # no cache rows
        ok(kv=kv[:0])
    odd = torch.empty(kv.numel() + 1, dtype=torch.bfloat16, device=DEV)[1:].view(kv.shape)
    with pytest.raises(dsa.DSAError):          # not 16-byte aligned
        ok(kv=odd)
    with pytest.raises(ValueError):
        ix.latent_attention_fp4(q, kv4, None, qo, co, SCALE)
    with pytest.raises(ValueError):
        ix.latent_attention_fp4(q, kv4, None, qo, co, SCALE, idx=torch.zeros((3, 4), dtype=torch.int32, device=DEV))
    with pytest.raises((TypeError, ValueError)):
        ix.latent_attention(q, kv, pos, qo, co, SCALE, out=torch.empty((2, 4, 576), dtype=torch.bfloat16, device=DEV))
    for bad in (lambda: ix.quantize_latent_fp4(kv.float()), lambda: ix.quantize_latent_fp4(kv[:, :512].contiguous()),
                lambda: ix.quantize_latent_fp4(kv, out=kv4[:10]),
                lambda: ix.quantize_latent_fp4(kv, rows=torch.arange(50, device=DEV)),
                lambda: ix.quantize_latent_fp4(kv, out=kv4, rows=torch.arange(49, device=DEV)),
                lambda: ix.dequantize_latent_fp4(kv), lambda: ix.dequantize_latent_fp4(kv4, rows=pos)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    w = _weights(1, 4).to(DEV)
    qe = q[:, :, :192].contiguous()
    ix.latent_attention_expanded(qe, kv, w, pos, qo, co, SCALE)
    for bad in (dict(w=w[:3].contiguous()), dict(q=q), dict(pos=None)):
        a = {**dict(q=qe, w=w, pos=pos), **bad}
        with pytest.raises(ValueError):
            ix.latent_attention_expanded(a["q"], kv, a["w"], a["pos"], qo, co, SCALE)
    # no tokens: nothing to do
    e, l = ix.latent_attention(q[:0], kv, pos[:0], torch.zeros_like(qo), co, SCALE)
    assert e.shape == (0, 4, 512) and l.shape == (0, 4)
    assert ix.quantize_latent_fp4(kv[:0]).shape == (0, 416)
    assert ix.device_error() == dsa.DSA_OK


def test_a_workspace_that_is_too_small_is_refused(dsa, ix):
    import ctypes
    from dsa_lightning_indexer_03_b200 import _lib
    lib = _lib.load()
    b = Batch(41, [50], [2], 4)
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    need = lib.dsa_indexer_latent_attention_workspace(ix._h, 2, 1, 4)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros((2, 4, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 4), device=DEV)
    call = lambda n: lib.dsa_indexer_latent_attention(ix._h, 2, p(q), 4, p(kv), 50, p(pos), p(qo), 1, p(co), SCALE,  # noqa: E731
                                                      p(out), p(lse), p(ws), n, None)
    assert call(need - 1) == dsa.DSA_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    assert call(need) == dsa.DSA_OK
    torch.cuda.synchronize()
    assert ix.device_error() == dsa.DSA_OK
