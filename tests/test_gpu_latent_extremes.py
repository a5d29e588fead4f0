"""Latent-cache operators on inputs at the ends of their number formats: zero queries and keys,
factors of a score far below one, and values of very different magnitude beside each other.

Tolerances (U = 2^-8 and F = 2^-11, the unit roundoffs of bf16 and fp16).  Everything a bound uses is
taken over the rows that the query attends to, none over rows it does not.
  * expanded: a key or value is rounded to fp16 under a scale that brings its row's largest
    magnitude to at least 2^6 (a tile's scale serves rows within 2^8 of its largest; others carry
    their own), so it is off by F of itself or, below fp16's normal range, by 2^-25 / 2^6 = 2^-31 of
    the row's largest.  A score moves by e_k = scale sum_d |q_d| (F |k_d| + 2^-31 max|k|) at most, and by
    the fp32 sums' e_s = 6 sqrt(192) 2^-24 scale |q| max|k| + 4 * 2^-24 max|x| + 2^-20.
    A weight is off by F of itself or by 2^-25 where the largest product of a weight and its
    value's scale is at least 2^7; scales are within 2^8 of what their row needs, so n such weights
    add at most n 2^-32 2^9 2 = n 2^-22 of the largest w_s max|v_s|.  With e = e_k + e_s:
    |o - o_ref| <= 1.01 U |o_ref| + (2.1 F + 2 expm1(e)) (mag + |o_ref|) + n 2^-22 max_s(w_s max|v_s|)
                   + 2^-30 sum_s w_s max|v_s|,   mag = sum_s w_s |v_s|.
  * 4-bit: values are exact, weights as above with the scales left out: n 2^-32 max|v|."""

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


def _check_seen(o, b, w, scale=SCALE, tokens=None):
    """o against the definition in 64 bits, each query from the rows it attends to alone."""
    q, kv, wd = f64(b.q), f64(b.kv), f64(w)
    pos, qo, co = b.pos.numpy(), b.qo.numpy(), b.co.numpy()
    for s in range(len(qo) - 1):
        r0 = int(co[s])
        ts = [t for t in range(int(qo[s]), int(qo[s + 1])) if tokens is None or t in tokens]
        n = max([int(pos[t]) + 1 for t in ts], default=0)
        c = kv[r0:r0 + n]
        for h in range(q.shape[1]):
            with np.errstate(all="ignore"):                  # rows that none of these queries sees whole
                k_all = np.concatenate((c[:, :512] @ wd[h, :128].T, c[:, 512:]), axis=1)
                v_all = c[:, :512] @ wd[h, 128:].T
            for t in ts:
                m = int(pos[t]) + 1
                if m == 0:
                    assert np.all(o[t, h] == 0)
                    continue
                k, v = k_all[:m], v_all[:m]
                x = scale * (k @ q[t, h])
                wt = np.exp(x - x.max())
                wt /= wt.sum()
                ref, mag, vmax, kmax = wt @ v, wt @ np.abs(v), np.abs(v).max(1), np.abs(k).max(1)
                e = scale * (np.abs(k) @ np.abs(q[t, h]) * F + 2.0 ** -31 * kmax * np.abs(q[t, h]).sum())
                e = e[wt > 1e-12].max()                      # a lighter row's move does not show
                e += 6 * np.sqrt(192) * 2.0 ** -24 * scale * np.linalg.norm(q[t, h]) * np.linalg.norm(k[wt > 1e-12], axis=1).max()
                e += 4 * 2.0 ** -24 * np.abs(x[wt > 1e-12]).max() + 2.0 ** -20
                tol = 1.01 * U * np.abs(ref) + (2.1 * F + 2 * np.expm1(min(e, 300.0))) * (mag + np.abs(ref))
                tol += m * 2.0 ** -22 * (wt * vmax).max() + 2.0 ** -30 * (wt * vmax).sum() + 1e-38
                err = np.abs(o[t, h] - ref)
                assert np.all(err <= tol), (t, h, err.max(), (err / tol).max())


def _shared(seed, n, nq, H):
    """A batch of one sequence beside two more, with few heads (shares of steps) or many (whole items)."""
    return Batch(seed, [n, 140], [nq, 20], H, dim=192), _weights(seed, H)


# ------------------------------------------------------------------------------ factors of a score

@pytest.mark.parametrize("what", ["q", "kv", "both", "a query", "a row", "a tile"])
@pytest.mark.parametrize("H", [2, 300])
def test_expanded_zeros(dsa, ix, what, H):
    b, w = _shared(101, 300, 150 if H == 2 else 40, H)
    if what in ("q", "both"):
        b.q.zero_()
    if what in ("kv", "both"):
        b.kv.zero_()
    if what == "a query":
        b.q[7] = 0
        b.q[3, 1] = 0
    if what == "a row":
        b.kv[5] = 0
        b.kv[131, 512:] = 0
    if what == "a tile":
        b.kv[128:256] = 0
        b.q[9] = 0
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_seen(o, b, w, tokens=None if H == 2 else {3, 7, 9, 39, 50})
    one = Batch(1, [1], [1], 1, dim=192)                     # a first token over a cache of zeros
    one.q.zero_(), one.kv.zero_()
    assert np.all(_expanded(ix, one, _weights(1, 1)) == 0)


@pytest.mark.parametrize("q_exp,kv_exp,s_exp", [(-60, -60, 0), (-100, -14, 0), (0, 0, -100), (0, 0, -120), (-100, 0, -20),
                                                (20, 20, -40), (-60, -60, 120)])
def test_expanded_factors_far_from_one(dsa, ix, q_exp, kv_exp, s_exp):
    b, w = _shared(102, 290, 100, 2)
    b.q = (b.q.float() * 2.0 ** q_exp).to(torch.bfloat16)
    b.kv = (b.kv.float() * 2.0 ** kv_exp).to(torch.bfloat16)
    b.q[4] = 0
    scale = SCALE * 2.0 ** s_exp
    o = _expanded(ix, b, w, scale)
    assert ix.device_error() == dsa.DSA_OK
    _check_seen(o, b, w, scale)


@pytest.mark.parametrize("s_exp", [0, -100, -125])
def test_4bit_zero_queries_and_small_scales(dsa, ix, s_exp):
    b = Batch(103, [300, 90], [3, 2], 24)
    b.q[1] = 0
    b.q[3, 5] = 0
    kv4, val = _quantized(b.kv)
    val[7], kv4[7] = 0, 0
    q, pos, qo, co = b.dev("q", "pos", "qo", "co")
    scale = 0.0625 * 2.0 ** s_exp
    o, lse = ix.latent_attention_fp4(q, kv4.to(DEV), pos, qo, co, scale)
    assert ix.device_error() == dsa.DSA_OK
    _check(f64(o), f64(lse), f64(b.q), val, b.pos.numpy(), b.qo.numpy(), b.co.numpy(), scale=scale)


def test_scales_at_the_end_of_the_range(dsa, ix):
    # a product of the largest scale with ln 2's inverse overflows: zero scores must stay zero
    b = Batch(104, [200], [2], 8)
    b.q.zero_()
    kv4, val = _quantized(b.kv)
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    for scale in (3.0e38, 2.0 ** -126, 1e-41):
        for o, lse, rows in ((*ix.latent_attention(q, kv, pos, qo, co, scale), f64(b.kv)),
                             (*ix.latent_attention_fp4(q, kv4.to(DEV), pos, qo, co, scale), val)):
            _check(f64(o), f64(lse), f64(b.q), rows, b.pos.numpy(), b.qo.numpy(), b.co.numpy(), scale=scale)
        e, w = Batch(105, [200], [2], 3, dim=192), _weights(3, 3)
        e.q.zero_()
        _check_seen(_expanded(ix, e, w, scale), e, w, scale)
    assert ix.device_error() == dsa.DSA_OK


# ------------------------------------------------------------------------------ rows computed again

_SLOW = """
import os, sys
os.environ["DSA_INDEXER_WAIT_TIMEOUT_MS"] = "20"
sys.path.insert(0, %r)
import torch, dsa_lightning_indexer_03_b200 as dsa
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
ix = dsa.Indexer(r(64, 4096), r(128, 128), r(128, 32), r(128), r(128), max_tokens=4096)
i = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")
for n, nq, H in ((30000, 200, 148), (30000, 200, 5)):
    q, kv, w = r(nq, H, 192), r(n, 576), r(H, 256, 512) * 512 ** -0.5
    pos, qo, co = torch.arange(n - nq, n, dtype=torch.int32, device="cuda"), i([0, nq]), i([0, n], torch.int64)
    args = (w, pos, qo, co, 192 ** -0.5)
    want = ix.latent_attention_expanded(q, kv, *args)
    assert ix.device_error() == dsa.DSA_OK
    kv[n - 40, 11] = float("nan")
    got = ix.latent_attention_expanded(q, kv, *args)
    assert ix.device_error() == dsa.DSA_OK, "timeout"
    seen = pos >= n - 40
    assert not bool(torch.isfinite(got[seen]).all(2).any())
    # fp32 weights instead of fp16 ones: 2^-11 of a sum of magnitudes, and a rounding of out either way
    d, m = (got - want)[~seen].float().abs(), want[~seen].float().abs()
    assert bool((d <= 2 * 2.0 ** -8 * m + 2.0 ** -11 * 0.1).all()), float(d.max())
print("fine")
"""


def test_expanded_rows_beside_a_nan_keep_nobody_waiting(dsa):
    # a limit of 20 ms on every wait in the kernels: computing a row of 30,000 tokens again takes part
    # in none (whole items and shares of steps)
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _SLOW % root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_expanded_infinite_values_stay_and_nan_rows_are_right(dsa, ix):
    # values of one head overflow to infinity while every score is finite: those outputs are
    # infinite, the other dims as ordinary; repeated bit for bit
    b, w = Batch(130, [600, 200], [300, 200], 3, dim=192), _weights(130, 3)
    w[1, :128] = 0
    w[1, 128 + 5] = 0
    w[1, 128 + 5, 3] = 3.0e38
    b.kv[:, 3] = 2.0
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    assert np.all(np.isposinf(o[:, 1, 5]))
    assert np.all(np.isfinite(np.delete(o[:, 1], 5, axis=1))) and np.all(np.isfinite(o[:, [0, 2]]))
    assert np.array_equal(o, _expanded(ix, b, w))
    fin = w.clone()
    fin[1, 128 + 5] = 0
    # a query of a tile that also holds rows it does not see (0 * inf) is computed again with fp32
    # weights instead of fp16 ones, so both results are held to the bound, not to each other's bits
    o[:, 1, 5] = 0
    _check_seen(o, b, fin)
    _check_seen(_expanded(ix, b, fin), b, fin)


@pytest.mark.parametrize("H", [3, 148])
def test_expanded_many_rows_beside_a_nan(dsa, ix, H):
    # whole tiles of queries in reverse order, most of which see neither of two broken rows
    b, w = Batch(131, [1100, 300], [256, 140], H, dim=192), _weights(131, H)
    b.pos = torch.cat((torch.arange(1099, 843, -1), torch.arange(299, 159, -1))).int()
    b.kv[1090, 8] = float("inf")
    b.kv[1100 + 250] = float("nan")
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    assert not np.any(np.isfinite(o[:10]).all(axis=2)) and not np.any(np.isfinite(o[256:306]).all(axis=2))
    b.kv = torch.nan_to_num(b.kv, 0, 0, 0)
    _check_seen(o, b, w, tokens={10, 11, 100, 127, 128, 255, 306, 307, 395})


# ------------------------------------------------------------------------------ magnitudes side by side

@pytest.mark.parametrize("v", [2.0 ** 20, 2.0 ** 30, 2.0 ** 60, 1e30, -1e30, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("H", [3, 300])
def test_expanded_a_large_row_that_only_later_queries_see(dsa, ix, v, H):
    b, w = Batch(110, [400, 150], [400, 150], H, dim=192), _weights(110, H)
    b.kv[200, 9] = v
    b.kv[210] = v
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_seen(o, b, w, tokens=set(range(0, 200, 7 if H == 3 else 67)) | {127, 128, 199} | set(range(400, 550, 49)))


@pytest.mark.parametrize("exp", [9, 16, 28, 40, 60, 100])
@pytest.mark.parametrize("n,nq,H", [(400, 130, 2), (2500, 100, 2), (400, 30, 300)])
def test_expanded_a_large_value_of_next_to_no_weight(dsa, ix, exp, n, nq, H):
    # channel 17 feeds the values alone, so row 150 has an ordinary key but a value 2^exp times the others'
    b, w = Batch(111, [n], [nq], H, dim=192), _weights(111, H)
    w[:, :128, 17] = 0
    b.kv[150, 17] = 2.0 ** exp
    b.q[:, :, 128:] = b.q[:, :, 128:].abs()
    b.kv[150, 512:] = -60.0                      # score near -200: weight below 2^-250
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_seen(o, b, w, tokens=set(range(0, nq, 13)))


@pytest.mark.parametrize("exp", [9, 16, 28, 40, 60])
def test_expanded_a_large_key_of_no_weight(dsa, ix, exp):
    b, w = Batch(112, [390], [140], 2, dim=192), _weights(112, 2)
    b.q[:, :, 128:] = b.q[:, :, 128:].abs()
    b.kv[260, 512:] = -2.0 ** exp
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_seen(o, b, w)


@pytest.mark.parametrize("step", [0.2, 1.0])
def test_expanded_every_value_larger_than_those_before(dsa, ix, step):
    # values grow by 2^step from row to row (2^-75 to 2^75 with the larger step), scores are
    # ordinary: a query's output is made of the rows just before it, all far below the tile's largest
    b, w = Batch(113, [150], [150], 2, dim=192), _weights(113, 2)
    w[:, :128] = 0
    b.kv[:, :512] = (b.kv[:, :512].float() * torch.exp2(step * (torch.arange(150.0) - 75))[:, None]).to(torch.bfloat16)
    if step == 1.0:
        b.kv[:10] = 0                            # and below 2^-60 a value may lose bits
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_seen(o, b, w, tokens=set(range(20 if step == 1.0 else 0, 150)))


def test_expanded_zero_values_beside_large_ones(dsa, ix):
    # the sum of the weights spans what lies between a tile of zero values and one of 2^110
    b, w = Batch(114, [384], [128], 2, dim=192), _weights(114, 2)
    w[:, :128] = 0                               # scores from the rope part alone
    b.kv[:256, :512] = 0
    b.kv[256:, :512] = (b.kv[256:, :512].float() * 2.0 ** 110).to(torch.bfloat16)
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK
    _check_seen(o, b, w)


# ------------------------------------------------------------------------------ light weights

@pytest.mark.parametrize("n", [4000, 60000])
@pytest.mark.parametrize("split", [False, True])
def test_4bit_many_light_tokens_beside_one_heavy(dsa, ix, n, split):
    # token 0 has score 18, the others 0: weights of 2^-26 of the heavy one, which together carry the
    # whole output (the heavy token's latent is zero)
    b = Batch(120, [n], [1], 16)
    b.q.zero_()
    b.q[:, :, 512] = 1.0
    b.kv[:, :512] = b.kv[:1, :512]
    b.kv[:, 512:] = 0
    b.kv[0, :512], b.kv[0, 512] = 0, 18.0
    kv4 = ix.quantize_latent_fp4(b.kv.to(DEV))
    val = f64(ix.dequantize_latent_fp4(kv4))
    qo, co = b.qo.to(DEV), b.co.to(DEV)
    idx = torch.arange(n, dtype=torch.int32, device=DEV)[None] if split else None
    o, lse = ix.latent_attention_fp4(b.q.to(DEV), kv4, b.pos.to(DEV), qo, co, 1.0, idx=idx)
    assert ix.device_error() == dsa.DSA_OK
    ref, lref, mag = oracle.latent_attention(f64(b.q), val, b.pos.numpy(), b.qo.numpy(), b.co.numpy(), 1.0)
    tol = 1.01 * U * np.abs(ref) + (1.05 * F + 2.0 ** -16) * (mag + np.abs(ref)) + n * 2.0 ** -32 * np.abs(val[1:, :512]).max(0)
    assert np.all(np.abs(f64(o) - ref) <= tol)
    assert np.all(np.abs(f64(lse) - lref) <= 1e-5)


# ------------------------------------------------------------------------------ rows that are not finite

@pytest.mark.parametrize("v", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("at", [(0, 0), (5, 17), (8, 511), (3, 300)])
def test_4bit_rows_report_what_is_not_finite(dsa, ix, v, at):
    g = torch.Generator().manual_seed(8)
    x = torch.randn((9, 576), generator=g).to(torch.bfloat16)
    want = ix.quantize_latent_fp4(x.to(DEV))
    assert ix.device_error() == dsa.DSA_OK
    x[at] = v
    got = ix.quantize_latent_fp4(x.to(DEV))
    assert ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS
    keep = [i for i in range(9) if i != at[0]]
    assert torch.equal(got[keep], want[keep])
    # the other blocks of the row are as they were
    blk = at[1] // 16
    codes = torch.ones(256, dtype=torch.bool)
    codes[8 * blk:8 * blk + 8] = False
    assert torch.equal(got[at[0], :256].cpu()[codes], want[at[0], :256].cpu()[codes])
    # a rope key is stored as it is, whatever it holds
    x = torch.randn((2, 576), generator=g).to(torch.bfloat16)
    x[1, 570] = v
    back = ix.dequantize_latent_fp4(ix.quantize_latent_fp4(x.to(DEV)))
    assert ix.device_error() == dsa.DSA_OK
    assert torch.equal(back[:, 512:].cpu().view(torch.int16), x[:, 512:].contiguous().view(torch.int16))


# ------------------------------------------------------------------------------ together

@pytest.mark.parametrize("n,nq,H", [(700, 300, 3), (400, 30, 300)])      # shares of steps; whole items
def test_expanded_slow_paths_on_two_streams_and_in_graphs(dsa, ix, n, nq, H):
    # a tile of own scales and a row to be computed again, at once on two streams, captured twice, and
    # replayed after the inputs lost both and got them back
    b, w = Batch(140, [n, 90], [nq, 20], H, dim=192), _weights(140, H)
    plain = b.kv.clone()
    b.kv[5, 300] = 2.0 ** 40
    b.kv[n - 3] = float("nan")
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    w, odd, plain = w.to(DEV), kv.clone(), plain.to(DEV)
    call = lambda **k: ix.latent_attention_expanded(q, kv, w, pos, qo, co, SCALE, **k)  # noqa: E731
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))  # noqa: E731
    want = call()
    kv.copy_(plain)
    ordinary = call()
    assert not bool(torch.isfinite(want).all()) and bool(torch.isfinite(ordinary).all())
    streams = [torch.cuda.Stream() for _ in range(2)]
    kv.copy_(odd)
    torch.cuda.synchronize()
    outs = [call(stream=s) for s in streams * 2]
    torch.cuda.synchronize()
    assert all(same(want, o) for o in outs)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = call()
        graphs.append((g, res))
    for k, (src, ref) in enumerate(((plain, ordinary), (odd, want), (odd, want), (plain, ordinary), (odd, want))):
        kv.copy_(src)
        g, res = graphs[k & 1]
        g.replay()
        torch.cuda.synchronize()
        assert same(res, ref)
    assert ix.device_error() == dsa.DSA_OK


def test_batches_of_nothing(dsa, ix):
    # queries that attend to nothing, tokens of no sequence only, sequences without rows, one idx row of -1s
    H = 5
    b, w = Batch(141, [50, 0], [4, 0], H), _weights(141, H).to(DEV)
    kv4 = ix.quantize_latent_fp4(b.kv.to(DEV))
    q, kv, co = b.dev("q", "kv", "co")
    qe = q[:, :, :192].contiguous()
    none = torch.full((4,), -1, dtype=torch.int32, device=DEV)
    all_in = torch.tensor([0, 4, 4], dtype=torch.int32, device=DEV)
    for qo in ([0, 4, 4], [0, 0, 0], [2, 2, 2], [4, 4, 4]):
        qo = torch.tensor(qo, dtype=torch.int32, device=DEV)
        kept = qo[0] == qo[2]
        for call in (lambda **k: ix.latent_attention(q, kv, none, qo, co, SCALE, **k),
                     lambda **k: ix.latent_attention_fp4(q, kv4, none, qo, co, SCALE, **k),
                     lambda **k: ix.latent_attention_fp4(q, kv4, None, qo, co, SCALE,
                                                         idx=torch.full((4, 130), -1, dtype=torch.int32, device=DEV), **k)):
            out = torch.full((4, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
            lse = torch.full((4, H), 7.0, device=DEV)
            call(out=out, lse=lse)
            assert bool((out == (7.0 if kept else 0.0)).all())
            assert bool((lse == 7.0).all() if kept else torch.isneginf(lse).all())
        out = torch.full((4, H, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        ix.latent_attention_expanded(qe, kv, w, none, qo, co, SCALE, out=out)
        assert bool((out == (7.0 if kept else 0.0)).all())
    # a query in a sequence without rows can only attend to nothing
    co0 = torch.tensor([0, 0, 50], dtype=torch.int64, device=DEV)
    out = ix.latent_attention_expanded(qe, kv, w, none, all_in, co0, SCALE)
    assert bool((out == 0).all()) and ix.device_error() == dsa.DSA_OK
    none[2] = 0
    out, lse = ix.latent_attention(q, kv, none, all_in, co0, SCALE)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    assert ix.device_error() == dsa.DSA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("n,nq,H", [(700, 200, 3), (400, 40, 300)])
def test_expanded_queries_that_see_nothing_of_a_tile_of_own_scales(dsa, ix, n, nq, H):
    # in one tile of queries some attend to nothing, some to the first rows only (with scores far below
    # zero), some to all; the tiles of tokens that only the last see carry scales of their own
    b, w = Batch(150, [n], [nq], H, dim=192), _weights(150, H)
    b.q[:, :, 128:] = b.q[:, :, 128:].abs()
    b.kv[:, 512:] = b.kv[:, 512:] * 0.125 - 60.0             # every score near -200
    b.kv[n - 150::37, 300] = 2.0 ** 30
    b.kv[3, 17] = 2.0 ** 12
    b.pos[::3] = -1
    b.pos[1::3] = torch.arange(len(b.pos[1::3])).int() % 140
    o = _expanded(ix, b, w)
    assert ix.device_error() == dsa.DSA_OK and np.all(o[::3] == 0)
    _check_seen(o, b, w, tokens=set(range(0, nq, 1 if H == 3 else 7)))


# ------------------------------------------------------------------------------ scores beyond fp32's fractions

def _winners(x, margin):
    """Rows whose largest score leads by so much that nothing but its token counts, and that token.
    x holds -inf where a row does not look.  The others weigh e^-40 each at most, in all less than
    1,000 * 4.3e-18 * 30 < 2e-13 of the output: LIGHT."""
    two = torch.topk(x, 2, dim=-1)
    lead = two.values[..., 0] - two.values[..., 1]
    return lead > margin * x.masked_fill(torch.isinf(x), 0).abs().amax(-1) + 40, two.indices[..., 0]


LIGHT = 2e-13


@pytest.mark.parametrize("exp", [6, 16, 20, 23, 25, 27, 30, 40, 80])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("n,nq,H", [(700, 200, 3), (400, 40, 300)])
def test_expanded_scores_up_to_2_to_the_80(dsa, ix, exp, spread, n, nq, H):
    # the heaviest token has all the weight, so out is its value whatever is lost of the score: the
    # value's rounding to fp16 (F, and 2^-31 of the value's largest), the weight's (F; its sum is not
    # rounded) and out's (U), and the fp32 sum of the value's 512 products, a walk of 6 sqrt(512) 2^-24 |w| |c|
    b, w = Batch(160 + exp, [n], [nq], H, dim=192), _weights(160, H)
    b.q = (b.q.float() * 2.0 ** exp).to(torch.bfloat16)
    if spread:
        b.kv[::50, :512] = b.kv[::50, :512] * 2.0 ** -12             # tiles of own scales
    o = torch.from_numpy(_expanded(ix, b, w))
    assert ix.device_error() == dsa.DSA_OK and bool(torch.isfinite(o).all())
    kv, q, wd = b.kv.double().to(DEV), b.q.double().to(DEV), w.double().to(DEV)
    late = torch.arange(n, device=DEV)[None] > b.pos.to(DEV)[:, None]
    for h in range(0, H, 1 if H == 3 else 23):
        up = kv[:, :512] @ wd[h].t()
        k, v = torch.cat((up[:, :128], kv[:, 512:]), 1), up[:, 128:]
        x = (SCALE * q[:, h] @ k.t()).masked_fill(late, -torch.inf)
        # fp16 keys move a score by up to F sum |q_d k_d|, far less than 2^-7 of the largest score
        sure, at = _winners(x, 2.0 ** -6)
        if exp >= 16:
            assert int(sure.sum()) > nq // 2
        ref = v[at][sure].cpu()
        tol = (1.01 * U + 2.02 * F) * ref.abs() + 2.0 ** -30 * ref.abs().amax(1, keepdim=True) + LIGHT
        walk = 6 * 512 ** 0.5 * 2.0 ** -24 * kv[at, :512].norm(dim=1)[:, None] * wd[h, 128:].norm(dim=1)[None]
        tol += walk[sure].cpu()
        assert bool(((o[:, h][sure.cpu()] - ref).abs() <= tol).all()), h


@pytest.mark.parametrize("exp", [6, 16, 20, 23, 25, 27, 30, 40, 80])
@pytest.mark.parametrize("fp4", [False, True])
def test_absorbed_scores_up_to_2_to_the_80(dsa, ix, exp, fp4):
    # out is the heaviest token's latent: allowed is one rounding of the weight's type and of out
    b = Batch(170 + exp, [900, 300], [40, 3], 24)
    b.q = (b.q.float() * 2.0 ** exp).to(torch.bfloat16)
    q, kv, pos, qo, co = b.dev("q", "kv", "pos", "qo", "co")
    if fp4:
        kv4 = ix.quantize_latent_fp4(kv)
        kv = ix.dequantize_latent_fp4(kv4)
        o, lse = ix.latent_attention_fp4(q, kv4, pos, qo, co, SCALE)
    else:
        o, lse = ix.latent_attention(q, kv, pos, qo, co, SCALE)
    assert ix.device_error() == dsa.DSA_OK and bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    for t in range(43):
        r0 = 0 if t < 40 else 900
        rows = kv[r0:r0 + int(pos[t]) + 1].double()
        x = SCALE * q[t].double() @ rows.t()
        sure, at = _winners(x, 2.0 ** -10)
        ref = rows[at][sure, :512]
        wt = F if fp4 else U
        assert bool(((o[t][sure].double() - ref).abs() <= (1.01 * U + 1.01 * wt) * ref.abs() + LIGHT).all()), t
        assert bool(((lse[t].double() - x.amax(1)).abs() <= 2.0 ** -18 * x.abs().amax(1) + 10).all()), t
