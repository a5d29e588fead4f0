"""Latent-cache operators at the sizes they are meant for, on sampled rows: prefixes of 131,072 tokens
whose pieces many thread blocks share, a prompt chunk after thousands of tokens, a prompt's
selections, and an 8,192-token prompt of 96 heads in the expanded form.  The reference is the
definition in 64 bits on the GPU, over the rows that a sampled query attends to.

Tolerances are those of test_gpu_latent.py (absorbed; weights as bf16, U = 2^-8) and of
test_gpu_latent_extremes.py (fp16 weights, F = 2^-11).  Over 131,072 tokens the fp32 sum of weights
walks further: six sigma of sqrt(n) roundings of 2^-24 are 6 * 362 * 2^-24 = 2^-13, relative to itself
and, for out, to mag = sum_s w_s |v_s|; a warp's partial sums make it far less."""

import math

import pytest
import torch

import workloads as W
from test_gpu_latent import DEV, SCALE, U

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


def _rand(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return g, lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _attend(q, k, v, scale):
    """q [H, D], k [n, D], v [n, E], all fp64: out, lse, mag and the score allowance per head."""
    x = scale * q @ k.t()
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x - lse[:, None])
    e = 6 * math.sqrt(k.shape[1]) * 2.0 ** -24 * scale * q.norm(dim=1) * k.norm(dim=1).max()
    e = e + 4 * 2.0 ** -24 * x.abs().amax(1) + 2.0 ** -20
    return w @ v, lse, w @ v.abs(), e, w


def _check_absorbed(o, lse, q, rows, fp16, scale=SCALE):
    n = rows.shape[0]
    ref, lref, mag, e, _ = _attend(q.double(), rows.double(), rows[:, :512].double(), scale)
    walk = 6 * math.sqrt(n) * 2.0 ** -24
    wt = 1.05 * F if fp16 else 1.01 * U
    tol = 1.01 * U * ref.abs() + (wt + walk + 2 * e[:, None]) * (mag + ref.abs()) + 1e-6
    if fp16:
        tol += n * 2.0 ** -32 * rows[:, :512].abs().max().double()
    assert bool(((o.double() - ref).abs() <= tol).all())
    assert bool(((lse.double() - lref).abs() <= e + walk + 2.0 ** -22 * (lref.abs() + 8) + 1e-6).all())


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("q_std", [1.0, 5.0])
def test_decode_over_131072_tokens(dsa, ix, fp4, q_std):
    lens, H = [131072, 70001, 3], 96
    g, r = _rand(1)
    kv, q = r(sum(lens), 576), (r(3, H, 576).float() * q_std).to(torch.bfloat16)
    co = [0, lens[0], lens[0] + lens[1], sum(lens)]
    pos = [n - 1 for n in lens]
    args = (_ints(pos), _ints([0, 1, 2, 3]), _ints(co, torch.int64), SCALE)
    if fp4:
        kv4 = ix.quantize_latent_fp4(kv)
        kv = ix.dequantize_latent_fp4(kv4)
        o, lse = ix.latent_attention_fp4(q, kv4, *args)
    else:
        o, lse = ix.latent_attention(q, kv, *args)
    assert ix.device_error() == dsa.DSA_OK
    for t in range(3):
        _check_absorbed(o[t], lse[t], q[t], kv[co[t]:co[t + 1]], fp4)


@pytest.mark.parametrize("fp4", [False, True])
def test_a_chunk_of_300_queries_after_6000_tokens(dsa, ix, fp4):
    n, nq, H = 6301, 301, 96
    g, r = _rand(2)
    kv, q = r(n, 576), r(nq, H, 576)
    args = (torch.arange(n - nq, n, dtype=torch.int32, device=DEV), _ints([0, nq]), _ints([0, n], torch.int64), SCALE)
    if fp4:
        kv4 = ix.quantize_latent_fp4(kv)
        kv = ix.dequantize_latent_fp4(kv4)
        o, lse = ix.latent_attention_fp4(q, kv4, *args)
    else:
        o, lse = ix.latent_attention(q, kv, *args)
    assert ix.device_error() == dsa.DSA_OK
    for t in (*range(0, nq, 23), nq - 1):
        _check_absorbed(o[t], lse[t], q[t], kv[:n - nq + t + 1], fp4)


def test_a_prompts_selections_over_the_4bit_cache(dsa, ix):
    # 1,200 queries of one prompt, each over 2,048 (or all, if fewer) selected positions
    n, H, k = 5000, 96, 2048
    T = 1200
    g, r = _rand(3)
    kv4 = ix.quantize_latent_fp4(r(n, 576))
    kv, q = ix.dequantize_latent_fp4(kv4), r(T, H, 576)
    pos = torch.arange(T, device=DEV) * 4 + 3
    idx = torch.rand((T, n), generator=g, device=DEV).masked_fill_(torch.arange(n, device=DEV)[None] > pos[:, None], 2.0).argsort(1)[:, :k].int()
    idx = torch.where(torch.arange(k, device=DEV)[None] <= pos[:, None], idx, -1).contiguous()
    o, lse = ix.latent_attention_fp4(q, kv4, None, _ints([0, T]), _ints([0, n], torch.int64), SCALE, idx=idx)
    assert ix.device_error() == dsa.DSA_OK
    for t in (*range(0, T, 61), T - 1):
        sel = idx[t][idx[t] >= 0].long()
        assert int(sel.max()) <= int(pos[t]) and sel.numel() == min(k, int(pos[t]) + 1)
        _check_absorbed(o[t], lse[t], q[t], kv[sel], True)


@pytest.mark.parametrize("n,nq,H", [(8192, 8192, 96), (20001, 1000, 16)])     # whole items; shares of steps
def test_expanded_prompts(dsa, ix, n, nq, H):
    g, r = _rand(4)
    kv, q = r(n, 576), r(nq, H, 192)
    w = (r(H, 256, 512).float() * 512 ** -0.5).to(torch.bfloat16)
    o = ix.latent_attention_expanded(q, kv, w, torch.arange(n - nq, n, dtype=torch.int32, device=DEV), _ints([0, nq]),
                                     _ints([0, n], torch.int64), SCALE)
    assert ix.device_error() == dsa.DSA_OK
    c = kv.double()
    for h in (*range(0, H, 7), H - 1):
        up = c[:, :512] @ w[h].double().t()
        k, v = torch.cat((up[:, :128], c[:, 512:]), 1), up[:, 128:]
        for t in (0, 1, 127, 128, *range(255, nq, 777), nq - 1):
            m = n - nq + t + 1
            ref, _, mag, e, wt = _attend(q[t, h][None].double(), k[:m], v[:m], SCALE)
            kabs, vmax = k[:m].abs(), v[:m].abs().amax(1)
            e = e + SCALE * (kabs @ q[t, h].abs().double() * F + 2.0 ** -31 * kabs.amax(1) * q[t, h].abs().sum().double()).max()
            tol = 1.01 * U * ref.abs() + (2.1 * F + 2 * torch.expm1(e)[:, None]) * (mag + ref.abs())
            tol += m * 2.0 ** -22 * (wt[0] * vmax).max() + 2.0 ** -30 * (wt[0] * vmax).sum()
            assert bool(((o[t, h].double() - ref[0]).abs() <= tol[0]).all()), (t, h)
