"""The latent oracle against torch's attention, loops and torch's e4m3 conversion, and the
entry points' refusals that need no GPU.  CPU only."""

import ctypes

import numpy as np
import pytest
import torch

import oracle


def _inputs(seed, lens, nq, H, dim=576):
    r = np.random.default_rng(seed)
    q = oracle.bf16_round(r.standard_normal((sum(nq), H, dim)))
    kv = oracle.bf16_round(r.standard_normal((sum(lens), 576)))
    qo, co = np.concatenate(([0], np.cumsum(nq))), np.concatenate(([0], np.cumsum(lens)))
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, nq)])
    return q, kv, pos, qo, co


def test_dense_absorbed_equals_torch_attention():
    q, kv, pos, qo, co = _inputs(1, [9, 30], [3, 2], 4)
    o, lse, _ = oracle.latent_attention(q, kv, pos, qo, co, 0.1)
    for t in range(5):
        b = 0 if t < 3 else 1
        rows = torch.from_numpy(kv[co[b]:co[b] + pos[t] + 1])
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[t])[:, None], rows[None].expand(4, -1, -1), rows[None, :, :512].expand(4, -1, -1), scale=0.1)
        np.testing.assert_allclose(o[t], want[:, 0].numpy(), rtol=0, atol=1e-12)
        np.testing.assert_allclose(lse[t], torch.logsumexp(0.1 * torch.from_numpy(q[t]) @ rows.T, 1).numpy(), atol=1e-12)


def test_a_selection_of_the_whole_prefix_is_the_dense_form():
    q, kv, pos, qo, co = _inputs(2, [12, 7], [2, 2], 3)
    idx = np.full((4, 12), -1)
    for t in range(4):
        idx[t, :pos[t] + 1] = np.random.default_rng(t).permutation(pos[t] + 1)
    for a, b in zip(oracle.latent_attention(q, kv, pos, qo, co, 0.2),
                    oracle.latent_attention(q, kv, pos, qo, co, 0.2, idx=idx)):
        np.testing.assert_allclose(a, b, rtol=0, atol=1e-12)


def test_expanded_equals_absorbed_without_the_rounding_of_keys_and_values():
    # powers of two in the weights, one latent value per up-projected row: bf16 rounding is exact
    r = np.random.default_rng(3)
    H = 2
    W = np.zeros((H, 256, 512))
    for h in range(H):
        for d in range(256):
            W[h, d, r.integers(512)] = 2.0 ** r.integers(-2, 2)
    q, kv, pos, qo, co = _inputs(4, [11], [4], H, dim=192)
    o, _ = oracle.latent_attention_expanded(q, kv, W, pos, qo, co, 0.3)
    qa = np.concatenate((np.einsum("thd,hdc->thc", q[:, :, :128], W[:, :128]), q[:, :, 128:]), axis=2)
    oa, _, _ = oracle.latent_attention(qa, kv, pos, qo, co, 0.3)
    np.testing.assert_allclose(o, np.einsum("thc,hdc->thd", oa, W[:, 128:]), rtol=0, atol=1e-12)


def test_empty_queries_and_tokens_of_no_sequence():
    q, kv, pos, _, co = _inputs(5, [6], [4], 2)
    pos = np.array([-1, 3, -1, 5])
    o, lse, _ = oracle.latent_attention(q, kv, pos, np.array([0, 3]), co, 0.3)
    assert np.all(o[0] == 0) and np.all(np.isneginf(lse[0])) and np.all(np.isnan(o[3]))


def test_fp4_codes_are_the_nearest_and_ties_go_to_even():
    x = np.zeros((1, 576))
    x[0, :16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.3, -2.4, 0, 5.5, -6]
    s, c, v = oracle.quantize_latent_fp4(x)
    assert s[0, 0] == 1.0
    np.testing.assert_array_equal(v[0, :16], [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4, 0.5, -2, 0, 6, -6])
    assert np.all(v[0, 16:512] == 0) and np.all(c[0, 16:] == 0)


def test_fp4_scale_is_torchs_e4m3_and_values_are_exact_in_bf16():
    r = np.random.default_rng(6)
    x = oracle.bf16_round(r.standard_normal((3, 576)) * 10.0 ** r.integers(-6, 5, (3, 1)))
    s, c, v = oracle.quantize_latent_fp4(x)
    amax = np.abs(x[:, :512].reshape(3, 32, 16)).max(2)
    want = torch.from_numpy(np.minimum(amax / 6, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(s, want)
    np.testing.assert_array_equal(oracle.bf16_round(v), v)
    # half a step of the grid (at most 1 between 4 and 6) times the scale, where it does not
    # saturate: the scale is off by at most 2^-4 of amax / 6 (subnormal: 2^-10)
    err = np.abs(v - x)[:, :512].reshape(3, 32, 16).max(2)
    assert np.all(err <= np.where(amax < 448 * 6, np.maximum(s, 6 * (amax / 6 - s)) + 1e-12, np.inf))
    np.testing.assert_array_equal(v[:, 512:], x[:, 512:])


@pytest.fixture(scope="module")
def lib():
    from dsa_lightning_indexer_03_b200 import _lib, build
    return _lib.load(build.build())


def test_refusals_without_a_handle(lib):
    p = ctypes.c_void_p(0x1000)
    assert lib.dsa_indexer_latent_attention_workspace(None, 1, 1, 96) == -1
    assert lib.dsa_indexer_latent_expanded_workspace(None, 1, 1, 96, 1) == -1
    assert lib.dsa_indexer_latent_attention(None, 1, p, 96, p, 1, p, p, 1, p, 0.1, p, p, p, 1 << 30, None) == 1
    assert lib.dsa_indexer_latent_attention_fp4(None, 1, p, 96, p, 1, p, p, 1, p, None, -1, 0.1, p, p, p, 1 << 30, None) == 1
    assert lib.dsa_indexer_quantize_latent_fp4(None, 1, p, None, p, 1, None) == 1
    assert lib.dsa_indexer_dequantize_latent_fp4(None, 1, p, 1, None, p, None) == 1
    assert lib.dsa_indexer_latent_attention_expanded(None, 1, p, 96, p, 1, p, p, p, 1, p, 0.1, p, p, 1 << 30, None) == 1
