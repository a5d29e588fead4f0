"""Host side of the latent-cache operators.  CPU only."""

import numpy as np
import pytest
import torch

import oracle
from dsa_lightning_indexer_03_b200.indexer import Indexer


class _Stream:
    """What the binding looks at of a stream."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)
        self.cuda_stream = 0


def test_a_stream_of_another_device_is_refused():
    ix = object.__new__(Indexer)
    ix.device = torch.device("cuda", 1)
    for index in (0, 2):
        with pytest.raises(ValueError, match="stream must be on cuda:1"):
            ix._on(_Stream(index))


def test_the_hash_of_the_traffic_figures_covers_the_entry_points(tmp_path, monkeypatch):
    # tensor maps, launch arguments and the choice of a path are in the entry points' files: a change
    # there asks for new figures; the latent-cache operators and comments do not
    import shutil

    from dsa_lightning_indexer_03_b200 import build
    monkeypatch.setattr(build, "CSRC", shutil.copytree(build.CSRC, tmp_path / "csrc"))
    base = build.source_hash()
    for name in build.SOURCES + build.HEADERS:
        f = tmp_path / "csrc" / name
        text = f.read_text()
        f.write_text(text + "\n// a comment\n")
        assert build.source_hash() == base, name
        f.write_text(text + "\nint a_change;\n")
        assert (build.source_hash() == base) == name.startswith("latent"), name
        f.write_text(text)


def test_the_oracles_expanded_form_without_rounding_is_the_absorbed_form():
    # any weights: (W_uk^T q) . c = q . (W_uk c), and W_uv (sum w c) = sum w (W_uv c)
    r = np.random.default_rng(2)
    H, n = 3, 40
    W, kv, q = r.standard_normal((H, 256, 512)) / 20, r.standard_normal((n, 576)), r.standard_normal((4, H, 192))
    pos, qo, co = np.array([39, 0, 17, -1]), np.array([0, 4]), np.array([0, n])
    o, mag = oracle.latent_attention_expanded(q, kv, W, pos, qo, co, 0.1, rounded=False)
    qa = np.concatenate((np.einsum("thd,hdc->thc", q[:, :, :128], W[:, :128]), q[:, :, 128:]), axis=2)
    oa, _, _ = oracle.latent_attention(qa, kv, pos, qo, co, 0.1)
    np.testing.assert_allclose(o, np.einsum("thc,hdc->thd", oa, W[:, 128:]), rtol=0, atol=1e-11)
    assert np.all(mag >= np.abs(o) - 1e-12)
    # and the rounded form is within a few steps of bf16 of it
    assert np.abs(oracle.latent_attention_expanded(q, kv, W, pos, qo, co, 0.1)[0] - o).max() < 0.05
