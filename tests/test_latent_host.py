"""Host side of the latent-cache operators.  CPU only."""

import pytest
import torch

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
