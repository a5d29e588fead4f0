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
