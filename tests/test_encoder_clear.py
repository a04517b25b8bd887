"""Which inputs EncoderStates.clear empties, on the device and in the host's lengths. On the CPU."""
import numpy as np
import pytest
import torch

import sparse_long_context_sfi_gb300.engine as engine


@pytest.mark.parametrize("which", [[0], [2, 0], [1, 1], [1, 1, 1], [2, 2, 0], [0, 1, 2], [2, 1, 0, 1], [], None,
                                   np.array([1, 1, 1]), range(2)])
def test_only_the_named_inputs(monkeypatch, which):
    """The same input may be named more than once; the others keep their states."""
    monkeypatch.setattr(engine, "_torch_stream", lambda stream: None)
    monkeypatch.setattr(engine, "_capturing", lambda stream: False)
    e = engine.EncoderStates(1, 3, 4, 2, 32, device="cpu")
    e.lens[:] = [5, 6, 7]
    e.seq_len.copy_(torch.tensor([5, 6, 7]))
    e.clear(which)
    gone = range(3) if which is None else which
    want = [0 if i in gone else 5 + i for i in range(3)]
    assert e.seq_len.tolist() == want and e.lens.tolist() == want
