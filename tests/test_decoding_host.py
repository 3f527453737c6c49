"""Host side of the decoding-step calls, without a GPU: which device results are made on."""

import pytest
import torch

from test_abi import pa  # noqa: F401  (builds and loads the library)


@pytest.mark.parametrize("asked,made_on", [(None, "cuda"), (0, 0), (1, 1), ("cpu", "cpu"), ("cuda:0", "cuda:0"),
                                           (torch.device("cuda", 0), torch.device("cuda", 0))])
def test_frequencies_are_made_on_the_device_that_is_asked_for(pa, monkeypatch, asked, made_on):  # noqa: F811
    """Device 0 is device 0, whichever is current; only None is the current one."""
    seen, tensor = [], torch.tensor
    monkeypatch.setattr(torch, "tensor", lambda data, dtype, device: (seen.append(device), tensor(data, dtype=dtype))[1])
    freq, attn = pa.pa_rotary_frequencies(8, device=asked)
    assert seen == [made_on] and type(seen[0]) is type(made_on)
    assert freq.shape == (4,) and attn == 1.0


@pytest.mark.parametrize("asked,made_on", [(None, "cuda"), (0, 0), (1, 1), ("cpu", "cpu")])
def test_workspaces_are_made_on_the_device_that_is_asked_for(pa, monkeypatch, asked, made_on):  # noqa: F811
    seen, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (seen.append(device), empty(n, dtype=dtype))[1])
    assert pa.workspace_tensor(512, asked).numel() == 512
    assert seen == [made_on] and type(seen[0]) is type(made_on)
