"""Refusals of the single operators' binding that need no GPU."""
import pytest

torch = pytest.importorskip("torch")


class Stream:
    def __init__(self, device):
        self.device, self.cuda_stream = torch.device(device), 0x5EED0


def test_stream_of_another_device():
    """A launch goes to the stream's device and its outputs to the tensors' one, so
    the two have to be the same."""
    from padding_free_pair_amd._single import _on
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        _on(torch, torch.device("cuda", 0), Stream("cuda:1"))
