"""The SSD layer's serving operators on the CPU: how packed sequences are cut, and what the binding decides before a launch."""
import pytest
import torch

import selective_state_space_55_amd as mscan


def test_ssd_a_long_sequence_among_short_ones_is_cut_without_a_hint():
    f = mscan.ssd_fwd_varlen_workspace_size
    shape = (64, 64, 128)   # 32 workgroups a piece
    # one of 58000, 50000 or 30000 tokens may be among these; the mean, two to four pieces, does not tell
    for nseq, total in ((20, 60000), (28, 60000), (16, 32768), (16, 65536), (20, 12000), (16, 4096)):
        assert f(nseq, total, *shape) > 0, (nseq, total)
    # with the longest sequence known, those that fill the GPU by themselves stay whole up to four pieces
    assert f(16, 4096, *shape, 1, 256) == 0 and f(20, 60000, *shape, 1, 4096) == 0
    assert f(20, 60000, *shape, 1, 58000) > 0


class OnDeviceOne(torch.Tensor):
    """Stands for a tensor on the second GPU."""
    is_cuda = True

    def get_device(self):
        return 1


def test_entry_points_launch_on_the_device_of_their_first_parameter(monkeypatch):
    """Whether it is passed by place, by name, or after other names."""
    entered = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *exc):
            entered.append(-1)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)

    @mscan._entry
    def call(x, weight=None, *, eps=0.0, stream=None):
        return list(entered)

    x, host = torch.zeros(2).as_subclass(OnDeviceOne), torch.zeros(2)
    for run in (lambda: call(x, host), lambda: call(x=x, weight=host), lambda: call(eps=1e-5, x=x), lambda: call(weight=host, x=x, eps=1.0)):
        entered.clear()
        assert run() == [1] and entered == [1, -1]
    entered.clear()
    assert call(host, x) == []


def test_a_workspace_of_another_device_is_refused():
    cuda = torch.device("cuda", 0)
    with pytest.raises(ValueError):
        mscan._scratch(100, torch.empty(1000, dtype=torch.uint8), cuda)   # host memory
    with pytest.raises(ValueError):
        mscan._scratch(100, torch.empty(2000, dtype=torch.uint8)[::2], torch.device("cpu"))
    ws = torch.empty(1000, dtype=torch.uint8)
    kept, at, size = mscan._scratch(100, ws, torch.device("cpu"))
    assert kept is ws and at % 256 == 0 and at + size == ws.data_ptr() + 1000
