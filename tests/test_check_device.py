"""CPU test: check(stream) reads the error record of the stream's own device (the
calls on packed prompts and slots run on their tensors' device, whichever is
current), with a fake of the library and of torch's device switch."""
import contextlib
import types

import pytest
import torch

import selective_state_space_selscan_b200 as ss


@pytest.fixture
def machine(monkeypatch):
    """Two devices; the record of device 1 holds a refused index."""
    m = types.SimpleNamespace(current=0, record={0: 0, 1: ss.STATUS_CODE["SELSCAN_ERR_INDEX"]},
                              asked=[])

    @contextlib.contextmanager
    def device(d):
        before, m.current = m.current, d.index
        try:
            yield
        finally:
            m.current = before

    def selscan_check(handle):
        m.asked.append((m.current, handle.value))
        err, m.record[m.current] = m.record[m.current], 0
        return err

    real = ss.lib()
    fake = types.SimpleNamespace(selscan_check=selscan_check, selscan_strerror=real.selscan_strerror)
    monkeypatch.setattr(ss, "lib", lambda: fake)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=10 + m.current))
    return m


def test_check_reads_the_record_of_the_streams_device(machine):
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77)
    ss.check()  # nothing on the current device
    with pytest.raises(ss.SelscanError, match="SELSCAN_ERR_INDEX"):
        ss.check(stream)
    ss.check(stream)  # read once
    assert machine.asked == [(0, 10), (1, 77), (1, 77)] and machine.current == 0
