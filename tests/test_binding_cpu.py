"""The binding's argument helpers, without a GPU: which stream a call without one
takes, and what passes as an address."""
import pytest
import torch

import gemm_epilogues_mlp_amd as sw


@pytest.fixture
def initialised(monkeypatch):
    """torch as it is once the device is set up, current stream 1234 of device 3."""
    monkeypatch.setattr(torch.cuda, "_initialized", True)
    monkeypatch.setattr(torch.cuda, "_is_in_bad_fork", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1231 + device,
                        raising=False)


def test_stream_is_torchs_current_one(initialised):
    assert sw._stream(None) == 1234
    assert sw._stream(77) == 77 and sw._stream(0) == 0


def test_forked_child_is_refused(initialised, monkeypatch):
    """A child forked after the device was set up must not launch on the parent's streams:
    torch's own error, also where the parent has made calls before."""
    assert sw._stream(None) == 1234
    monkeypatch.setattr(torch.cuda, "_is_in_bad_fork", lambda: True)
    with pytest.raises(RuntimeError, match="forked subprocess"):
        sw._stream(None)


def test_torch_without_the_raw_handle(initialised, monkeypatch):
    """A torch build that lacks the raw handle's private name: the public stream serves."""
    class Stream:
        cuda_stream = 4321
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    assert sw._stream(None) == 4321


def test_an_address_is_taken_as_it_is():
    """Addresses are told apart by type, before anything is asked of them (an exception a
    pointer made calls with plain addresses 0.3 us slower for each)."""
    class Address(int):
        def __getattr__(self, name):
            pytest.fail(f"asked for {name}")
    assert sw._ptr(Address(4096)) == 4096 and sw._ptr(0) == 0 and sw._ptr(None) is None
    t = torch.zeros(4)
    assert sw._ptr(t) == t.data_ptr()
    with pytest.raises(AttributeError):
        sw._ptr("4096")
