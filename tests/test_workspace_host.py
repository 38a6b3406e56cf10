"""The binding's workspace as it grows: what is asked for, kept and given back
(no GPU needed: the allocations are stand-ins)."""

import pytest
import torch

from long_context_causal_gqa_gb300 import binding


class Buffer:
    def __init__(self, n, device):
        self.n, self.device = n, torch.device(device)

    def numel(self):
        return self.n

    def data_ptr(self):
        return 4096


class Memory:
    """A device with `free` bytes."""

    def __init__(self, free):
        self.free, self.registered, self.status, self.asked = free, [], binding.GQA_OK, []

    def empty(self, n, dtype, device):
        assert dtype is torch.uint8
        self.asked.append(n)
        if n > self.free:
            raise torch.cuda.OutOfMemoryError("out of memory")
        return Buffer(n, device)

    def gqa_set_workspace(self, idx, ptr, n):
        self.registered.append((idx, n))
        return self.status

    @staticmethod
    def gqa_status_string(status):
        return b"status"


@pytest.fixture
def memory(monkeypatch):
    m = Memory(1 << 40)
    monkeypatch.setattr(binding, "load", lambda: m)
    monkeypatch.setattr(binding, "_ws", {})
    monkeypatch.setattr(binding, "_outgrown", [])
    monkeypatch.setattr(torch, "empty", m.empty)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda idx=None: None)
    return m


def test_grows_by_half_and_keeps_the_old(memory):
    a = binding.ensure_workspace(10000, 0)
    assert a.numel() == 10000 and binding.ensure_workspace(9000, 0) is a
    b = binding.ensure_workspace(10001, 0)
    assert b.numel() == 15000 and binding._outgrown == [a]
    c = binding.ensure_workspace(40000, 0)
    assert c.numel() == 40000 and binding._outgrown == [a, b]
    assert memory.registered == [(0, 10000), (0, 15000), (0, 40000)]


def test_takes_what_is_needed_where_more_does_not_fit(memory):
    a = binding.ensure_workspace(10000, 0)
    memory.free = 12000
    b = binding.ensure_workspace(11000, 0)
    assert b.numel() == 11000 and binding._outgrown == [a]
    assert memory.registered[-1] == (0, 11000)


def test_a_workspace_that_cannot_be_replaced_stays(memory):
    a = binding.ensure_workspace(10000, 0)
    memory.free = 10500
    with pytest.raises(torch.cuda.OutOfMemoryError):
        binding.ensure_workspace(11000, 0)
    memory.free = 1 << 40
    memory.status = binding.GQA_ERR_CUDA
    with pytest.raises(binding.GQAError):
        binding.ensure_workspace(11000, 0)
    assert binding._ws == {0: a} and binding._outgrown == []
    memory.asked.clear()
    assert binding.ensure_workspace(10000, 0) is a and memory.asked == []


def test_outgrown_workspaces_are_given_back(memory):
    a = binding.ensure_workspace(10000, 0)
    binding.ensure_workspace(20000, 0)
    d = binding.ensure_workspace(5000, 1)
    binding.ensure_workspace(6000, 1)
    assert binding._outgrown == [a, d]
    assert binding.release_outgrown(0) == 10000 and binding._outgrown == [d]
    assert binding.release_outgrown(0) == 0
    assert binding.release_outgrown("cuda:1") == 5000
    assert binding._outgrown == [] and set(binding._ws) == {0, 1}
