"""Which tests run where (no GPU needed)."""
import types

import pytest
import torch

import conftest
import test_abi_host
import test_kvcache_host
import test_packed_host


class Item:
    def __init__(self, module, *keywords):
        self.module, self.keywords, self.marks = module, keywords, []

    def add_marker(self, mark):
        self.marks.append(mark)


def skipped(module, *keywords):
    item = Item(module, *keywords)
    conftest.pytest_collection_modifyitems(None, [item])
    return [m.name for m in item.marks] == ["skip"]


@pytest.mark.parametrize("gpu", (False, True))
def test_calls_with_addresses_of_no_memory_stay_off_a_gpu(monkeypatch, gpu):
    """Some of them pass every check of arguments, and would be launched where there is a GPU."""
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    for module in (test_abi_host, test_kvcache_host, test_packed_host):
        assert skipped(module) == gpu
    other = types.ModuleType("other")
    assert not skipped(other)
    assert skipped(other, "gpu") == (not gpu)
