"""The test suite's own hook, on the host: no test whose call would be launched
on made-up addresses runs where a GPU is visible.
"""
import conftest
import torch


class Item:
    def __init__(self, nodeid):
        self.nodeid, self.keywords, self.marks = nodeid, {}, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def test_accepted_calls_do_not_run_beside_a_gpu(monkeypatch):
    for gpu, marks in ((True, ["skip"]), (False, [])):
        monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
        items = [Item("tests/test_ops_abi.py::test_attn_range_of_scale[2e-30-None]"),
                 Item("tests/test_ops_abi.py::test_attn_range_of_scale[1e-38-1]")]
        conftest.pytest_collection_modifyitems(None, items)
        assert items[0].marks == marks and items[1].marks == []
