"""What the collection hook skips: tests marked gpu without a device, and with one the host tests that would launch a
kernel on made-up addresses."""
import pytest
import torch

from tests import conftest


class Item:
    def __init__(self, name, *keywords):
        self.name, self.keywords, self.skipped = name, keywords, False

    def add_marker(self, mark):
        self.skipped = self.skipped or mark.name == "skip"


@pytest.mark.parametrize("device", [False, True])
def test_collection_skips(monkeypatch, device):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: device)
    made_up = Item("test_rope_refuses_tensors_of_a_call_that_share_elements")
    host, gpu = Item("test_rope_rejects_bad_arguments"), Item("test_rope", "gpu")
    conftest.pytest_collection_modifyitems(None, [made_up, host, gpu])
    assert made_up.skipped == device and gpu.skipped != device and not host.skipped


def test_the_skipped_host_tests_exist():
    import tests.test_paged_host as host
    for name in conftest.ONLY_WITHOUT_A_DEVICE:
        assert callable(getattr(host, name))
