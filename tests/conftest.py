import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
    config.addinivalue_line("markers", "slow: takes more than ~20 s on the CPU")


# Host tests whose accepted calls end where they ask for a GPU: with one present
# they would run on made-up addresses.
ENDS_WITHOUT_A_GPU = ("test_block_host.py::test_columns_of_one_matrix_do_not_overlap",)


def pytest_collection_modifyitems(config, items):
    import pytest
    import torch

    for item in items:
        if item.nodeid.endswith(ENDS_WITHOUT_A_GPU):
            item.add_marker(pytest.mark.skipif(torch.cuda.device_count() > 0, reason="its calls would run"))
