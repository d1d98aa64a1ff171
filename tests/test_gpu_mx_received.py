"""Packing by a dispatch's splits where the buffers hold no rows at all."""
import pytest
import torch

pytestmark = pytest.mark.gpu

a2av = pytest.importorskip("variable_size_all_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a2av.build()


def test_splits_are_checked_without_any_rows():
    x = [torch.empty(0, 64, device="cuda") for _ in range(2)]
    rows = [torch.empty(0, a2av.mx_row_bytes(64, "mxfp8"), dtype=torch.uint8, device="cuda") for _ in range(2)]
    splits = torch.zeros(2, 2, dtype=torch.int64, device="cuda")
    with a2av.A2av(2) as eng:
        calls = [lambda: eng.quantise(x, rows, "mxfp8", in_splits=splits),
                 lambda: eng.dequantise(rows, x, "mxfp8", in_splits=splits)]
        for call in calls:
            for value, want in ((0, a2av.OK), (1, a2av.ERR_BAD_SPLITS), (-1, a2av.ERR_BAD_SPLITS),
                                (0, a2av.OK)):
                splits[1, 0] = value
                call()
                assert eng.status() == want
