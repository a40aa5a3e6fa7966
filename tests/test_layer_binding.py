"""The binding of include/csa2_layer.h without a GPU: what layer.py hands to the library. Host tensors stand in for
device ones (their device number, -1, is taken for the current one), and a library that only records its calls for the real
one; calls that the real one has to refuse go to it (it refuses them before anything is launched)."""
import pytest
import torch

import compressed_sparse_attention_append_b200 as csa
from compressed_sparse_attention_append_b200 import layer

INVALID = csa.CSA2_ERR_INVALID_ARG


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def host(monkeypatch):
    """layer.py on host tensors, into a recorder."""
    rec = Recorder()
    monkeypatch.setattr(layer, "_device", lambda: -1)
    monkeypatch.setattr(layer, "_fast", None)
    monkeypatch.setattr(layer, "_lib", rec)
    return rec


def _product(m, n, k=128):
    e4m3 = lambda rows: torch.zeros(rows, k, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return e4m3(m), torch.zeros(1, m), e4m3(n), torch.zeros(-(-n // 128), 1)


OUTPUTS = [  # (m, n, output, its row stride as the library has to get it)
    (4, 8, lambda: torch.empty(4, 8), 8),
    (4, 8, lambda: torch.empty(4, 20)[:, 3:11], 20),
    (4, 8, lambda: torch.empty(1, 8).expand(4, 8), 0),                # one row of storage
    (4, 8, lambda: torch.empty(11).as_strided((4, 8), (1, 1)), 1),    # overlapping rows
    (4, 1, lambda: torch.empty(1, 1).expand(4, 1), 0),
    (4, 1, lambda: torch.empty(4, 6)[:, :1], 6),
    (1, 8, lambda: torch.empty(8).as_strided((1, 8), (3, 1)), 8),     # a single row: its stride means nothing
    (0, 8, lambda: torch.empty(0, 8), 8),
]


@pytest.mark.parametrize("m,n,out,stride", OUTPUTS)
def test_a_product_gets_its_outputs_own_row_stride(host, m, n, out, stride):
    csa.csa2_fp8_gemm(*_product(m, n), out(), stream=0)
    (name, a), = host.calls
    assert name == "csa2_fp8_gemm" and a[:3] == (m, n, 128) and a[9] == stride


@pytest.mark.parametrize("m,n,out,stride", [c for c in OUTPUTS if c[3] < c[1]])
def test_a_product_into_overlapping_rows_is_refused(host, monkeypatch, m, n, out, stride):
    monkeypatch.setattr(layer, "_lib", csa.lib())  # (refused before anything is launched)
    with pytest.raises(csa.Csa2Error) as e:
        csa.csa2_fp8_gemm(*_product(m, n), out(), stream=0)
    assert e.value.status == INVALID
