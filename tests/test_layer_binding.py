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


class Foreign(torch.Tensor):
    """A host tensor that says it lies on device 1."""

    def get_device(self):
        return 1


def _on_device_1(monkeypatch, make):
    with monkeypatch.context() as m:
        m.setattr(layer, "_device", lambda: 1)
        return make()


def test_a_rotation_of_another_device_is_refused(host, monkeypatch):
    rope = lambda: csa.Rope(torch.ones(8, dtype=torch.float64).as_subclass(Foreign))
    far = _on_device_1(monkeypatch, rope)
    x, pos = torch.zeros(3, 2, 16), torch.zeros(3, dtype=torch.int64)
    own = csa.Rope(torch.ones(8, dtype=torch.float64))
    cache = csa.PagedCache(2, 64, 1, 2, device="cpu")
    row = torch.zeros(1, 1, 512, dtype=torch.bfloat16)
    key = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    calls = [
        lambda r: csa.csa2_rope(r, pos, x, x, stream=0),
        lambda r: csa.csa2_norm_rope(r, pos, 1e-6, x, None, x, stream=0),
        lambda r: csa.csa2_paged_append(cache, 1, 1, pos[:1], row, rope=r, stream=0),
        lambda r: csa.csa2_paged_append(cache, 1, 1, pos[:1], None, key, idx_rope=r, stream=0),
        lambda r: csa.csa2_paged_append(cache, 1, 1, pos[:1], swa=row, swa_rope=r, stream=0),
    ]
    for call in calls:
        call(own)
        assert len(host.calls) == 1
        with pytest.raises(AssertionError, match="rotation of the current device"):
            call(far)
        with pytest.raises(AssertionError, match="rotation of the current device"):
            call(_on_device_1(monkeypatch, far.transposed))
        assert len(host.calls) == 1
        host.calls.clear()


class Ws:
    nbytes = 1 << 20

    def __init__(self, buf):
        self.buf, self.ptr = buf, buf.data_ptr()


def test_a_workspace_of_another_device_is_refused(host):
    buf = torch.zeros(256, dtype=torch.uint8)
    own, far = Ws(buf), Ws(buf.as_subclass(Foreign))
    cache = csa.PagedCache(2, 64, 1, 2, device="cpu")
    pos, idx = torch.zeros(1, dtype=torch.int64), torch.zeros(1, 4, dtype=torch.int32)
    q, out = torch.zeros(1, 64, 512, dtype=torch.bfloat16), torch.zeros(1, 64, 512, dtype=torch.bfloat16)
    calls = [
        lambda ws: csa.csa2_fp8_gemm(*_product(4, 8), torch.empty(4, 8), status=ws, stream=0),
        lambda ws: csa.csa2_paged_append(cache, 1, 1, pos, q[:, :1, :], ws=ws, stream=0),
        lambda ws: csa.csa2_paged_gather(cache, 1, idx, torch.zeros(1, 4, 512, dtype=torch.bfloat16), ws=ws, stream=0),
        lambda ws: csa.csa2_paged_attend(cache, 1, 1, pos, q, idx, 4, out, ws=ws, stream=0),
        lambda ws: csa.csa2_paged_index_topk(cache, 1, 1, pos, q[:, :4, :128].contiguous(), 4, idx, ws, stream=0),
    ]
    for call in calls:
        call(own)
        assert len(host.calls) == 1 and own.ptr in host.calls[0][1]
        with pytest.raises(AssertionError, match="workspace of the current device"):
            call(far)
        assert len(host.calls) == 1
        host.calls.clear()


def test_what_a_struct_was_made_from_cannot_be_replaced(host):
    """A new tensor in its place would not reach the library, which keeps the old one's address."""
    cache = csa.PagedCache(2, 64, 1, 2, device="cpu", swa_slot=torch.zeros(1, dtype=torch.int32))
    rope = csa.Rope(torch.ones(8, dtype=torch.float64), offset=2, mscale=1.5)
    for what in (cache, rope):
        for name, value in list(vars(what).items()):
            with pytest.raises(AttributeError, match="fixed"):
                setattr(what, name, value)
    cache.table[0, 1] = 1  # in place it is the caller's
    assert cache.table.data_ptr() == cache.c.table and cache.swa_slot.data_ptr() == cache.c.swa_slot
    assert rope.inv_freq.data_ptr() == rope.c.spec.inv_freq


def test_the_inverse_of_a_rotation_takes_its_scale_out(host):
    f = torch.ones(8, dtype=torch.float64)
    for mscale in (1.0, 1.277, 0.5, 0.0):  # (0 stands for 1)
        rope = csa.Rope(f, offset=2, interleaved=True, mscale=mscale)
        back, again, t = rope.inverted(), rope.inverted().inverted(), rope.transposed()
        m = mscale or 1.0
        for r, scale, turned in ((back, 1.0 / m, 1), (again, m, 0), (t, mscale, 1)):
            s = r.c.spec
            assert (s.inv_freq, s.rot, s.offset, s.layout, s.transposed) == (f.data_ptr(), 16, 2, 1, turned)
            assert abs(s.mscale - scale) <= 2.0 ** -23 * scale
