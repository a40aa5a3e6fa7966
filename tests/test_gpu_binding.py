"""The binding of include/csa2_layer.h on the GPU: calls that it has to refuse, through the native marshalling and through
the Python code alike. Everything here is refused on the host: no kernel runs on what is refused."""
import pytest
import torch

import compressed_sparse_attention_append_b200 as csa
from compressed_sparse_attention_append_b200 import layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(params=["native", "python"])
def path(request, monkeypatch):
    layer._load()
    assert layer._fast is not None
    if request.param == "python":
        monkeypatch.setattr(layer, "_fast", None)
    return request.param


def test_a_product_into_overlapping_rows_is_refused(path):
    m, n, k = 4, 8, 128
    x, xs = torch.zeros(m, k, device=DEV, dtype=torch.uint8), torch.ones(1, m, device=DEV)
    w, ws = torch.zeros(n, k, device=DEV, dtype=torch.uint8), torch.ones(1, 1, device=DEV)
    for dtype in (torch.bfloat16, torch.float32):
        store = torch.full((m * n,), 7.0, device=DEV, dtype=dtype)
        for strides in ((0, 1), (1, 1), (7, 1)):
            with pytest.raises(csa.Csa2Error) as e:
                csa.csa2_fp8_gemm(x, xs, w, ws, store.as_strided((m, n), strides))
            assert e.value.status == csa.CSA2_ERR_INVALID_ARG
        assert bool((store == 7.0).all())
        csa.csa2_fp8_gemm(x[:1], xs[:, :1].contiguous(), w, ws, store.as_strided((1, n), (3, 1)))  # a single row
        assert not bool(store[:n].any()) and bool((store[n:] == 7.0).all())


def test_rotations_and_workspaces_of_another_device_are_refused(path):
    """(They are this device's and only say that they are another's: nothing foreign is ever reached.)"""
    own, far = (csa.Rope(torch.ones(8, device=DEV, dtype=torch.float64)) for _ in range(2))
    far.c.dev = torch.cuda.current_device() + 1
    x, pos = torch.ones(3, 2, 16, device=DEV), torch.arange(3, device=DEV)
    cache = csa.PagedCache(2, 64, 1, 2)
    cache.table.copy_(torch.arange(2, dtype=torch.int32, device=DEV))
    row = torch.ones(1, 1, 512, device=DEV, dtype=torch.bfloat16)
    for call in (lambda r: csa.csa2_rope(r, pos, x, x), lambda r: csa.csa2_norm_rope(r, pos, 1e-6, x, None, x),
                 lambda r: csa.csa2_paged_append(cache, 1, 1, pos[:1], row, rope=r),
                 lambda r: csa.csa2_paged_append(cache, 1, 1, pos[:1], swa=row, rope=own, swa_rope=r)):
        call(own)
        torch.cuda.synchronize()
        before = [t.clone() for t in (x, cache.l_data, cache.swa)]
        with pytest.raises(AssertionError, match="rotation of the current device"):
            call(far)
        assert all(torch.equal(a, b) for a, b in zip(before, (x, cache.l_data, cache.swa)))

    class Ws:
        nbytes = 256

        def __init__(self, buf):
            self.buf, self.ptr = buf, buf.data_ptr()

    class Foreign(torch.Tensor):
        def get_device(self):
            return torch.cuda.current_device() + 1

    buf = torch.zeros(256, dtype=torch.uint8, device=DEV)
    csa.csa2_paged_append(cache, 1, 1, pos[:1], row, ws=Ws(buf))
    with pytest.raises(AssertionError, match="workspace of the current device"):
        csa.csa2_paged_append(cache, 1, 1, pos[:1], row, ws=Ws(buf.as_subclass(Foreign)))


def _spoiled(t):
    yield "type", t.double() if t.dtype is not torch.float64 else t.float()
    yield "device", t.cpu()
    yield "subset", t[:0] if t.shape[0] else t.unsqueeze(0)
    yield "dimension", t.unsqueeze(0)
    yield "rows", torch.cat([t.view(torch.uint8)] * 2).view(t.dtype)
    if t.shape[-1] > 1:
        yield "strides", torch.stack([t.view(torch.uint8).view(t.shape + (-1,))] * 2, -2).view(t.dtype).squeeze(-1)[..., 0]


def test_every_tensor_of_every_call_is_checked(path):
    """One tensor of a good call at a time: of another type, on the host, of another shape, not dense along its last axis."""
    import test_marshal

    for fn, args, kw, _, outs in test_marshal._calls():
        for where in [*range(len(args)), *kw]:
            t = args[where] if isinstance(where, int) else kw[where]
            if not isinstance(t, torch.Tensor):
                continue
            for what, bad in _spoiled(t):
                a, k = list(args), dict(kw)
                if isinstance(where, int):
                    a[where] = bad
                else:
                    k[where] = bad
                torch.cuda.synchronize()
                before = [o.clone() for o in outs]
                with pytest.raises((AssertionError, AttributeError, ValueError, csa.Csa2Error)):
                    fn(*a, **k)
                    pytest.fail(f"{fn.__name__}: argument {where} with another {what} was taken")
                torch.cuda.synchronize()
                assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, outs))
