"""The native marshalling of the binding (csrc/marshal.cpp): it takes plain calls only, makes the same call as the
Python code of layer.py, and leaves everything else, refusals among them, to that code."""
import pytest
import torch

import compressed_sparse_attention_append_b200 as csa
from compressed_sparse_attention_append_b200 import build, layer

NAMES = {"rope": 5, "norm_rope": 10, "quantize": 4, "gemm": 8, "append": 21, "gather": 10, "attend": 19}


@pytest.fixture(scope="module")
def fast():
    build.build_marshal()
    layer._load()
    assert layer._fast is not None
    return layer._fast


@pytest.mark.parametrize("name", NAMES)
def test_takes_nothing_but_cuda_tensors(fast, name):
    f, n = getattr(fast, name), NAMES[name]
    t = torch.zeros(4, 4, 4, dtype=torch.bfloat16)
    for args in ((), (None,) * n, (0,) * n, (1 << 80,) * n, (t,) * n, ("x",) * n, (0,) * (n + 1), (t[0, 0],) * n, (-1,) * n):
        assert f(*args) is None


def test_refuses_bad_addresses(fast):
    with pytest.raises(TypeError):
        fast.bind(1, 2)
    with pytest.raises(ValueError):
        fast.bind(*[0] * 7)
    with pytest.raises(TypeError):
        fast.bind(*["x"] * 7)


def _calls():
    """(entry point, arguments, keywords, index of a tensor to spoil, outputs) on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)
    i64 = lambda *v: torch.tensor(v, device="cuda")
    b, t, heads, d = 2, 3, 5, 128
    rope = csa.Rope.for_context(64, offset=448)
    small = csa.Rope.for_context(32, offset=64)
    x = r(6, 2 * heads, d)[:, ::2]
    out = torch.empty(6, heads, d, device="cuda", dtype=torch.bfloat16)
    yield csa.csa2_rope, (small, torch.arange(6, device="cuda"), x, out), {}, 2, [out]
    ko = torch.empty(6, 1, d, device="cuda", dtype=torch.bfloat16)
    out = torch.empty_like(out)
    yield csa.csa2_norm_rope, (small, torch.arange(6, device="cuda"), 1e-6, x, r(d), out, x[:, :1], r(d), ko), {}, 3, [out, ko]
    f32 = torch.empty(6, heads, d, device="cuda")
    yield csa.csa2_norm_rope, (None, None, 1e-6, r(6, heads, d, dtype=torch.float32), None, f32), {}, 3, [f32]
    e8 = lambda *s: torch.empty(*s, device="cuda", dtype=torch.float8_e4m3fn)
    xs, wide = torch.empty(3, 9, device="cuda"), r(9, 400)
    q = e8(9, 272)
    yield csa.csa2_fp8_quantize, (wide[:, :272], q, xs), {}, 0, [q.view(torch.uint8), xs]
    w, ws = e8(130, 272), torch.empty(2, 3, device="cuda")
    csa.csa2_fp8_quantize_weight(r(130, 272), w, ws)
    csa.csa2_fp8_quantize(wide[:, :272], q, xs)
    for o, bytes_ in ((torch.empty(9, 130, device="cuda"), False), (torch.zeros(9, 200, device="cuda", dtype=torch.bfloat16)[:, :130], True)):
        yield csa.csa2_fp8_gemm, (q.view(torch.uint8) if bytes_ else q, xs, w, ws, o), {}, 2, [o]
    cache = csa.PagedCache(4, 64, b, 2)
    cache.table.copy_(torch.arange(4, dtype=torch.int32, device="cuda").view(b, 2))
    pos, lens = i64(3, 60), torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    planes = [cache.l_data, cache.l_scale, cache.k_data, cache.k_scale, cache.swa]
    yield (csa.csa2_paged_append, (cache, b, t, pos, r(b, t, 512), r(b, t, 128), r(b, t, 512)),
           dict(rope=rope, idx_rope=small, w_latent=r(512), w_swa=r(512), length=lens), 4, planes)
    yield (csa.csa2_paged_append, (cache, b, t, pos), dict(swa=r(b, t, 512), swa_rope=rope, rpos=torch.arange(6, device="cuda").view(b, t)),
           3, [cache.swa])
    idx = torch.tensor([[3, 4, -1], [60, 61, 5]], dtype=torch.int32, device="cuda")
    lo, ko = torch.empty(b, 3, 512, device="cuda", dtype=torch.bfloat16), torch.empty(b, 3, 128, device="cuda", dtype=torch.bfloat16)
    yield csa.csa2_paged_gather, (cache, b, idx, lo, ko), {}, 3, [lo, ko]
    out, lse = torch.empty(b, 64, 512, device="cuda", dtype=torch.bfloat16), torch.empty(b, 64, device="cuda")
    yield (csa.csa2_paged_attend, (cache, b, 1, i64(5, 61), r(b, 64, 512), idx, 3, out), dict(lse=lse, swa_begin=i64(3, 60)), 4,
           [out, lse])


@pytest.mark.gpu
def test_same_call_as_the_python_code(fast, monkeypatch):
    """Same bytes as the Python path, on the current stream and on a named one; the native code took the call."""
    taken = []

    class Spy:
        def __getattr__(self, name):
            def call(*args):
                taken.append(getattr(fast, name)(*args))
                return taken[-1]
            return call

    for fn, args, kw, _, outs in _calls():
        stream = torch.cuda.Stream()
        got = []
        for native, s in ((Spy(), None), (Spy(), stream.cuda_stream), (None, None)):
            monkeypatch.setattr(layer, "_fast", native)
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            fn(*args, **kw, stream=s)
            torch.cuda.synchronize()
            got.append([o.contiguous().clone() for o in outs])
        assert taken[-2:] == [0, 0], fn.__name__
        assert all(o.view(torch.uint8).any() for o in got[2]), fn.__name__
        for a, b, c in zip(*got):
            assert torch.equal(a.view(torch.uint8), c.view(torch.uint8)), fn.__name__
            assert torch.equal(b.view(torch.uint8), c.view(torch.uint8)), fn.__name__


@pytest.mark.gpu
def test_refusals_stay(fast):
    for fn, args, kw, at, _ in _calls():
        t = args[at]
        optional = fn in (csa.csa2_paged_append, csa.csa2_paged_gather)
        for bad in (t.double(), t.cpu(), t[:1], t.unsqueeze(0), "x", *([] if optional else [None])):
            with pytest.raises((AssertionError, AttributeError, ValueError, TypeError, csa.Csa2Error)):
                fn(*args[:at], bad, *args[at + 1:], **kw)
    torch.cuda.synchronize()
