"""include/csa2_layer.h without a GPU: every declared symbol is exported, the header is plain C, the
frequency helper follows the published rules, and calls that cannot be right return their error before
anything is launched (the pointers below are host memory or not real)."""
import ctypes
import math
import os
import re
import subprocess
import tempfile

import pytest
import torch

import compressed_sparse_attention_append_b200 as csa
from conftest import ROOT

OK, INVALID, SHAPE, CAPACITY, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from compressed_sparse_attention_append_b200 import build

    build.build()
    return csa.lib()


def test_every_declared_symbol_is_exported(L):
    src = open(os.path.join(ROOT, "include", "csa2_layer.h")).read()
    names = re.findall(r"CSA2_API\s+[\w\s\*]+?\b(csa2_\w+)\s*\(", src)
    assert sorted(names) == sorted(csa.LAYER_EXPORTS) and len(set(names)) == len(names)
    for n in names:
        assert hasattr(L, n) and hasattr(csa, n)


def test_a_plain_c_program_uses_the_header(L):
    prog = r"""
#include <stdio.h>
#include "csa2_layer.h"
int main(void) {
    double f[32];
    float m = 0.f;
    csa2_paged_cache c = {0};
    csa2_heads h = {0};
    csa2_append_row r = {0};
    csa2_rope_spec s = {0};
    (void)h; (void)r; (void)s;
    int a = csa2_rope_frequencies(64, 10000.0, CSA2_ROPE_YARN, 16.0, 4096, 32.0, 1.0, f, &m);
    int b = csa2_paged_gather(&c, 0, 0, NULL, NULL, NULL, NULL, 0, NULL);
    c.page = 64;
    int d = csa2_paged_gather(&c, 0, 0, NULL, NULL, NULL, NULL, 0, NULL);
    printf("%d %.17g %.9g %d %d\n", a, f[31], m, b, d);
    return 0;
}
"""
    libdir = os.path.dirname(csa.lib()._name)
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(c, "w").write(prog)
        subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), c, "-o", exe,
                               "-L", libdir, "-l:libcsa2.so", f"-Wl,-rpath,{libdir}"])
        out = subprocess.run([exe], capture_output=True, text=True, timeout=60, check=True).stdout.split()
    f, m = csa.csa2_rope_frequencies(64, 10000.0, "yarn", 16.0, 4096)
    assert out[0] == "0" and float(out[1]) == float(f[31]) and abs(float(out[2]) - m) < 1e-6
    assert int(out[3]) == INVALID and int(out[4]) == OK


def test_frequencies(L):
    rot, base = 64, 10000.0
    plain, m = csa.csa2_rope_frequencies(rot, base)
    j = torch.arange(rot // 2, dtype=torch.float64)
    assert m == 1.0 and torch.allclose(plain, base ** (-2 * j / rot), rtol=1e-14, atol=0)
    lin, m = csa.csa2_rope_frequencies(rot, base, "linear", 8.0)
    assert m == 1.0 and torch.allclose(lin, plain / 8, rtol=1e-14, atol=0)
    ntk, m = csa.csa2_rope_frequencies(rot, base, "ntk", 8.0)
    # the fastest pair keeps its frequency, the slowest is stretched by the factor
    assert m == 1.0 and ntk[0] == 1.0 and abs(float(plain[-1] / ntk[-1]) - 8.0) < 1e-9
    yarn, m = csa.csa2_rope_frequencies(rot, base, "yarn", 8.0, 4096, 32.0, 1.0)
    assert abs(m - (0.1 * math.log(8.0) + 1.0)) < 1e-6
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], plain[turns > 40])
    slow = turns < 0.7
    assert torch.allclose(yarn[slow], plain[slow] / 8, rtol=1e-14, atol=0)
    ratio = yarn / plain
    assert bool((ratio[1:] <= ratio[:-1] + 1e-12).all())  # a ramp between them
    mid = (ratio < 1) & (ratio > 1 / 8 + 1e-9)
    step = ratio[1:][mid[1:] & mid[:-1]] - ratio[:-1][mid[1:] & mid[:-1]]
    assert step.numel() > 3 and torch.allclose(step, step[:1].expand_as(step), rtol=1e-9, atol=0)  # linear
    assert csa.csa2_rope_frequencies(0)[0].numel() == 0
    for bad in ((63, base, "plain", 1.0), (-2, base, "plain", 1.0), (64, 1.0, "plain", 1.0), (64, base, "linear", 0.5),
                (64, base, "linear", float("nan")), (64, base, "yarn", 2.0), (2, base, "ntk", 2.0)):
        with pytest.raises(csa.Csa2Error) as e:
            csa.csa2_rope_frequencies(*bad)
        assert e.value.status == INVALID
    m = ctypes.c_float(0)
    buf = (ctypes.c_double * 32)()
    assert L.csa2_rope_frequencies(64, base, 7, 1.0, 0, 0.0, 0.0, buf, ctypes.byref(m)) == INVALID
    assert L.csa2_rope_frequencies(64, base, 3, 2.0, 4096, 1.0, 32.0, buf, ctypes.byref(m)) == INVALID
    assert L.csa2_rope_frequencies(64, base, 0, 1.0, 0, 0.0, 0.0, None, ctypes.byref(m)) == INVALID
    assert L.csa2_rope_frequencies(64, base, 0, 1.0, 0, 0.0, 0.0, buf, None) == INVALID


FAKE = 1 << 41  # never dereferenced: every call below is refused, or has nothing to do


def _spec(rot=64, offset=0, layout=0, transposed=0, mscale=1.0, f=FAKE):
    return ctypes.byref(csa.csa2_rope_spec(f, rot, offset, layout, transposed, mscale))


def _heads(x=FAKE, out=FAKE + 4096, xt=512, xh=64, ot=512, oh=64, w=None, n=8):
    return ctypes.byref(csa.csa2_heads(x, out, xt, xh, ot, oh, w, n))


def test_rotation_refusals(L):
    r, nr = L.csa2_rope, L.csa2_norm_rope
    assert r(_spec(), 0, 0, 64, None, _heads(), None) == OK          # no token
    assert r(_spec(), 0, 5, 64, FAKE, _heads(n=0), None) == OK       # no head
    assert nr(None, 0, 0, 64, None, 0.0, _heads(w=FAKE), None, None) == OK
    for spec in (_spec(rot=63), _spec(rot=66), _spec(rot=-2), _spec(offset=1), _spec(offset=-1), _spec(layout=2),
                 _spec(transposed=2), _spec(mscale=float("nan")), _spec(mscale=float("inf")), _spec(f=None),
                 _spec(f=FAKE + 4)):
        assert r(spec, 0, 4, 64, FAKE, _heads(), None) == INVALID
        assert nr(spec, 0, 4, 64, FAKE, 1e-6, _heads(), None, None) == INVALID
    assert r(None, 0, 4, 64, FAKE, _heads(), None) == INVALID
    assert r(_spec(), 0, 4, 64, None, _heads(), None) == INVALID     # positions are needed
    assert r(_spec(), 2, 4, 64, FAKE, _heads(), None) == INVALID     # no such element type
    assert r(_spec(), 0, -1, 64, FAKE, _heads(), None) == INVALID
    assert r(_spec(), 0, 4, 64, FAKE, None, None) == INVALID
    assert r(_spec(), 0, 4, 64, FAKE, _heads(w=FAKE), None) == INVALID  # a weight without a norm
    assert r(_spec(rot=0), 0, 4, 0, FAKE, _heads(), None) == SHAPE
    assert r(_spec(), 0, 4, 1025, FAKE, _heads(), None) == SHAPE
    assert r(_spec(), 0, 4, 64, FAKE, _heads(n=65537), None) == SHAPE
    for h in (_heads(x=None), _heads(out=None), _heads(x=FAKE + 1), _heads(xt=-1), _heads(oh=-64), _heads(n=-1),
              _heads(out=FAKE, ot=1024)):                            # in place, with other strides
        assert r(_spec(), 0, 4, 64, FAKE, h, None) == INVALID
        assert nr(_spec(), 0, 4, 64, FAKE, 1e-6, _heads(), h, None) == INVALID
    assert r(_spec(), 1, 4, 64, FAKE, _heads(x=FAKE + 2), None) == INVALID  # fp32 at a 2-byte address
    for eps in (-1e-6, float("nan"), float("inf")):
        assert nr(_spec(), 0, 4, 64, FAKE, eps, _heads(), None, None) == INVALID


def test_fp8_refusals(L):
    q, w, g = L.csa2_fp8_quantize, L.csa2_fp8_quantize_weight, L.csa2_fp8_gemm
    assert q(0, 128, None, 128, None, None, None) == OK and w(0, 128, None, None, None, None) == OK
    for k in (0, -16, 8, 100):
        assert q(4, k, FAKE, 128, FAKE, FAKE, None) == INVALID
        assert w(4, k, FAKE, FAKE, FAKE, None) == INVALID
        assert g(4, 4, k, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 4, None, 0, None) == INVALID
    assert q(-1, 128, FAKE, 128, FAKE, FAKE, None) == INVALID
    assert q(4, 128, FAKE, 129, FAKE, FAKE, None) == INVALID
    for bad in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (FAKE + 8, FAKE, FAKE), (FAKE, FAKE + 8, FAKE),
                (FAKE, FAKE, FAKE + 2)):
        assert q(4, 128, bad[0], 128, bad[1], bad[2], None) == INVALID
        assert w(4, 128, *bad, None) == INVALID
    assert g(0, 4, 128, None, None, None, None, 0, None, 4, None, 0, None) == OK
    assert g(4, 0, 128, None, None, None, None, 0, None, 0, None, 0, None) == OK
    assert g(4, 8, 128, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 7, None, 0, None) == INVALID
    assert g(4, 8, 128, FAKE, FAKE, FAKE, FAKE, 5, FAKE, 8, None, 0, None) == INVALID
    assert g(4, 8, 128, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, FAKE, 128, None) == WORKSPACE
    assert g(1 << 31, 8, 128, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, None, 0, None) == SHAPE
    for i, bad in ((3, None), (4, None), (5, None), (6, None), (8, None), (3, FAKE + 8), (5, FAKE + 4), (4, FAKE + 2),
                   (8, FAKE + 1)):
        a = [4, 8, 128, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, None, 0, None]
        a[i] = bad
        assert g(*a) == INVALID
    assert g(4, 8, 128, FAKE, FAKE, FAKE, FAKE, 1, FAKE + 2, 8, None, 0, None) == INVALID


def _paged(page=64, n_pages=100, max_pages=50, swa_cap=128, n_slots=4, **kw):
    c = csa.csa2_paged_cache(*[FAKE + 4096 * i for i in range(6)], None, n_pages, max_pages, n_slots, swa_cap, page)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _row(x=FAKE, xb=512, xt=512, w=None, rope=None):
    return ctypes.byref(csa.csa2_append_row(x, xb, xt, w, ctypes.pointer(rope) if rope is not None else None))


def test_paged_refusals(L):
    a, ga, at, ix = L.csa2_paged_append, L.csa2_paged_gather, L.csa2_paged_attend, L.csa2_paged_index_topk

    def app(c=None, batch=1, t=1, pos=FAKE, eps=1e-6, lat=None, key=None, swa=None, ws=None, n=0):
        return a(c or _paged(), batch, t, pos, None, None, eps, lat or _row(), key, swa, ws, n, None)

    def att(c=None, batch=1, tq=1, qpos=FAKE, q=FAKE, idx=FAKE, k=8, win=128, ratio=1, scale=0.0, out=FAKE, of=None, ws=None, n=0):
        return at(c or _paged(), batch, tq, qpos, q, idx, k, None, win, ratio, scale, out, of, None, ws, n, None)

    def top(c=None, batch=1, tq=1, qpos=FAKE, iq=FAKE, hi=4, k=8, ratio=1, ctx=64, flags=0, out=FAKE, ws=FAKE, n=1 << 20):
        return ix(c or _paged(), batch, tq, qpos, iq, hi, k, ratio, ctx, flags, out, ws, n, None)

    assert app(batch=0) == OK and app(t=0) == OK and att(batch=0) == OK and top(batch=0) == OK
    assert a(_paged(), 1, 1, FAKE, None, None, 1e-6, None, None, None, None, 0, None) == OK  # nothing to append
    for f in (app, att, top):
        assert f(c=_paged(page=0)) == INVALID and f(c=_paged(page=48)) == INVALID and f(c=_paged(page=4)) == INVALID
        assert f(c=_paged(page=1 << 17)) == INVALID and f(c=_paged(n_pages=-1)) == INVALID
        assert f(c=_paged(n_pages=(1 << 31) // 64)) == CAPACITY and f(c=_paged(max_pages=(1 << 30) // 64 + 1)) == CAPACITY
        assert f(c=_paged(table=None)) == INVALID and f(batch=-1) == INVALID
    for f in (app, att):
        assert f(c=_paged(l_data=None)) == INVALID and f(c=_paged(l_scale=FAKE + 8)) == INVALID
        assert f(ws=FAKE, n=64) == WORKSPACE
    assert app(pos=None) == INVALID and app(t=-1) == INVALID and app(eps=-1.0) == INVALID and app(eps=float("nan")) == INVALID
    assert app(lat=_row(x=FAKE + 8)) == INVALID and app(lat=_row(w=FAKE + 2)) == INVALID
    assert app(lat=_row(xt=511)) == INVALID and app(lat=_row(xb=-8)) == INVALID
    spec = csa.csa2_rope_spec(FAKE, 64, 448, 0, 0, 1.0)
    assert app(batch=0, lat=_row(rope=spec)) == OK
    for bad in (csa.csa2_rope_spec(FAKE, 64, 449, 0, 0, 1.0), csa.csa2_rope_spec(FAKE, 64, 448, 0, 1, 1.0),
                csa.csa2_rope_spec(None, 64, 448, 0, 0, 1.0)):
        assert app(lat=_row(rope=bad)) == INVALID
    wide = csa.csa2_rope_spec(FAKE, 256, 0, 0, 0, 1.0)
    assert app(key=_row(rope=wide)) == INVALID  # wider than the key
    assert app(key=_row(), c=_paged(k_data=None)) == INVALID
    assert app(swa=_row(), c=_paged(swa_cap=100)) == INVALID and app(swa=_row(), c=_paged(swa=None)) == INVALID
    assert ga(_paged(), 1, 1, None, FAKE, None, None, 0, None) == INVALID
    assert ga(_paged(), 1, 1, FAKE, FAKE + 2, None, None, 0, None) == INVALID
    assert ga(_paged(), 1, -1, FAKE, FAKE, None, None, 0, None) == INVALID
    assert ga(_paged(), 1, 1, FAKE, None, None, None, 0, None) == OK
    assert ga(_paged(k_scale=None), 1, 1, FAKE, None, FAKE, None, 0, None) == INVALID
    assert att(k=2049) == INVALID and att(k=-1) == INVALID and att(tq=0) == INVALID and att(idx=None) == INVALID
    assert att(win=129) == SHAPE and att(ratio=3) == SHAPE and att(scale=-1.0) == INVALID and att(scale=float("nan")) == INVALID
    assert att(q=FAKE + 8) == INVALID and att(out=None) == INVALID and att(of=FAKE + 4) == INVALID and att(qpos=None) == INVALID
    assert att(c=_paged(swa_cap=64)) == CAPACITY and att(c=_paged(swa=None)) == INVALID
    assert top(hi=0) == INVALID and top(hi=65) == INVALID and top(k=0) == INVALID and top(ratio=0) == SHAPE
    assert top(flags=2) == INVALID and top(ctx=0) == INVALID and top(ws=None) == WORKSPACE and top(n=256) == WORKSPACE
    assert top(c=_paged(k_data=None)) == INVALID and top(iq=FAKE + 2) == INVALID


def test_the_binding_checks_shapes_types_and_devices(L):
    f = torch.ones(8, dtype=torch.float64)
    with pytest.raises(AssertionError, match="CUDA"):
        csa.Rope(f)
    with pytest.raises(AssertionError, match="float64"):
        csa.Rope(f.float())
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(AssertionError, match="bfloat16"):
        csa.csa2_fp8_quantize(x.float(), q, torch.zeros(1, 4))
    with pytest.raises(AssertionError, match="dense rows"):
        csa.csa2_fp8_quantize(x.T, q, torch.zeros(1, 4))
    with pytest.raises(AssertionError, match="CUDA"):
        csa.csa2_fp8_gemm(q, torch.zeros(1, 4), q, torch.zeros(1, 1), torch.zeros(4, 4))
    with pytest.raises(AssertionError, match="bf16 or fp32"):
        csa.csa2_fp8_gemm(q, torch.zeros(1, 4), q, torch.zeros(1, 1), torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(AssertionError, match="window ring"):
        csa.PagedCache(4, 64, 2, 2, n_slots=1, device="cpu")
    with pytest.raises(AssertionError, match="CUDA"):
        csa.PagedCache(4, 64, 2, 2, device="cpu")
