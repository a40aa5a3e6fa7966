"""Measured cases of the operators around the CSA2 core: FP8 products, rotary positions, per-head
norms, the paged latent cache and the attention that reads it. Each has a plain form in elementary
torch operations, the framework's own calls, and its definition in 64 bits (`exact`)."""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6
PAGE = 64      # entries per cache page
RING = 128     # window rows kept per sequence


def listed():
    return [
        # one token through a small projection: launch latency
        {"name": "linear_token", "op": "linear", "m": 1, "k": 1024, "n": 1536, "out": "bf16"},
        # 128 decode sequences through the query projection (64 heads x 512): the weights' bytes
        {"name": "linear_decode", "op": "linear", "m": 128, "k": 4096, "n": 32768, "out": "bf16"},
        # ragged batch, contraction that ends inside a scale block, odd output width, fp32 logits
        {"name": "linear_ragged", "op": "linear", "m": 777, "k": 4112, "n": 4099, "out": "f32"},
        # a prefill chunk of 4096 tokens through the query projection: arithmetic
        {"name": "linear_prefill", "op": "linear", "m": 4096, "k": 4096, "n": 32768, "out": "bf16"},
        # queries of 128 decode sequences at far positions, frequencies stretched for a long context
        {"name": "rope_decode", "op": "rope", "t": 128, "heads": 64, "d": 512, "rot": 64, "offset": 448,
         "interleaved": True, "dtype": "bf16", "inverse": False, "start": 1 << 20, "factor": 16.0},
        # the attention output of a prefill chunk turned back (keys and values share the rotation)
        {"name": "rope_prefill_back", "op": "rope", "t": 4096, "heads": 64, "d": 512, "rot": 64, "offset": 448,
         "interleaved": True, "dtype": "bf16", "inverse": True, "start": 1 << 20, "factor": 16.0},
        # one token's 16 query heads and its key head, whole head rotated in halves: launch latency
        {"name": "norm_rope_token", "op": "norm_rope", "t": 1, "hq": 16, "hk": 1, "d": 128, "rot": 128, "offset": 0,
         "interleaved": False, "dtype": "bf16", "start": 4096, "factor": 1.0},
        # a prefill chunk's queries (64 heads) and latent out of one fused projection
        {"name": "norm_rope_prefill", "op": "norm_rope", "t": 4096, "hq": 64, "hk": 1, "d": 512, "rot": 64,
         "offset": 448, "interleaved": True, "dtype": "bf16", "start": 1 << 20, "factor": 16.0},
        # one new token of each of 128 sequences appended: latent, indexer key, window row
        {"name": "append_decode", "op": "append", "b": 128, "t": 1, "start": 131071, "ragged": False, "rot": 64,
         "interleaved": True},
        # prefill chunks of 16 sequences of unequal lengths appended together
        {"name": "append_prefill", "op": "append", "b": 16, "t": 2048, "start": 1000, "ragged": True, "rot": 64,
         "interleaved": True},
        # a single sequence's decode row with many selected entries: one row to spread over the GPU
        {"name": "attend_token", "op": "attend", "b": 1, "tq": 1, "k": 2048, "n": 32768},
        # 128 sequences, 512 selected entries each, pages in any order
        {"name": "attend_decode", "op": "attend", "b": 128, "tq": 1, "k": 512, "n": 32768},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rope", "norm_rope", "append", "attend"])
    if op == "linear":
        m, k, n = _log(rng, 1, 4096), 16 * _log(rng, 8, 512), _log(rng, 64, 32768)
        return {"op": op, "m": m, "k": k, "n": max(1, min(n, (1 << 39) // (m * k))),
                "out": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("rope", "norm_rope"):
        d = rng.choice([64, 128, 192, 512])
        heads = rng.choice([1, 3, 4, 16, 32, 64])
        rot = rng.choice([d, d // 2, d // 2, 40])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c = {"op": op, "t": _log(rng, 1, 4096 if dtype == "bf16" else 2048), "d": d, "rot": rot,
             "offset": rng.choice([0, d - rot]), "interleaved": rng.random() < 0.5, "dtype": dtype,
             "start": _log(rng, 1, 1 << 20), "factor": rng.choice([1.0, 4.0, 16.0])}
        if op == "rope":
            return {**c, "heads": heads, "inverse": rng.random() < 0.5}
        return {**c, "hq": heads, "hk": rng.choice([1, 4])}
    if op == "append":
        t = _log(rng, 1, 2048)
        return {"op": op, "b": _log(rng, 1, max(1, min(128, 32768 // t))), "t": t, "start": _log(rng, 1, 131072),
                "ragged": rng.random() < 0.5, "rot": rng.choice([32, 64, 128]), "interleaved": rng.random() < 0.5}
    tq = rng.choice([1, 1, 2, 5])
    return {"op": op, "b": _log(rng, 1, 128 // tq), "tq": tq, "k": _log(rng, 1, 512), "n": _log(rng, 16, 32768)}


# ---- inputs -----------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _frequencies(rot, factor):
    """Angles per position, base 10000; `factor` > 1: the slow channels interpolated (a linear ramp over
    the number of turns in 4096 positions, 32 to 1), the fast ones kept, and the scale that goes with it."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    f = f * keep + f / factor * (1.0 - keep) if factor != 1.0 else f
    return f.contiguous(), 0.1 * math.log(factor) + 1.0 if factor != 1.0 else 1.0


def _positions(g, t, start):
    return start + torch.randint(0, 4096, (t,), generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    return {"case": case, **globals()["_prepare_" + case["op"]](case, g)}


def _prepare_linear(c, g):
    m, k, n = c["m"], c["k"], c["n"]
    x = torch.randn(m, k, generator=g, device=DEV)
    x *= torch.where(torch.rand(k, generator=g, device=DEV) < 0.01, 8.0, 1.0)  # a few large channels
    w = (torch.randn(n, k, generator=g, device=DEV) * 96.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(-(-n // 128), -(-k // 128), generator=g, device=DEV) * 3e-4 + 1e-4
    out = torch.empty(m, n, device=DEV, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    return {"x": x.to(torch.bfloat16), "w": w, "ws": ws, "out": out,
            "xq": torch.empty(m, k, device=DEV, dtype=torch.float8_e4m3fn),
            "xs": torch.empty(-(-k // 128), m, device=DEV)}


def _rope_state(c, g):
    f, mscale = _frequencies(c["rot"], c["factor"])
    s = {"freq": f, "mscale": mscale, "pos": _positions(g, c["t"], c["start"])}
    if own:
        import compressed_sparse_attention_append_b200 as csa

        s["rope"] = csa.Rope(f, offset=c["offset"], interleaved=c["interleaved"], mscale=mscale,
                             inverse=c.get("inverse", False))
    return s


def _prepare_rope(c, g):
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    x = _normal(g, c["t"], c["heads"], c["d"], dtype=dt)
    return {**_rope_state(c, g), "x": x, "out": torch.empty_like(x)}


def _prepare_norm_rope(c, g):
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    t, hq, hk, d = c["t"], c["hq"], c["hk"], c["d"]
    fused = _normal(g, t, (hq + hk) * d, dtype=dt)  # one projection's output: queries, then keys
    return {**_rope_state(c, g), "q": fused[:, :hq * d].view(t, hq, d), "k": fused[:, hq * d:].view(t, hk, d),
            "wq": 1.0 + 0.1 * _normal(g, d, dtype=dt), "wk": 1.0 + 0.1 * _normal(g, d, dtype=dt),
            "q_out": torch.empty(t, hq, d, device=DEV, dtype=dt), "k_out": torch.empty(t, hk, d, device=DEV, dtype=dt)}


def _page_table(g, b, pages):
    return torch.randperm(b * pages, generator=g, device=DEV).to(torch.int32).view(b, pages)


def _prepare_append(c, g):
    b, t = c["b"], c["t"]
    pages = -(-(c["start"] + 64 + t) // PAGE)
    s = {"latent": _normal(g, b, t, 512), "key": _normal(g, b, t, 128), "swa": _normal(g, b, t, 512),
         "w_latent": 1.0 + 0.1 * _normal(g, 512), "w_key": 1.0 + 0.1 * _normal(g, 128),
         "w_swa": 1.0 + 0.1 * _normal(g, 512),
         "pos": c["start"] + torch.randint(0, 64, (b,), generator=g, device=DEV),
         "len": torch.randint(0 if c["ragged"] else t, t + 1, (b,), generator=g, device=DEV).to(torch.int32)}
    s["freq"], s["mscale"] = _frequencies(c["rot"], 1.0)
    s["kfreq"], _ = _frequencies(64, 1.0)
    i = torch.arange(t, device=DEV)
    s["rows"] = torch.where(i < s["len"][:, None], s["pos"][:, None] + i, -1).to(torch.int32)  # entries to read back
    s["latent_out"] = torch.empty(b, t, 512, device=DEV, dtype=torch.bfloat16)
    s["key_out"] = torch.empty(b, t, 128, device=DEV, dtype=torch.bfloat16)
    if own:
        import compressed_sparse_attention_append_b200 as csa

        s["cache"] = csa.PagedCache(b * pages, PAGE, b, pages, RING, page_table=_page_table(g, b, pages))
        s["rope"] = csa.Rope(s["freq"], offset=512 - c["rot"], interleaved=c["interleaved"])
        s["key_rope"] = csa.Rope(s["kfreq"], offset=64, interleaved=c["interleaved"])
    return s


def _prepare_attend(c, g):
    b, tq, k, n = c["b"], c["tq"], c["k"], c["n"]
    pages = -(-n // PAGE)
    rows = b * tq
    qpos = n - 1 - (tq - 1) + torch.arange(tq, device=DEV)
    qpos = qpos.repeat(b).clamp_min(0)
    # distinct visible entries in ascending order, padded with -1 where fewer are visible
    pick = torch.rand(rows, max(n - tq + 1, k), generator=g, device=DEV)
    pick[:, max(n - tq + 1, 0):] = 2.0
    near, at = torch.topk(pick, k, dim=1, largest=False)
    idx = torch.where(near < 1.0, at, 1 << 30).sort(dim=1).values
    s = {"q": _normal(g, rows, 64, 512), "qpos": qpos, "idx": torch.where(idx < 1 << 30, idx, -1).to(torch.int32),
         "l_data": torch.randint(0, 256, (b * pages, PAGE, 256), generator=g, device=DEV, dtype=torch.uint8),
         "l_scale": torch.randint(0x20, 0x39, (b * pages, PAGE, 32), generator=g, device=DEV, dtype=torch.uint8),
         # several rows of a sequence reach further back than one
         "swa": torch.randn(b, RING if tq == 1 else 2 * RING, 512, generator=g, device=DEV).to(torch.float8_e4m3fn),
         "table": _page_table(g, b, pages),
         "out": torch.empty(rows, 64, 512, device=DEV, dtype=torch.bfloat16),
         "lse": torch.empty(rows, 64, device=DEV)}
    if own:
        import compressed_sparse_attention_append_b200 as csa

        s["cache"] = csa.PagedCache(b * pages, PAGE, b, pages, s["swa"].shape[1], indexer=False, page_table=s["table"],
                                    l_data=s["l_data"], l_scale=s["l_scale"], swa=s["swa"].view(torch.uint8))
    return s


# ---- one pass ---------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](state["case"], state)


def _own_linear(c, s):
    import compressed_sparse_attention_append_b200 as csa

    csa.csa2_fp8_quantize(s["x"], s["xq"], s["xs"])
    csa.csa2_fp8_gemm(s["xq"], s["xs"], s["w"], s["ws"], s["out"])
    return s["out"]


def _own_rope(c, s):
    import compressed_sparse_attention_append_b200 as csa

    csa.csa2_rope(s["rope"], s["pos"], s["x"], s["out"])
    return s["out"]


def _own_norm_rope(c, s):
    import compressed_sparse_attention_append_b200 as csa

    csa.csa2_norm_rope(s["rope"], s["pos"], EPS, s["q"], s["wq"], s["q_out"], s["k"], s["wk"], s["k_out"])
    return s["q_out"], s["k_out"]


def _own_append(c, s):
    import compressed_sparse_attention_append_b200 as csa

    csa.csa2_paged_append(s["cache"], c["b"], c["t"], s["pos"], s["latent"], s["key"], s["swa"], rope=s["rope"],
                          idx_rope=s["key_rope"], w_latent=s["w_latent"], w_idx_k=s["w_key"], w_swa=s["w_swa"],
                          eps=EPS, length=s["len"])
    csa.csa2_paged_gather(s["cache"], c["b"], s["rows"], s["latent_out"], s["key_out"])
    return s["latent_out"], s["key_out"], s["cache"].swa.view(torch.float8_e4m3fn)


def _own_attend(c, s):
    import compressed_sparse_attention_append_b200 as csa

    csa.csa2_paged_attend(s["cache"], c["b"], c["tq"], s["qpos"], s["q"], s["idx"], c["k"], s["out"], lse=s["lse"])
    return s["out"], s["lse"]


# ---- plain forms ------------------------------------------------------------------------------------
def _blocks(x, size):
    """The last axis padded with zeros to whole blocks: [..., blocks, size]."""
    pad = -x.shape[-1] % size
    return torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (-1, size))


def _plain_linear(c, s):
    m, k, n = c["m"], c["k"], c["n"]
    x = _blocks(s["x"].float(), 128)
    # (a quotient by a tensor: one by a number is a product with its rounded inverse, another scale)
    scale = x.abs().amax(-1, keepdim=True) / x.new_full((), 448.0)
    q = torch.where(scale > 0, x / scale, 0.0).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    x = (q * scale).flatten(1)[:, :k]
    ws = s["ws"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return (x @ (s["w"].float() * ws).T).to(s["out"].dtype)


def _rotate(x, pos, freq, offset, interleaved, mscale, inverse):
    """x [tokens, heads, d] rotated at its tokens' positions; angles in 64 bits."""
    half = freq.numel()
    a = pos.to(torch.float64)[:, None, None] * freq
    cos, sin = (torch.cos(a) * mscale).to(x.dtype), (torch.sin(a) * mscale).to(x.dtype)
    sin = -sin if inverse else sin
    r = x[..., offset:offset + 2 * half]
    u, v = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y = (u * cos - v * sin, v * cos + u * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([x[..., :offset], y, x[..., offset + 2 * half:]], -1)


def _plain_rope(c, s):
    y = _rotate(s["x"].float(), s["pos"], s["freq"], c["offset"], c["interleaved"], s["mscale"], c["inverse"])
    return y.to(s["x"].dtype)


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_norm_rope(c, s):
    turn = (s["pos"], s["freq"], c["offset"], c["interleaved"], s["mscale"], False)
    q = _rotate(_norm(s["q"].float(), s["wq"].float()), *turn)
    k = _rotate(_norm(s["k"].float(), s["wk"].float()), *turn)
    return q.to(s["q"].dtype), k.to(s["k"].dtype)


def _e4m3(x):
    """The nearest 8-bit value, decided in x's own precision (a cast goes through 32 bits first)."""
    step = torch.exp2((torch.frexp(x).exponent - 4).clamp(min=-9).to(x.dtype))
    return (torch.round(x / step) * step).clamp(-448, 448).to(torch.float8_e4m3fn)


def _e2m1(x):
    a = x.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, x)


def _plain_append(c, s):
    b, t = c["b"], c["t"]
    at = (s["pos"][:, None] + torch.arange(t, device=DEV)).flatten()
    # next to a rounding border of a 4-bit code 32 bits decide wrongly: norm, rotation and code in 64
    rows = lambda x, w, f, off: _rotate(_norm(x.double().flatten(0, 1), w.double())[:, None], at, f, off,  # noqa: E731
                                        c["interleaved"], 1.0, False).view(b, t, -1)
    latent = rows(s["latent"], s["w_latent"], s["freq"], 512 - c["rot"])
    key = rows(s["key"], s["w_key"], s["kfreq"], 64)
    swa = rows(s["swa"], s["w_swa"], s["freq"], 512 - c["rot"])
    there = (torch.arange(t, device=DEV) < s["len"][:, None])[..., None]
    x = _blocks(latent, 16)
    scale = _e4m3(x.abs().amax(-1, keepdim=True) / x.new_full((), 6.0)).double()
    latent = torch.where(scale > 0, _e2m1(x / scale) * scale, 0.0).flatten(-2)
    x = _blocks(key, 32)
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2((torch.frexp(top).exponent - 3).clamp(-127, 127).double())
    key = torch.where(top > 0, _e2m1(x / scale) * scale, 0.0).flatten(-2)
    # the ring keeps the latest RING tokens, position p in slot p % RING
    last = (s["pos"] + s["len"] - 1)[:, None]
    p = last - (last - torch.arange(RING, device=DEV)) % RING
    i = p - s["pos"][:, None]
    ring = torch.gather(swa, 1, i.clamp(0, t - 1)[..., None].expand(-1, -1, 512))
    ring = _e4m3(torch.where((i >= 0)[..., None], ring, 0.0))
    return torch.where(there, latent, 0.0).to(torch.bfloat16), torch.where(there, key, 0.0).to(torch.bfloat16), ring


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _attend_keys(c, s, dtype):
    """The rows' keys [rows, k + 128, 512] (selected entries, then the window) and which of them count."""
    b = torch.arange(c["b"] * c["tq"], device=DEV) // c["tq"]
    idx = s["idx"].long().clamp_min(0)
    at = s["table"][b[:, None], idx // PAGE].long() * PAGE + idx % PAGE
    codes = s["l_data"].flatten(0, 1)[at]
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    scale = s["l_scale"].flatten(0, 1)[at].view(torch.float8_e4m3fn).to(dtype)
    picked = torch.tensor(E2M1, device=DEV, dtype=dtype)[codes] * scale.repeat_interleave(16, -1)
    p = s["qpos"][:, None] - torch.arange(128, device=DEV)
    window = s["swa"][b[:, None], p % s["swa"].shape[1]].to(dtype)
    return torch.cat([picked, window], 1), torch.cat([s["idx"] >= 0, p >= 0], 1)


def _plain_attend(c, s):
    keys, there = _attend_keys(c, s, torch.float32)
    logits = s["q"].float() @ keys.transpose(1, 2) / math.sqrt(512)
    logits = logits.masked_fill(~there[:, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    return (p @ keys / total).to(torch.bfloat16), (top + torch.log(total))[..., 0]


# ---- what the bytes and operations cannot be without --------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        m, k, n = c["m"], c["k"], c["n"]
        scales = 4 * -(-n // 128) * -(-k // 128)
        return {"bytes": 2 * m * k + n * k + scales + m * n * (2 if c["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if c["op"] in ("rope", "norm_rope"):
        size = 2 if c["dtype"] == "bf16" else 4
        heads = c["heads"] if c["op"] == "rope" else c["hq"] + c["hk"]
        n = c["t"] * heads * c["d"]
        return {"bytes": 2 * n * size + 8 * c["t"] + 4 * c["rot"],
                "flops": 3 * c["t"] * heads * c["rot"] + (0 if c["op"] == "rope" else 4 * n)}
    if c["op"] == "append":
        # rows in, codes and window rows out, and the entries read back as values
        n = c["b"] * c["t"]
        return {"bytes": n * (2304 + 288 + 68 + 288 + 68 + 1280) + c["b"] * min(c["t"], RING) * 512,
                "flops": n * 1152 * 8}
    rows = c["b"] * c["tq"]
    keys = c["k"] + min(128, c["n"])
    return {"bytes": rows * (c["k"] * 288 + 4 * c["k"] + 2 * 65536 + 256) + c["b"] * min(128 + c["tq"], c["n"]) * 512,
            "flops": 4 * rows * 64 * 512 * keys}


# ---- the definitions in 64 bits -----------------------------------------------------------------------
def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, prepare(case, seed))


def _nearest(x, table):
    """x rounded to the nearest of +-table (ascending, from 0), a tie to the even place, beyond it to its end."""
    table = torch.as_tensor(table, device=DEV, dtype=torch.float64)
    mid = (table[1:] + table[:-1]) / 2
    a = x.abs().contiguous()
    at = torch.bucketize(a, mid)
    tie = (a == mid[at.clamp(max=mid.numel() - 1)]) & (at < mid.numel()) & (at % 2 == 1)
    return torch.copysign(table[at + tie], x)


def _e4m3_table():
    return torch.arange(127, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def _exact_linear(c, s):
    m, k, n = c["m"], c["k"], c["n"]
    out = torch.zeros(m, n, device=DEV, dtype=torch.float64)
    for j, k0 in enumerate(range(0, k, 128)):
        x = s["x"][:, k0:k0 + 128].double()
        # the scale is a 32-bit number, and the code is that of the 32-bit quotient
        scale = (x.abs().amax(1, keepdim=True).float() / torch.tensor(448.0, device=DEV)).double()
        code = _nearest((x / scale).nan_to_num(0.0).float().double(), _e4m3_table())
        w = s["w"][:, k0:k0 + 128].double() * s["ws"][:, j].double().repeat_interleave(128)[:n, None]
        out += (code * scale) @ w.T
    return out


def _turn(x, pos, freq, offset, interleaved, mscale, inverse):
    n = freq.numel()
    z = torch.polar(torch.full((), mscale, device=DEV, dtype=torch.float64),
                    pos.double()[:, None] * (-freq if inverse else freq))[:, None]
    out = x.double().clone()
    r = x[..., offset:offset + 2 * n].double()
    r = torch.view_as_complex(r.unflatten(-1, (n, 2)).contiguous()) if interleaved else torch.complex(r[..., :n], r[..., n:])
    r = r * z
    out[..., offset:offset + 2 * n] = torch.view_as_real(r).flatten(-2) if interleaved else torch.cat([r.real, r.imag], -1)
    return out


def _exact_rope(c, s):
    return _turn(s["x"], s["pos"], s["freq"], c["offset"], c["interleaved"], s["mscale"], c["inverse"])


def _scaled(x, w):
    x = x.double()
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()


def _exact_norm_rope(c, s):
    turn = (s["pos"], s["freq"], c["offset"], c["interleaved"], s["mscale"], False)
    return _turn(_scaled(s["q"], s["wq"]), *turn), _turn(_scaled(s["k"], s["wk"]), *turn)


def _exact_append(c, s):
    b, t = c["b"], c["t"]
    latent_out = torch.zeros(b, t, 512, device=DEV, dtype=torch.float64)
    key_out = torch.zeros(b, t, 128, device=DEV, dtype=torch.float64)
    ring = torch.zeros(b, RING, 512, device=DEV, dtype=torch.float64)
    table = _e4m3_table()
    for j, n in enumerate(s["len"].tolist()):
        if not n:
            continue
        pos = s["pos"][j] + torch.arange(n, device=DEV)
        one = lambda x, w, f, off: _turn(_scaled(x[j, :n, None], w), pos, f, off, c["interleaved"], 1.0, False)[:, 0]  # noqa: E731
        x = one(s["latent"], s["w_latent"], s["freq"], 512 - c["rot"]).view(n, 32, 16)
        scale = _nearest(x.abs().amax(-1, keepdim=True) / 6, table)
        latent_out[j, :n] = ((_nearest(x / scale, E2M1[:8])).nan_to_num(0.0) * scale).flatten(1)
        x = one(s["key"], s["w_key"], s["kfreq"], 64).view(n, 4, 32)
        scale = torch.exp2(torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))) - 2)
        key_out[j, :n] = (_nearest(x / scale, E2M1[:8]) * scale).flatten(1)
        x = _nearest(one(s["swa"], s["w_swa"], s["freq"], 512 - c["rot"]), table)
        keep = min(n, RING)
        ring[j, pos[-keep:] % RING] = x[-keep:]
    return latent_out, key_out, ring


def _exact_attend(c, s):
    out, lse = [], []
    for r in range(c["b"] * c["tq"]):
        j, p = r // c["tq"], int(s["qpos"][r])
        e = s["idx"][r][s["idx"][r] >= 0].long()
        page, slot = s["table"][j][e // PAGE].long(), e % PAGE
        codes = s["l_data"][page, slot].long()
        value = torch.tensor(E2M1, device=DEV, dtype=torch.float64)
        keys = torch.empty(e.numel(), 512, device=DEV, dtype=torch.float64)
        keys[:, 0::2], keys[:, 1::2] = value[codes % 16], value[codes // 16]
        keys = (keys.view(-1, 32, 16) * s["l_scale"][page, slot].view(torch.float8_e4m3fn).double()[..., None]).flatten(1)
        window = torch.arange(max(0, p - 127), p + 1, device=DEV)
        keys = torch.cat([keys, s["swa"][j, window % s["swa"].shape[1]].double()])
        logits = s["q"][r].double() @ keys.T / math.sqrt(512)
        lse.append(torch.logsumexp(logits, -1))
        out.append(torch.softmax(logits, -1) @ keys)
    return torch.stack(out), torch.stack(lse)
