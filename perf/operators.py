"""The serving operators around the indexer and its consumer, as they are timed and compared.

Four operators: the rotation of queries and keys by their positions; the norm of each head with that
rotation in the same pass; latent rows written into a 4-bit paged cache and read back; attention over the
selected rows of that cache.  `run` computes each in plain torch (fp32, rounded once at the end) or, with
`own`, through the library.

The 4-bit record of one latent row (512 latent + 64 positional features), 416 bytes:
  [0, 256)    512 codes n in -7..7, two's complement nibbles.  The 32-bit little-endian word i holds
              features 8i .. 8i+7: the even ones in its low half, the odd ones in its high half, each half
              from its lowest nibble up.
  [256, 288)  32 scale codes c, one for each 16 features: s = (1 + (c & 7) / 8) * 2^((c >> 3) - 20), the
              smallest such value with 7 s >= max|x| of the group; n = x / s to the nearest, ties to even.
  [288, 416)  the 64 positional features in bf16.
A value reads back as n * s, which bf16 holds exactly.
"""
import math

import torch

own = False

LATENT, ROPE, WIDTH, GROUP, RECORD = 512, 64, 576, 16, 416
SCALE = 192 ** -0.5


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 sequences: the indexer's 64 query heads, half of each head rotated
        {"name": "rotary_decode_64", "op": "rotary", "tokens": 64, "heads": 64, "dim": 128, "rot": 64, "offset": 0,
         "interleaved": False, "dtype": "bf16", "last": 131072, "factor": 1.0},
        # the indexer's queries of a whole 32K prompt
        {"name": "rotary_prefill_32k", "op": "rotary", "tokens": 32768, "heads": 64, "dim": 128, "rot": 64, "offset": 0,
         "interleaved": True, "dtype": "bf16", "last": 32767, "factor": 1.0},
        # one decode step's new indexer keys: layer norm and rotation of one row for each sequence
        {"name": "norm_rotary_decode_64", "op": "norm_rotary", "tokens": 64, "heads": 1, "dim": 128, "norm": "layer",
         "norm_dim": 128, "rot": 64, "offset": 0, "interleaved": True, "dtype": "bf16", "last": 131072, "factor": 1.0,
         "gap": 0},
        # the latent rows of a 32K prompt cut out of a wider projection: norm of the 512 latent features, rotation
        # of the 64 positional ones at positions scaled for a long context
        {"name": "norm_rotary_latent_32k", "op": "norm_rotary", "tokens": 32768, "heads": 1, "dim": 576, "norm": "rms",
         "norm_dim": 512, "rot": 64, "offset": 512, "interleaved": True, "dtype": "bf16", "last": 163840, "factor": 40.0,
         "gap": 192},
        # fp32 queries of a ragged batch, the whole head normed and rotated
        {"name": "norm_rotary_heads_fp32", "op": "norm_rotary", "tokens": 4099, "heads": 40, "dim": 128, "norm": "rms",
         "norm_dim": 128, "rot": 128, "offset": 0, "interleaved": False, "dtype": "f32", "last": 8191, "factor": 1.0,
         "gap": 0},
        # one decode step's rows written to the cache and read back
        {"name": "kv4_write_read_64", "op": "write_read", "rows": 64, "page": 64, "pages": 4096, "skip": False},
        # a 64K prompt (not a whole number of pages, some rows padding) written and read back
        {"name": "kv4_write_read_64k", "op": "write_read", "rows": 65519, "page": 64, "pages": 1100, "skip": True},
        # a cached 128K prefix read back to bf16
        {"name": "kv4_read_128k", "op": "read", "rows": 131072, "page": 128, "pages": 1100},
        # one new token of one sequence: latency
        {"name": "attend_decode_1", "op": "attend", "batch": 1, "queries": 1, "heads": 128, "keys": 131072, "top_k": 2048,
         "page": 64, "ragged": False},
        # the decode step of 64 sequences at 128K
        {"name": "attend_decode_64", "op": "attend", "batch": 64, "queries": 1, "heads": 128, "keys": 131072,
         "top_k": 2048, "page": 64, "ragged": False},
        # a ragged batch with one eighth of the heads, two tokens for each sequence, some shorter than the
        # selection and some empty
        {"name": "attend_ragged_16h", "op": "attend", "batch": 23, "queries": 2, "heads": 16, "keys": 5000, "top_k": 1500,
         "page": 64, "ragged": True},
        # 1024 queries of a prefill chunk over a 64K prefix
        {"name": "attend_chunk_64k", "op": "attend", "batch": 1, "queries": 1024, "heads": 128, "keys": 65536,
         "top_k": 2048, "page": 128, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "norm_rotary", "write_read", "read", "attend", "attend"])
    if op == "rotary":
        dim = rng.choice([64, 80, 128, 192, 576])
        rot = dim if dim <= 128 and rng.random() < 0.4 else 64
        heads = rng.choice([1, 3, 16, 40, 64, 128])
        return {"op": op, "tokens": _log(rng, 1, 32768 * 8192 // (heads * dim)), "heads": heads, "dim": dim, "rot": rot,
                "offset": rng.choice([0, dim - rot]), "interleaved": rng.random() < 0.5,
                "dtype": "bf16", "last": _log(rng, 100, 1000000), "factor": rng.choice([1.0, 4.0, 40.0])}
    if op == "norm_rotary":
        heads, dim = rng.choice([(1, 128), (1, 576), (5, 64), (8, 128), (40, 128), (64, 128), (128, 192)])
        rot = dim if dim <= 128 and rng.random() < 0.5 else 64
        norm_dim = 512 if dim == 576 else dim
        return {"op": op, "tokens": _log(rng, 1, 4099 * 40 * 128 // (heads * dim)), "heads": heads, "dim": dim,
                "norm": rng.choice(["rms", "layer"]), "norm_dim": norm_dim, "rot": rot, "offset": rng.choice([0, dim - rot]),
                "interleaved": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f32"]),
                "last": _log(rng, 100, 1000000), "factor": rng.choice([1.0, 4.0, 40.0]), "gap": rng.choice([0, 64, 192])}
    if op in ("write_read", "read"):
        page = rng.choice([1, 16, 64, 128])
        rows = _log(rng, 1, 65519)
        case = {"op": op, "rows": rows, "page": page, "pages": -(-rows // page) + rng.randint(1, 200)}
        return dict(case, skip=rng.random() < 0.5) if op == "write_read" else case
    heads = rng.choice([1, 8, 16, 32, 64, 96, 128, 128, 256])
    top_k = _log(rng, 1, 4096)
    batch = _log(rng, 1, 64)
    queries = _log(rng, 1, max(1, min(1024, 1024 * 128 * 2048 // (batch * max(128, heads) * max(256, top_k)))))
    return {"op": op, "batch": batch, "queries": queries, "heads": heads, "keys": _log(rng, 64, 65536), "top_k": top_k,
            "page": rng.choice([16, 64, 128]), "ragged": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _inv_freq(rot, factor):
    """Radians per position of each pair, base 10000; with factor > 1 the pairs that turn less than once over
    4096 positions are slowed by it, those that turn over 32 times are kept, with a ramp between."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if factor > 1:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns.log() - math.log(1.0)) / (math.log(32.0) - math.log(1.0))).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f, 1.0 if factor <= 1 else 0.1 * math.log(factor) + 1.0


def _pack(x):
    """Records [n, 416] (uint8) of rows x [n, 576] (bf16)."""
    lat = x[:, :LATENT].float().view(-1, LATENT // GROUP, GROUP)
    mant, expo = torch.frexp(lat.abs().amax(-1).double() / 7)
    code = (expo - 1 + 20) * 8 + (torch.ceil(mant * 16) - 8).to(torch.int32)
    code = torch.where(mant == 0, torch.zeros_like(code), code).clamp(0, 255)
    n = torch.round(lat / _scale(code)[..., None]).clamp(-7, 7).to(torch.int32) & 15
    n = n.view(-1, LATENT // 8, 8)
    b = torch.stack([n[..., 0] | n[..., 2] << 4, n[..., 4] | n[..., 6] << 4,
                     n[..., 1] | n[..., 3] << 4, n[..., 5] | n[..., 7] << 4], -1)
    return torch.cat([b.view(-1, LATENT // 2).to(torch.uint8), code.to(torch.uint8),
                      x[:, LATENT:].contiguous().view(torch.uint8)], 1)


def _scale(code):
    return torch.ldexp(1 + (code & 7).float() / 8, (code >> 3) - 20)


def _unpack(rec):
    """The rows (fp32 [..., 576]) that records (uint8 [..., 416]) stand for."""
    lead = rec.shape[:-1]
    b = rec[..., :256].reshape(*lead, LATENT // 8, 4).to(torch.int32)
    n = torch.stack([b[..., 0] & 15, b[..., 2] & 15, b[..., 0] >> 4, b[..., 2] >> 4,
                     b[..., 1] & 15, b[..., 3] & 15, b[..., 1] >> 4, b[..., 3] >> 4], -1)
    n = ((n ^ 8) - 8).float().view(*lead, LATENT // GROUP, GROUP)
    lat = (n * _scale(rec[..., 256:288].to(torch.int32))[..., None]).view(*lead, LATENT)
    pos = rec[..., 288:].contiguous().view(torch.bfloat16).float()
    return torch.cat([lat, pos], -1)


def _latent_rows(n, g):
    """Latent rows as the norm and the rotation leave them: unit size, some channels larger than others."""
    x = _randn((n, WIDTH), g)
    return (x * torch.exp(0.3 * _randn((1, WIDTH), g))).to(torch.bfloat16)


def _filled_cache(pages, page, g):
    rec = torch.empty((pages * page, RECORD), dtype=torch.uint8, device="cuda")
    for r0 in range(0, pages * page, 1 << 18):
        part = rec[r0:r0 + (1 << 18)]
        part.copy_(_pack(_latent_rows(part.shape[0], g)))
    return rec.view(pages, page, RECORD)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("rotary", "norm_rotary"):
        T, H, d = case["tokens"], case["heads"], case["dim"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide = torch.empty((T, H * d + case.get("gap", 0)), dtype=dt, device="cuda")
        for t0 in range(0, T, 4096):
            wide[t0:t0 + 4096] = _randn(wide[t0:t0 + 4096].shape, g)
        f, amp = _inv_freq(case["rot"], case["factor"])
        st = {"case": case, "x": wide[:, :H * d].view(T, H, d), "inv_freq": f, "amplitude": amp,
              "positions": torch.randint(0, case["last"] + 1, (T,), generator=g, device="cuda", dtype=torch.int32)}
        if op == "norm_rotary":
            st["weight"] = 1 + 0.1 * _randn((case["norm_dim"],), g)
            st["bias"] = 0.1 * _randn((case["norm_dim"],), g) if case["norm"] == "layer" else None
        return st
    if op in ("write_read", "read"):
        n, page, pages = case["rows"], case["page"], case["pages"]
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(torch.int32)
        if op == "read":
            return {"case": case, "cache": _filled_cache(pages, page, g), "slots": slots}
        if case["skip"]:
            slots[torch.rand(n, generator=g, device="cuda") < 0.02] = -1
        return {"case": case, "rows": _latent_rows(n, g), "slots": slots,
                "cache": torch.zeros((pages, page, RECORD), dtype=torch.uint8, device="cuda")}
    B, Q, H, L, K, page = (case[k] for k in ("batch", "queries", "heads", "keys", "top_k", "page"))
    per = -(-L // page)
    cache = _filled_cache(B * per, page, g)
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    idx = torch.full((B, Q, K), -1, dtype=torch.int32, device="cuda")
    seen = torch.full((B,), L, device="cuda")
    if case["ragged"]:  # lengths from none to all
        seen = (torch.rand(B, generator=g, device="cuda") ** 2 * (L + 1)).long().clamp(0, L)
        seen[0] = 0
    step = max(1, (1 << 26) // L)
    flat, seen = idx.view(B * Q, K), seen.repeat_interleave(Q)
    for r0 in range(0, B * Q, step):  # distinct positions of each row's visible prefix, in random order
        s = seen[r0:r0 + step, None]
        u = torch.rand((s.shape[0], L), generator=g, device="cuda")
        u.masked_fill_(torch.arange(L, device="cuda") >= s, -1.0)
        v, at = u.topk(min(K, L), dim=1)
        flat[r0:r0 + step, :min(K, L)] = torch.where(v >= 0, at, torch.full_like(at, -1)).to(torch.int32)
    return {"case": case, "cache": cache, "page_table": table, "idx": idx,
            "q": _randn((B, Q, H, WIDTH), g).to(torch.bfloat16)}


# ----------------------------------------------------------------- one pass

def _rotated(y, positions, inv_freq, amp, rot, offset, interleaved):
    """y [T, H, d] fp32 with its features [offset, offset + rot) rotated."""
    ang = positions.double()[:, None] * inv_freq
    c, s = (torch.cos(ang) * amp).float()[:, None], (torch.sin(ang) * amp).float()[:, None]
    part = y[..., offset:offset + rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        new = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        new = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y[..., :offset], new, y[..., offset + rot:]], -1)


def run(state):
    case = state["case"]
    if own:
        from hierarchical_top_key_b200 import binding as hb
    if case["op"] == "rotary":
        if own:
            return hb.hisa_rotary(state["x"], state["positions"], state["inv_freq"], offset=case["offset"],
                                  interleaved=case["interleaved"], amplitude=state["amplitude"])
        return _rotated(state["x"].float(), state["positions"], state["inv_freq"], state["amplitude"], case["rot"],
                        case["offset"], case["interleaved"]).to(state["x"].dtype)
    if case["op"] == "norm_rotary":
        nd = case["norm_dim"]
        if own:
            return hb.hisa_norm_rotary(state["x"], state["positions"], state["inv_freq"], weight=state["weight"],
                                       bias=state["bias"], norm=case["norm"], eps=1e-6, norm_dim=nd,
                                       offset=case["offset"], interleaved=case["interleaved"],
                                       amplitude=state["amplitude"])
        x = state["x"].float()
        y = x[..., :nd]
        if case["norm"] == "layer":
            y = y - y.mean(-1, keepdim=True)
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * state["weight"]
        if case["norm"] == "layer":
            y = y + state["bias"]
        return _rotated(torch.cat([y, x[..., nd:]], -1), state["positions"], state["inv_freq"], state["amplitude"],
                        case["rot"], case["offset"], case["interleaved"]).to(state["x"].dtype)
    if case["op"] in ("write_read", "read"):
        cache, slots = state["cache"], state["slots"]
        if own:
            if case["op"] == "write_read":
                hb.hisa_kv4_write(state["rows"], slots, cache)
            return hb.hisa_kv4_read(cache, slots)
        rec = cache.view(-1, RECORD)
        live = slots >= 0
        if case["op"] == "write_read":
            new = _pack(state["rows"])
            rec[slots[live].long()] = new[live]
        return (_unpack(rec[slots.clamp(min=0).long()]) * live[:, None]).to(torch.bfloat16)
    if own:
        return hb.hisa_sparse_attention_kv4(state["q"], state["cache"], state["page_table"], state["idx"], scale=SCALE,
                                            num_keys=case["keys"])
    idx, page = state["idx"].long(), case["page"]
    live = idx >= 0
    at = idx.clamp(min=0)
    batch = torch.arange(case["batch"], device=idx.device)[:, None, None]
    slot = state["page_table"].long()[batch, at // page] * page + at % page
    kv = _unpack(state["cache"].view(-1, RECORD)[slot])
    logit = torch.matmul(state["q"].float(), kv.transpose(-1, -2)) * SCALE
    logit = logit.masked_fill(~live[:, :, None, :], -math.inf)
    top = logit.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(logit - top)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, kv[..., :LATENT]) / z.clamp(min=torch.finfo(torch.float32).tiny)
    return o.to(torch.bfloat16), (top + torch.log(z))[..., 0]


def work(case):
    if case["op"] in ("rotary", "norm_rotary"):
        n = case["tokens"] * case["heads"] * case["dim"] * (2 if case["dtype"] == "bf16" else 4)
        small = 4 * case["tokens"] + 4 * case["rot"]
        if case["op"] == "rotary":
            return {"bytes": 2 * n + small, "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
        return {"bytes": 2 * n + small + 8 * case["norm_dim"],
                "flops": case["tokens"] * case["heads"] * (3 * case["rot"] + 5 * case["norm_dim"])}
    if case["op"] == "read":
        return {"bytes": case["rows"] * (4 + RECORD + 2 * WIDTH), "flops": case["rows"] * LATENT}
    if case["op"] == "write_read":
        return {"bytes": case["rows"] * (8 + 2 * RECORD + 4 * WIDTH), "flops": case["rows"] * 4 * LATENT}
    rows, H = case["batch"] * case["queries"], case["heads"]
    n = min(case["top_k"], case["keys"])
    # of a ragged batch's rows a third of the keys are visible in the mean, and a selection is no longer than that
    keys = int(rows * n * (_ragged_share(n, case["keys"]) if case["ragged"] else 1.0))
    return {"bytes": min(case["batch"] * case["keys"], keys) * RECORD + rows * (H * (2 * WIDTH + 2 * LATENT + 4) + 4 * case["top_k"]),
            "flops": 2 * H * keys * (WIDTH + LATENT)}


def _ragged_share(n, keys):
    """Mean of min(n, visible) / n for visible = u^2 keys, u uniform."""
    r = n / keys
    return 1 - math.sqrt(r) + r ** 0.5 / 3 if r < 1 else 1 / 3


# ----------------------------------------------------------------- from the definitions, in 64 bits

def _exact_rotation(y, state, case):
    T = y.shape[0]
    half = case["rot"] // 2
    ang = state["positions"].double().reshape(T, 1) * state["inv_freq"].reshape(1, half)
    turn = torch.polar(torch.full_like(ang, state["amplitude"]), ang)
    out = y.clone()
    o = case["offset"]
    part = out[:, :, o:o + case["rot"]]
    if case["interleaved"]:
        pair = part.reshape(T, -1, half, 2).contiguous()
        part.copy_(torch.view_as_real(torch.view_as_complex(pair) * turn[:, None]).reshape(part.shape))
    else:
        pair = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn[:, None]
        part.copy_(torch.cat([pair.real, pair.imag], -1))
    return out


def _exact_row(x):
    """What a row [n, 576] (float64) reads back as, from the definition of the format."""
    out = x.clone()
    groups = out[:, :LATENT].reshape(-1, GROUP)
    grid = torch.tensor([(1 + m / 8) * 2.0 ** (e - 20) for e in range(32) for m in range(8)], dtype=torch.float64,
                        device=x.device)
    s = grid[torch.searchsorted(7 * grid, groups.abs().amax(1)).clamp(max=255)][:, None]
    out[:, :LATENT] = (torch.round(groups / s).clamp(-7, 7) * s).reshape(-1, LATENT)
    return out


def _exact_record(rec):
    """Rows (float64) of records, nibble by nibble."""
    r = rec.to(torch.int64)
    out = torch.empty((r.shape[0], WIDTH), dtype=torch.float64, device=rec.device)
    place = [(0, 0), (2, 0), (0, 4), (2, 4), (1, 0), (3, 0), (1, 4), (3, 4)]  # byte of the word, shift, by feature mod 8
    for f, (byte, shift) in enumerate(place):
        n = r[:, byte:256:4] >> shift & 15
        out[:, f:LATENT:8] = torch.where(n > 7, n - 16, n).double()
    c = r[:, 256:288].repeat_interleave(GROUP, dim=1)
    out[:, :LATENT] *= (8 + c % 8).double() * torch.pow(2.0, (c // 8 - 23).double())
    out[:, LATENT:] = rec[:, 288:].contiguous().view(torch.bfloat16).double()
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotation(state["x"].double(), state, case)
    if case["op"] == "norm_rotary":
        x = state["x"].double()
        n = case["norm_dim"]
        y = x[..., :n]
        mean = y.sum(-1, keepdim=True) / n if case["norm"] == "layer" else torch.zeros_like(y[..., :1])
        var = ((y - mean) ** 2).sum(-1, keepdim=True) / n
        x = x.clone()
        x[..., :n] = (y - mean) / torch.sqrt(var + 1e-6) * state["weight"].double()
        if case["norm"] == "layer":
            x[..., :n] += state["bias"].double()
        return _exact_rotation(x, state, case)
    if case["op"] in ("write_read", "read"):
        slots = state["slots"].long()
        if case["op"] == "read":
            return _exact_record(state["cache"].reshape(-1, RECORD)[slots])
        rows = _exact_row(state["rows"].double())
        rows[slots < 0] = 0
        return rows
    B, Q, H = case["batch"], case["queries"], case["heads"]
    o = torch.zeros((B, Q, H, LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    rec = state["cache"].reshape(-1, RECORD)
    for b in range(B):
        for t in range(Q):
            s = state["idx"][b, t]
            s = s[s >= 0].long()
            if not s.numel():
                continue
            kv = _exact_record(rec[state["page_table"][b, s // case["page"]].long() * case["page"] + s % case["page"]])
            logit = SCALE * (state["q"][b, t].double() @ kv.T)
            lse[b, t] = torch.logsumexp(logit, -1)
            o[b, t] = torch.exp(logit - lse[b, t][:, None]) @ kv[:, :LATENT]
    return o, lse
