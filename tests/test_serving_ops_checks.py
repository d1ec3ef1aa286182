"""Rotary, head norms, the 4-bit latent cache and attention over it, without a
GPU: argument checks (all made before any launch), the frequencies, and the
cache oracle against its definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

from hierarchical_top_key_b200 import binding as hb
from oracle import latent_cache as lc

f32 = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    return hb.load()


def _rot(L, **kw):
    a = dict(x=0x1000, xt=128, xh=128, pos=0x2000, f=0x3000, tokens=4, heads=1, dim=128, rot=64, offset=0, inter=0,
             rev=0, amp=f32(1.0), dt=hb.HISA_BF16, out=0x9000, ot=128, oh=128)
    a.update(kw)
    return L.hisa_rotary(*(a[k] for k in ("x", "xt", "xh", "pos", "f", "tokens", "heads", "dim", "rot", "offset",
                                          "inter", "rev", "amp", "dt", "out", "ot", "oh")), None)


def _norm(L, **kw):
    a = dict(x=0x1000, xt=128, xh=128, pos=0x2000, f=0x3000, tokens=4, heads=1, dim=128, norm=1, nd=128, w=0x4000,
             b=None, eps=f32(1e-6), rot=64, offset=0, inter=0, amp=f32(1.0), dt=hb.HISA_F32, out=0x9000, ot=128, oh=128)
    a.update(kw)
    return L.hisa_norm_rotary(*(a[k] for k in ("x", "xt", "xh", "pos", "f", "tokens", "heads", "dim", "norm", "nd", "w",
                                               "b", "eps", "rot", "offset", "inter", "amp", "dt", "out", "ot", "oh")),
                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=hb.HISA_E4M3), 2), (dict(dim=1025), 2), (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(rot=63), 1),
    (dict(rot=0), 1), (dict(offset=65), 1), (dict(offset=-1), 1), (dict(rot=130), 1), (dict(ot=127), 1),
    (dict(heads=2, oh=64, ot=256), 1), (dict(xt=-128), 1), (dict(out=0x1000, xt=256), 1), (dict(x=None), 1),
    (dict(pos=None), 1), (dict(f=0x3004), 1), (dict(x=0x1001), 1), (dict(pos=0x2002), 1),
    (dict(amp=f32(float("nan"))), 1), (dict(tokens=0, x=None, out=None, pos=None), 0)])
def test_rotary_arguments(L, kw, status):
    assert _rot(L, **kw) == status


@pytest.mark.parametrize("kw", [
    dict(heads=2, ot=128, oh=128),                  # token 1's head 0 is token 0's head 1
    dict(heads=3, ot=192, oh=128), dict(heads=2, tokens=3, ot=128, oh=256),
    dict(heads=4, tokens=2, ot=511, oh=128)])
def test_rotary_refuses_rows_of_out_that_overlap(L, kw):
    assert _rot(L, **kw) == 1 and _norm(L, **kw) == 1


def test_rotary_refuses_more_rows_than_it_can_count(L):
    assert _rot(L, heads=4, tokens=1 << 62, ot=1 << 20) == 2
    assert _rot(L, heads=2, tokens=1 << 62, ot=1 << 62, oh=1 << 62, rot=63) == 2     # 2^63 rows


@pytest.mark.parametrize("kw,status", [
    (dict(norm=0), 1), (dict(norm=3), 1), (dict(nd=0), 1), (dict(nd=129), 1), (dict(b=0x5000), 1),
    (dict(w=None), 1), (dict(eps=f32(-1.0)), 1), (dict(eps=f32(float("inf"))), 1), (dict(w=0x4002), 1),
    (dict(x=0x1002), 1), (dict(norm=2, b=0x5002), 1), (dict(tokens=0), 0)])
def test_norm_rotary_arguments(L, kw, status):
    assert _norm(L, **kw) == status


def test_cache_row_arguments(L):
    ok = dict(rows=0x1000, stride=576, slots=0x2000, n=4, cache=0x4000, num=64)

    def both(**kw):
        a = dict(ok, **kw)
        w = L.hisa_kv4_write(a["rows"], a["stride"], a["slots"], a["n"], a["cache"], a["num"], None)
        r = L.hisa_kv4_read(a["cache"], a["num"], a["slots"], a["n"], a["rows"], a["stride"], None)
        assert w == r
        return w
    assert both(stride=568) == 1 and both(stride=577) == 1 and both(n=-1) == 1 and both(num=0) == 1
    assert both(num=1 << 31) == 1 and both(rows=0x1008) == 1 and both(cache=0x4008) == 1 and both(slots=0x2002) == 1
    assert both(rows=None) == 1 and both(slots=None) == 1 and both(cache=None) == 1
    assert both(n=0, rows=None, slots=None) == 0


def test_attention_arguments(L):
    ok = dict(q=0x1000, cache=0x2000, pages=8, page=64, table=0x3000, idx=0x4000, batch=1, Q=4, L=100, H=128, k=64,
              scale=f32(0.07), o=0x5000, lse=0x6000, ws=None, wsb=0)

    def call(**kw):
        a = dict(ok, **kw)
        return L.hisa_sparse_attention_kv4(*(a[k] for k in ("q", "cache", "pages", "page", "table", "idx", "batch", "Q",
                                                            "L", "H", "k", "scale", "o", "lse", "ws", "wsb")), None)
    assert call(H=0) == 1 and call(batch=0) == 1 and call(Q=0) == 1 and call(L=0) == 1
    assert call(pages=0) == 1 and call(page=0) == 1 and call(pages=1 << 20, page=1 << 12) == 2
    assert call(k=0) == 2 and call(k=4097) == 2 and call(scale=f32(float("nan"))) == 1
    for name in ("q", "cache", "table", "idx", "o", "lse"):
        assert call(**{name: None}) == 1, name
    assert call(q=0x1008) == 1 and call(cache=0x2008) == 1 and call(idx=0x4002) == 1 and call(table=0x3002) == 1
    assert call(o=0x5008) == 1 and call(lse=0x6002) == 1 and call(ws=0x7008, wsb=1 << 20) == 3
    assert call(batch=1 << 20, Q=1 << 20) == 2
    assert call() == 3 and call(ws=0x7000, wsb=64 * 4 + 3) == 3


def test_attention_workspace_rule(L):
    def size(**kw):
        s = dict(batch=1, num_keys=1000, num_queries=1, heads=128, head_dim=0, block_size=0, top_m=0, top_k=2048,
                 dtype=hb.HISA_BF16)
        s.update(kw)
        return hb.workspace_size(hb.OP_ATTENTION_KV4, hb.Shape(**s))
    # a record list and its length for each query; parts' outputs only where there are few queries and keys to split
    assert size(num_queries=4096) == 4096 * (2048 * 4 + 4)
    assert size(top_k=64) == 64 * 4 + 4 and size(top_k=1) == 4 * 4 + 4
    one = size() - (2048 * 4 + 4)
    assert one > 0 and one % (128 * 513 * 4) == 0 and 2 <= one // (128 * 513 * 4) <= 32
    n = ctypes.c_size_t(0)
    for bad, status in ((dict(heads=0), 1), (dict(batch=0), 1), (dict(top_k=4097), 2)):
        s = dict(batch=1, num_keys=1000, num_queries=1, heads=128, head_dim=0, block_size=0, top_m=0, top_k=2048, dtype=1)
        s.update(bad)
        assert L.hisa_workspace_size(hb.OP_ATTENTION_KV4, ctypes.byref(hb.Shape(**s)), ctypes.byref(n)) == status


def test_binding_refuses_host_and_wrong_tensors():
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        hb.hisa_rotary(x, pos, f)
    with pytest.raises(ValueError):
        hb.hisa_norm_rotary(x, pos, f, weight=torch.ones(128))
    cache, rows = torch.zeros((2, 8, 416), dtype=torch.uint8), torch.zeros((4, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hb.hisa_kv4_write(rows, pos, cache)
    with pytest.raises(ValueError):
        hb.hisa_kv4_read(cache, pos)
    with pytest.raises(ValueError):
        hb.hisa_sparse_attention_kv4(torch.zeros((1, 1, 128, 576), dtype=torch.bfloat16), cache,
                                     torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1, 1, 4), dtype=torch.int32),
                                     scale=1.0, num_keys=16)


def test_inv_freq():
    f, a = hb.rotary_inv_freq(8, base=10000.0, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64
    np.testing.assert_allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    g, a = hb.rotary_inv_freq(8, scaling="linear", factor=4.0, device="cpu")
    np.testing.assert_allclose(g.numpy(), f.numpy() / 4, rtol=1e-15)
    g, a = hb.rotary_inv_freq(8, scaling="ntk", factor=16.0, device="cpu")
    assert g[0] == 1.0 and abs(float(g[-1] / f[-1]) * 16 - 1) < 1e-12
    # the ramp keeps the fast pairs, slows the slow ones by the factor and is monotone between
    f, _ = hb.rotary_inv_freq(64, device="cpu")
    g, a = hb.rotary_inv_freq(64, scaling="ramp", factor=40.0, original_positions=4096, device="cpu")
    r = (f / g).numpy()
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert np.all(np.abs(r[turns > 40] - 1) < 1e-12) and np.all(np.abs(r[turns < 0.7] - 40) < 1e-9)
    assert np.all(np.diff(r) >= -1e-12) and abs(a - (0.1 * math.log(40) + 1)) < 1e-12
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="x"), dict(rotary_dim=8, base=1.0),
                dict(rotary_dim=8, scaling="ramp", factor=0.5), dict(rotary_dim=8, factor=0.0)):
        with pytest.raises(ValueError):
            hb.rotary_inv_freq(**{**dict(device="cpu"), **bad})


def test_cache_oracle():
    """The oracle keeps the format's promises: no clipping, half a step at most,
    and no smaller scale would do."""
    rng = np.random.default_rng(0)
    for k in range(200):
        x = rng.standard_normal(16) * 2.0 ** rng.integers(-12, 10)
        c, n = lc.quantise_group(x)
        s = lc.scale_of(c)
        assert 7 * s >= np.abs(x).max() and np.all(np.abs(x - n * s) <= s / 2 * (1 + 1e-12))
        assert c == 0 or 7 * lc.scale_of(c - 1) < np.abs(x).max()
    assert lc.quantise_group(np.zeros(16)) == (0, pytest.approx(np.zeros(16)))
    c, n = lc.quantise_group([np.inf, -np.inf, np.nan, 1e9] + [0.0] * 12)
    assert c == 255 and n[:4].tolist() == [7, -7, 0, 7]
    # ties to even: s = 1, 2.5 -> 2, 3.5 -> 4
    c, n = lc.quantise_group([7.0, 2.5, -3.5, 0.5, 1.5] + [0.0] * 11)
    assert lc.scale_of(c) == 1.0 and n[:5].tolist() == [7, 2, -4, 0, 2]
    # the record's places, and the way back
    row = np.zeros(512)
    row[:16] = [7, -1, 2, -3, 4, -5, 6, -7, 1, 0, 0, 0, 0, 0, 0, 0]
    rec = lc.encode(row, np.arange(64))
    assert rec[:4].tolist() == [0x27, 0x64, 0xDF, 0x9B] and lc.scale_of(rec[256]) == 1.0
    back = lc.decode(rec)
    assert np.array_equal(back[:512], row)
    assert np.array_equal((back[512:].astype(np.float32).view(np.uint32) >> 16), np.arange(64))


def test_rotary_refuses_what_wants_a_gradient():
    """They compute no gradient: a tensor that wants one is refused while gradients are recorded, before all else."""
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    pos, f, w = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64), torch.ones(128)
    for call, names in ((lambda a: hb.hisa_rotary(a["x"], pos, a["f"], out=a["out"]), ("x", "f", "out")),
                        (lambda a: hb.hisa_norm_rotary(a["x"], pos, a["f"], weight=a["w"], bias=a["b"], norm="layer",
                                                       out=a["out"]), ("x", "f", "out", "w", "b"))):
        for name in names:
            a = dict(x=x, f=f, w=w, b=w, out=x.clone())
            a[name] = a[name].clone().requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call(a)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):      # the next check
                call(a)


def test_norm_rotary_refuses_a_missing_weight():
    with pytest.raises(ValueError, match="weight"):
        hb.hisa_norm_rotary(torch.zeros((4, 2, 128)), torch.zeros(4, dtype=torch.int32),
                            torch.zeros(32, dtype=torch.float64), weight=None)
