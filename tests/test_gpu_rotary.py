"""hisa_rotary and hisa_norm_rotary against the extended-precision oracle.

Tolerance, from the arithmetic.  u = 2^-24 is fp32's half step.  The angle in
half turns is rounded to fp32 (pi u at most), cut at 2^-32 turns, sincospi adds
2 ulp (4 u), the amplitude, the two products and the sum one u each: under
12 u, so 16 u on |a| + |b| (times the amplitude).  The norm sums at most 1024
squares as at most 32 + 5 terms in sequence: under 40 u on the mean square, 20 u
after the root, and 6 more roundings; the layer norm's mean likewise on
mean|x|: 64 u on (|x| + mean|x|) / rms * |weight|, 2 u on |bias|.  A bf16 result
adds half its step, 2^-8 of the value (and of the fp32 error: 1.01)."""
import numpy as np
import pytest
import torch

from oracle import rotary as orot

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _hb():
    from hierarchical_top_key_b200 import binding as hb
    return hb


def _inputs(T, H, d, dtype, seed, last=100000, gap=0, batch=None):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn((T, H * d + gap), generator=g) * 2).to(dtype).cuda()
    x = wide[:, :H * d].view(T, H, d)
    pos = torch.randint(0, last + 1, (T,), generator=g, dtype=torch.int32)
    if T > 2:
        pos[0], pos[1], pos[2] = 0, last, -7
    return x, pos.cuda()


def _pair_size(x, f, offset, inter, amp):
    """|a| + |b| of each feature's pair (times the amplitude), 0 outside the part."""
    R = 2 * len(f)
    out = np.zeros(x.shape)
    part = np.abs(x[..., offset:offset + R]).astype(np.float64)
    if inter:
        s = np.repeat(part[..., 0::2] + part[..., 1::2], 2, axis=-1)
    else:
        s = np.tile(part[..., :R // 2] + part[..., R // 2:], 2)
    out[..., offset:offset + R] = s * abs(amp)
    return out


def _compare(got, ref, err, dtype, what=""):
    got = got.double().cpu().numpy()
    ref = np.asarray(ref, np.float64)
    tol = err * 1.01 + (2.0 ** -8 * np.abs(ref) + 1e-38 if dtype == torch.bfloat16 else U * np.abs(ref))
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {np.argwhere(bad)[:3].tolist()} {got[bad][:3]} {ref[bad][:3]}"


CASES = [  # tokens, heads, dim, rot, offset
    (1, 1, 64, 64, 0), (7, 64, 128, 64, 0), (5, 3, 80, 64, 16), (33, 16, 576, 64, 512), (4, 2, 2, 2, 0),
    (3, 5, 77, 30, 13), (2, 1, 1024, 1024, 0), (130, 1, 128, 128, 0), (9, 2, 192, 64, 128), (11, 7, 96, 24, 72)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("T,H,d,rot,offset", CASES)
def test_rotary(lib, T, H, d, rot, offset, inter, dtype):
    hb = _hb()
    x, pos = _inputs(T, H, d, dtype, seed=d + rot, gap=0 if d % 3 else 24)
    f, amp = hb.rotary_inv_freq(rot, scaling="ramp", factor=8.0)
    xn, pn, fn = x.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy()
    for rev in (False, True):
        out = hb.hisa_rotary(x, pos, f, offset=offset, interleaved=inter, amplitude=amp, reverse=rev)
        ref = orot.rotate(xn, pn, fn, offset, inter, amp, rev)
        _compare(out, ref, 16 * U * _pair_size(xn, fn, offset, inter, amp), dtype, f"reverse={rev}")
        keep = np.ones(d, bool)
        keep[offset:offset + rot] = False
        assert np.array_equal(out.double().cpu().numpy()[..., keep], xn[..., keep])      # copied as they are


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("T,H,d,rot,offset", CASES)
def test_norm_rotary(lib, T, H, d, rot, offset, norm, dtype):
    hb = _hb()
    for inter, norm_dim in ((True, d), (False, 512 if d == 576 else max(1, d - 5))):
        x, pos = _inputs(T, H, d, dtype, seed=d + rot, gap=0 if d % 3 else 24)
        f, amp = hb.rotary_inv_freq(rot)
        g = torch.Generator().manual_seed(d)
        w = (1 + 0.3 * torch.randn(norm_dim, generator=g)).cuda()
        b = torch.randn(norm_dim, generator=g).cuda() if norm == "layer" and inter else None
        out = hb.hisa_norm_rotary(x, pos, f, weight=w, bias=b, norm=norm, eps=1e-5, norm_dim=norm_dim, offset=offset,
                                  interleaved=inter)
        xn, pn, fn = x.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy()
        wn, bn = w.cpu().numpy(), None if b is None else b.cpu().numpy()
        y = orot.norm(xn, norm, norm_dim, wn, bn, float(np.float32(1e-5)))
        part = xn[..., :norm_dim]
        mean = part.mean(-1, keepdims=True) if norm == "layer" else 0.0
        rms = np.sqrt(((part - mean) ** 2).mean(-1, keepdims=True) + 1e-5)
        e = np.zeros(xn.shape)
        e[..., :norm_dim] = 64 * U * (np.abs(part) + np.abs(part).mean(-1, keepdims=True)) / rms * np.abs(wn) + \
            (2 * U * np.abs(bn) if bn is not None else 0)
        ref = orot.rotate(y, pn, fn, offset, inter)
        turned = _pair_size(e, fn, offset, inter, 1.0)
        inside = np.zeros(d, bool)
        inside[offset:offset + rot] = True
        e = np.where(inside, turned, e) + 16 * U * _pair_size(np.asarray(y, np.float64), fn, offset, inter, 1.0)
        _compare(out, ref, e, dtype, f"interleaved={inter} norm_dim={norm_dim}")


def test_far_positions(lib):
    """Positions up to 2^31 - 1: the angle keeps its precision (an fp32 product would be off by whole turns)."""
    hb = _hb()
    x = torch.randn((6, 2, 64), generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 1 << 30, 999_999_937, 16_777_217, 1_048_575], dtype=torch.int32).cuda()
    f, _ = hb.rotary_inv_freq(64)
    out = hb.hisa_rotary(x, pos, f)
    ref = orot.rotate(x.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy())
    # inv_freq / 2 pi is one fp64 product: 2^-53 of a turn's part (and the rounded
    # 1 / 2 pi another) times the position
    extra = 2 * np.pi * np.abs(pos.cpu().numpy().astype(np.float64))[:, None, None] * 2.0 ** -52 * 0.16
    size = _pair_size(x.cpu().numpy(), f.cpu().numpy(), 0, False, 1.0)
    _compare(out, ref, (16 * U + extra) * size, torch.float32)


@pytest.mark.parametrize("d,rot,offset", [(576, 64, 512), (128, 64, 0), (77, 30, 13), (64, 64, 0)])
def test_in_place_and_strided(lib, d, rot, offset):
    """In place over a slice of a wider tensor: the same bits, and nothing else is touched."""
    hb = _hb()
    T, H = 37, 3
    f, _ = hb.rotary_inv_freq(rot)
    pos = torch.arange(T, dtype=torch.int32).cuda() * 1000
    wide = torch.randn((T, H + 1, d + 8), generator=torch.Generator().manual_seed(d)).to(torch.bfloat16).cuda()
    w = torch.ones(d, device="cuda")
    for run in (lambda x, o: hb.hisa_rotary(x, pos, f, offset=offset, out=o),
                lambda x, o: hb.hisa_norm_rotary(x, pos, f, weight=w, offset=offset, out=o)):
        buf = wide.clone()
        view = buf[:, 1:, :d]
        want = run(view.contiguous(), None)
        assert run(view, view) is view
        assert torch.equal(view, want)
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[:, 1:, :d] = False
        assert torch.equal(buf[rest], wide[rest])
        out = torch.full_like(wide, 7.0)                      # out with strides of its own
        run(wide[:, 1:, :d], out[:, :H, 8:] if d % 2 else out[:, :H, :d])
        assert torch.equal(out[:, :H, 8:] if d % 2 else out[:, :H, :d], want)
        assert (out[:, H] == 7.0).all()
    x4 = wide[:36, :3, :d].reshape(4, 9, 3, d)
    got = hb.hisa_rotary(x4, pos[:36].view(4, 9), f, offset=offset)
    assert torch.equal(got.view(36, 3, d), hb.hisa_rotary(x4.reshape(36, 3, d), pos[:36].contiguous(), f, offset=offset))


def test_reverse_is_the_gradient_and_the_inverse(lib):
    """<g, rotate(x)> = <reverse(g), x>, and turning back with 1 / amplitude returns x."""
    hb = _hb()
    T, H, d, rot, offset, amp = 40, 4, 96, 64, 16, 1.3
    g_ = torch.Generator().manual_seed(2)
    x, g = (torch.randn((T, H, d), generator=g_).cuda() for _ in range(2))
    f, _ = hb.rotary_inv_freq(rot)
    pos = torch.arange(T, dtype=torch.int32).cuda() * 997
    y = hb.hisa_rotary(x, pos, f, offset=offset, amplitude=amp)
    gx = hb.hisa_rotary(g, pos, f, offset=offset, amplitude=amp, reverse=True)
    a, b = (g.double() * y.double()).sum(), (gx.double() * x.double()).sum()
    # each of the two sums has T*H*d terms of size up to 2 amp |g||x| with error 16 u of it
    assert abs(a - b) <= 2 * 16 * U * 2 * amp * float((g.abs().double() * 4 * x.abs().max().double()).sum())
    # against differences: the map is linear, so a difference quotient has no error of its own
    step = torch.zeros_like(x)
    step[3, 1, offset + 5] = 1.0
    dy = hb.hisa_rotary(x + step, pos, f, offset=offset, amplitude=amp).double() - y.double()
    size = 4 * 16 * U * amp * 2 * float(x.abs().max() + 1)
    assert abs(float((g.double() * dy).sum()) - float(gx[3, 1, offset + 5])) <= size * float(g.abs().max()) * 2
    back = hb.hisa_rotary(y, pos, f, offset=offset, amplitude=1 / amp, reverse=True)
    assert (back - x).abs().max() <= 4 * 16 * U * 2 * float(x.abs().max())


def test_no_tokens_streams_and_graphs(lib):
    hb = _hb()
    f, _ = hb.rotary_inv_freq(64)
    empty = hb.hisa_rotary(torch.empty((0, 4, 128), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert empty.shape == (0, 4, 128)
    x, pos = _inputs(50, 8, 128, torch.bfloat16, 3)
    w = torch.ones(128, device="cuda")
    want = hb.hisa_norm_rotary(x, pos, f, weight=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = hb.hisa_norm_rotary(x, pos, f, weight=w)
    side.synchronize()
    assert torch.equal(got, want)
    xs, out = torch.zeros_like(x), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        hb.hisa_norm_rotary(xs, pos, f, weight=w, out=out)
    xs.copy_(x)
    g.replay()
    assert torch.equal(out, want)


def test_values_that_are_not_finite_stay_in_their_row(lib):
    hb = _hb()
    x, pos = _inputs(6, 2, 128, torch.bfloat16, 4)
    f, _ = hb.rotary_inv_freq(64)
    w = torch.ones(128, device="cuda")
    want = hb.hisa_norm_rotary(x, pos, f, weight=w)
    y = x.clone()
    y[2, 1, 5] = float("nan")
    y[4, 0, 100] = float("inf")
    got = hb.hisa_norm_rotary(y, pos, f, weight=w)
    touched = torch.zeros((6, 2), dtype=torch.bool)
    touched[2, 1] = touched[4, 0] = True
    assert torch.equal(got[~touched.cuda()], want[~touched.cuda()])
    assert got[2, 1].isnan().all()


def _check_norm_rotary(x, pos, f, norm, norm_dim, w, b, offset, inter, out, what=""):
    """out against the oracle, within the bounds at the top."""
    xn, pn, fn = x.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy()
    wn, bn = w.cpu().numpy(), None if b is None else b.cpu().numpy()
    d, rot = xn.shape[-1], 2 * len(fn)
    y = orot.norm(xn, norm, norm_dim, wn, bn, float(np.float32(1e-5)))
    part = xn[..., :norm_dim]
    mean = part.mean(-1, keepdims=True) if norm == "layer" else 0.0
    rms = np.sqrt(((part - mean) ** 2).mean(-1, keepdims=True) + 1e-5)
    e = np.zeros(xn.shape)
    e[..., :norm_dim] = 64 * U * (np.abs(part) + np.abs(part).mean(-1, keepdims=True)) / rms * np.abs(wn) + \
        (2 * U * np.abs(bn) if bn is not None else 0)
    inside = np.zeros(d, bool)
    inside[offset:offset + rot] = True
    e = np.where(inside, _pair_size(e, fn, offset, inter, 1.0), e) + \
        16 * U * _pair_size(np.asarray(y, np.float64), fn, offset, inter, 1.0)
    _compare(out, orot.rotate(y, pn, fn, offset, inter), e, x.dtype, what)


@pytest.mark.parametrize("T,H,d,rot,offset,dtype,norm,inter", [
    (20011, 1, 576, 64, 512, torch.bfloat16, "rms", True), (20011, 1, 576, 64, 512, torch.bfloat16, "rms", False),
    (40009, 1, 128, 64, 0, torch.bfloat16, "layer", True), (4099, 40, 128, 128, 0, torch.float32, "rms", False),
    (4099, 40, 128, 128, 0, torch.float32, "layer", True), (5003, 64, 128, 64, 0, torch.bfloat16, None, True),
    (5003, 64, 128, 64, 0, torch.bfloat16, None, False), (1009, 64, 576, 64, 512, torch.bfloat16, None, False),
    (3001, 40, 80, 64, 16, torch.float32, None, False)])
def test_more_rows_than_a_wave_of_blocks(lib, T, H, d, rot, offset, dtype, norm, inter):
    """Blocks that take several rows a lane group, ragged at the end: every row as in calls of few tokens, whose
    blocks take one, out of place and in place (strided); some against the oracle."""
    hb = _hb()
    x, pos = _inputs(T, H, d, dtype, seed=T + d, gap=64, last=160000)
    f, amp = hb.rotary_inv_freq(rot, scaling="ramp", factor=8.0) if norm is None else hb.rotary_inv_freq(rot)
    nd = 512 if d == 576 else d
    g = torch.Generator().manual_seed(T)
    w = (1 + 0.3 * torch.randn(nd, generator=g)).cuda()
    b = torch.randn(nd, generator=g).cuda() if norm == "layer" else None

    def run(x, pos, out=None):
        if norm is None:
            return hb.hisa_rotary(x, pos, f, offset=offset, interleaved=inter, amplitude=amp, out=out)
        return hb.hisa_norm_rotary(x, pos, f, weight=w, bias=b, norm=norm, eps=1e-5, norm_dim=nd, offset=offset,
                                   interleaved=inter, out=out)
    got = run(x, pos)
    few = max(1, 800 // H)
    for t in range(0, T, few):
        assert torch.equal(got[t:t + few], run(x[t:t + few], pos[t:t + few])), f"tokens {t} to {t + few}"
    at = torch.unique(torch.cat([torch.tensor([0, 1, T - 2, T - 1]), torch.randint(0, T, (20,), generator=g)]))
    xa, pa, ga = x[at.cuda()], pos[at.cuda()], got[at.cuda()]
    if norm is None:
        xn, fn = xa.double().cpu().numpy(), f.cpu().numpy()
        _compare(ga, orot.rotate(xn, pa.cpu().numpy(), fn, offset, inter, amp),
                 16 * U * _pair_size(xn, fn, offset, inter, amp), dtype)
    else:
        _check_norm_rotary(xa, pa, f, norm, nd, w, b, offset, inter, ga)
    assert run(x, pos, out=x) is x
    assert torch.equal(x, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("norm,biased", [("rms", False), ("layer", True), ("layer", False)])
@pytest.mark.parametrize("T,H,d,rot,offset,norm_dim", [
    (33, 4, 128, 128, 0, 128), (37, 3, 128, 64, 0, 128), (9, 2, 128, 64, 64, 128),    # half-layout partners in a lane
    (21, 5, 80, 64, 16, 80), (12, 2, 192, 64, 128, 192), (7, 1, 576, 64, 512, 576), (3, 2, 1024, 1024, 0, 1024),
    (11, 3, 96, 64, 16, 48), (14, 4, 128, 64, 0, 32)])                                # the norm ends inside the part
def test_norms_of_whole_vectors(lib, T, H, d, rot, offset, norm_dim, norm, biased, inter, dtype):
    """Rows, parts and norms of whole 16-byte vectors, both layouts, weight and bias unlike 1 and 0."""
    hb = _hb()
    x, pos = _inputs(T, H, d, dtype, seed=d + rot + norm_dim)
    f, _ = hb.rotary_inv_freq(rot)
    g = torch.Generator().manual_seed(norm_dim)
    w = (1 + 0.3 * torch.randn(norm_dim, generator=g)).cuda()
    b = torch.randn(norm_dim, generator=g).cuda() if biased else None
    out = hb.hisa_norm_rotary(x, pos, f, weight=w, bias=b, norm=norm, eps=1e-5, norm_dim=norm_dim, offset=offset,
                              interleaved=inter)
    _check_norm_rotary(x, pos, f, norm, norm_dim, w, b, offset, inter, out)
