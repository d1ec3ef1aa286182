"""The 4-bit latent cache: records bit for bit as the oracle's, and back."""
import numpy as np
import pytest
import torch

from oracle import latent_cache as lc

pytestmark = pytest.mark.gpu


def _hb():
    from hierarchical_top_key_b200 import binding as hb
    return hb


def _rows(n, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, 576), generator=g) * torch.exp(torch.randn((n, 1), generator=g))).to(torch.bfloat16)


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _records(rows):
    return np.stack([lc.encode(r[:512].double().numpy(), _bits(r[512:])) for r in rows])


def test_records_are_the_oracles(lib):
    """Random rows, and every group that is hard: ties, scales that just fit, zeros,
    the largest and smallest values, infinities and NaN."""
    hb = _hb()
    rows = _rows(24, 0)
    rows[0] = 0
    s = torch.tensor(lc.SCALES[100:228:4], dtype=torch.float32)
    # amax exactly 7 s (fits), then half steps of it: all ties
    tie = (s[:, None] * torch.tensor([7, .5, 1.5, 2.5, 3.5, 4.5, 5.5, 6.5, -.5, -1.5, -2.5, -3.5, -4.5, -5.5, -6.5, 1.]))
    rows[1, :512] = tie.reshape(-1).to(torch.bfloat16)
    up = (7 * s).to(torch.bfloat16).view(torch.int16)
    rows[2, :512] = 0.1
    rows[2, 0:512:16] = (up + 1).view(torch.bfloat16)                 # one step past 7 s: the next scale
    rows[3, 0:512:16] = (up - 1).view(torch.bfloat16) * 0.5
    rows[4] = 3e38
    rows[5, :512] = 1e-7
    rows[6, ::7] = float("inf")
    rows[6, 3::11] = float("-inf")
    rows[7, ::5] = float("nan")
    rows[8, :512] = float("nan")
    rows[9, :512] = 1e-40                                             # bf16 subnormals
    rows[10, :16] = 26880.0
    rows[11, :512] = -0.0
    cache = torch.full((4, 8, 416), 0xA5, dtype=torch.uint8, device="cuda")
    slots = torch.randperm(32, generator=torch.Generator().manual_seed(1))[:24].to(torch.int32)
    hb.hisa_kv4_write(rows.cuda(), slots.cuda(), cache)
    want = np.full((32, 416), 0xA5, np.uint8)
    want[slots.numpy()] = _records(rows)
    np.testing.assert_array_equal(cache.view(32, 416).cpu().numpy(), want)
    back = hb.hisa_kv4_read(cache, slots.cuda())
    np.testing.assert_array_equal(_bits(back[:, 512:]), _bits(rows[:, 512:]))
    np.testing.assert_array_equal(back[:, :512].double().cpu().numpy(), lc.decode_many(want[slots.numpy()])[:, :512])
    hb.get_status()


def test_every_code_and_scale_reads_back(lib):
    """All 256 scales with all 16 nibbles (-8 too, which no write makes)."""
    hb = _hb()
    rng = np.random.default_rng(3)
    recs = rng.integers(0, 256, (64, 416), dtype=np.uint8)
    recs[:, 256:288] = (np.arange(64 * 32) % 256).reshape(64, 32)
    recs[:, 288:] = np.arange(64 * 64, dtype=np.uint16).reshape(64, 64).view(np.uint8)
    cache = torch.from_numpy(recs).cuda().view(8, 8, 416)
    back = hb.hisa_kv4_read(cache, torch.arange(64, dtype=torch.int32, device="cuda"))
    want = lc.decode_many(recs)
    np.testing.assert_array_equal(back.double().cpu().numpy(), want)


@pytest.mark.parametrize("n", [1, 2, 31, 64, 1000])
def test_sizes_strides_and_padding(lib, n):
    hb = _hb()
    page = 16
    pages = -(-n // page) + 3
    wide = _rows(n, n).cuda()
    wide = torch.cat([torch.zeros((n, 8), dtype=torch.bfloat16, device="cuda"), wide,
                      torch.ones((n, 24), dtype=torch.bfloat16, device="cuda")], 1)
    rows = wide[:, 8:584]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    slots[n // 2] = -1 if n > 1 else slots[0]
    cache = torch.full((pages, page, 416), 0x5A, dtype=torch.uint8, device="cuda")
    hb.hisa_kv4_write(rows, slots.cuda(), cache)
    live = (slots >= 0).numpy()
    want = np.full((pages * page, 416), 0x5A, np.uint8)
    want[slots.numpy()[live]] = _records(rows.cpu())[live]
    np.testing.assert_array_equal(cache.view(-1, 416).cpu().numpy(), want)
    out = torch.full_like(wide, 9.0)
    assert hb.hisa_kv4_read(cache, slots.cuda(), out=out[:, 8:584]).data_ptr() == out[:, 8:584].data_ptr()
    got = out.cpu()
    assert (got[:, :8] == 9.0).all() and (got[:, 584:] == 9.0).all()
    ref = lc.decode_many(want[np.maximum(slots.numpy(), 0)]) * live[:, None]
    np.testing.assert_array_equal(got[:, 8:584].double().numpy(), ref)
    hb.get_status()


def test_nothing_to_write(lib):
    hb = _hb()
    cache = torch.zeros((1, 1, 416), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    hb.hisa_kv4_write(torch.empty((0, 576), dtype=torch.bfloat16, device="cuda"), none, cache)
    assert hb.hisa_kv4_read(cache, none).shape == (0, 576)


def test_slots_past_the_cache_are_reported(lib):
    hb = _hb()
    rows = _rows(3, 5).cuda()
    cache = torch.zeros((2, 4, 416), dtype=torch.uint8, device="cuda")
    hb.get_status()
    hb.hisa_kv4_write(rows, torch.tensor([1, 8, 2], dtype=torch.int32, device="cuda"), cache)
    with pytest.raises(hb.HisaError) as e:
        hb.get_status()
    assert e.value.status == 1
    back = hb.hisa_kv4_read(cache, torch.tensor([1, 2 ** 31 - 1, 2], dtype=torch.int32, device="cuda"))
    with pytest.raises(hb.HisaError):
        hb.get_status()
    hb.get_status()                                            # cleared
    assert (back[1] == 0).all() and (back[0] != 0).any() and (back[2] != 0).any()


def test_records_past_four_gigabytes(lib):
    hb = _hb()
    pages, page = 84000, 128                                   # 4.47 GB
    cache = torch.empty((pages, page, 416), dtype=torch.uint8, device="cuda")
    rows = _rows(4, 6)
    slots = torch.tensor([pages * page - 1, 0, 10_400_000, 10_324_441], dtype=torch.int32)
    hb.hisa_kv4_write(rows.cuda(), slots.cuda(), cache)
    got = cache.view(-1, 416)[slots.long().cuda()].cpu().numpy()
    np.testing.assert_array_equal(got, _records(rows))
    np.testing.assert_array_equal(hb.hisa_kv4_read(cache, slots.cuda()).double().cpu().numpy(), lc.decode_many(got))


def test_streams_and_graphs(lib):
    hb = _hb()
    rows, cache = _rows(40, 7).cuda(), torch.zeros((8, 8, 416), dtype=torch.uint8, device="cuda")
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    src, dst = torch.zeros_like(rows), torch.empty_like(rows)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hb.hisa_kv4_write(src, slots, cache)
        hb.hisa_kv4_read(cache, slots, out=dst)
    src.copy_(rows)
    g.replay()
    other = torch.zeros_like(cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hb.hisa_kv4_write(rows, slots, other)
        back = hb.hisa_kv4_read(other, slots)
    side.synchronize()
    assert torch.equal(other, cache) and torch.equal(back, dst)
