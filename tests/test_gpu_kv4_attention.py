"""hisa_sparse_attention_kv4 against the CPU oracle on the rows its records stand for.

Tolerance, from the arithmetic.  The products of bf16 values are exact; a
logit's 576 of them are summed in fp32 in at most 36 + 8 steps, each off by at
most 2^-23 (the tensor cores truncate) of the largest partial sum: d = 44 *
2^-23 * scale * sum|q||k| on a logit, with exp and the log-sum 2^-18 more:
lse within d + 2^-18 + 2^-22 |lse|.  A weight is off by 2 d + 2^-18 (d in it
and in the normaliser) and by bf16's half step 2^-8, the output by its own 2^-8
and the fp32 sum over at most 4096 keys, 2^-11:
|o - ref| <= (2^-8 + 2^-11 + 2 d) sum p|v| + 2^-8 |ref| + 2^-126 (n max|v| + 1),
the last because fp32 has nothing between 0 and 2^-126 (subnormals aside): a
weight below that, relative to the largest, may be lost whole."""
import numpy as np
import pytest
import torch

from oracle import latent_cache as lc
from oracle import sparse_attention as sa
from hierarchical_top_key_b200 import synthetic

pytestmark = pytest.mark.gpu
SCALE = synthetic.ATTN_SCALE


def _hb():
    from hierarchical_top_key_b200 import binding as hb
    return hb


class Case:
    """A paged cache (pages in random order), written by hisa_kv4_write, and what its records stand for."""

    def __init__(self, B, L, page, seed, scale_rows=1.0):
        hb = _hb()
        g = torch.Generator().manual_seed(seed)
        self.B, self.L, self.page = B, L, page
        per = -(-L // page)
        rows = (torch.randn((B * L, 576), generator=g) * scale_rows).to(torch.bfloat16)
        self.table = torch.randperm(B * per + 3, generator=g)[:B * per].to(torch.int32).view(B, per)
        self.cache = torch.zeros((B * per + 3, page, 416), dtype=torch.uint8, device="cuda")
        s = torch.arange(L)
        self.slots = torch.stack([self.table[b, s // page] * page + s % page for b in range(B)]).to(torch.int32)
        hb.hisa_kv4_write(rows.cuda(), self.slots.view(-1).cuda(), self.cache)
        back = hb.hisa_kv4_read(self.cache, self.slots.view(-1).cuda())
        self.kv = back.float().cpu().numpy().reshape(B, L, 576)

    def rewrite(self, b, s, row):
        hb = _hb()
        t = torch.from_numpy(np.asarray(row, np.float32)).to(torch.bfloat16).view(1, 576).cuda()
        slot = self.slots[b, s].view(1).cuda()
        hb.hisa_kv4_write(t, slot, self.cache)
        self.kv[b, s] = hb.hisa_kv4_read(self.cache, slot).float().cpu().numpy()[0]

    def run(self, q, idx, scale=SCALE):
        hb = _hb()
        o, lse = hb.hisa_sparse_attention_kv4(q.cuda(), self.cache, self.table.cuda(), torch.from_numpy(idx).cuda(),
                                              scale=scale, num_keys=self.L)
        hb.get_status()
        return o, lse

    def check(self, q, idx, o, lse, what="", rows=None):
        q, o, lse = q.float().numpy(), o.float().cpu().numpy(), lse.cpu().numpy()
        for b, t in rows if rows is not None else np.ndindex(q.shape[:2]):
            sel = sa.selected_positions(idx[b, t], self.L)
            name = f"{what} sequence {b} query {t}"
            if sel.size == 0:
                assert np.all(o[b, t] == 0) and np.all(np.isneginf(lse[b, t])), f"{name}: empty set"
                continue
            kv = self.kv[b].astype(np.float64)
            ro, rl = sa.sparse_attention_query(q[b, t], kv, kv[:, :512], idx[b, t], SCALE)
            qd = q[b, t].astype(np.float64)
            d = 44 * 2.0 ** -23 * SCALE * (np.abs(qd) @ np.abs(kv[sel]).T).max(1)
            p = np.exp(SCALE * (qd @ kv[sel].T) - rl[:, None])
            pv = p @ np.abs(kv[sel, :512])
            tol = (2.0 ** -8 + 2.0 ** -11 + 2 * d[:, None]) * pv + 2.0 ** -8 * np.abs(ro) + \
                2.0 ** -126 * (sel.size * np.abs(kv[sel, :512]).max() + 1)
            bad = ~(np.abs(o[b, t] - ro) <= tol)
            assert not bad.any(), f"{name}: o off at {np.argwhere(bad)[:4].tolist()} of {bad.sum()}"
            bad = ~(np.abs(lse[b, t] - rl) <= d + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl))
            assert not bad.any(), f"{name}: lse {lse[b, t][bad][:3]} {rl[bad][:3]}"


def _q(B, Q, H, seed):
    return torch.randn((B, Q, H, 576), generator=torch.Generator().manual_seed(seed + 1000)).to(torch.bfloat16)


@pytest.mark.parametrize("H", [1, 5, 16, 64, 127, 128, 129, 256])
def test_heads(lib, H):
    c = Case(1, 700, 64, H)
    q = _q(1, 3, H, H)
    idx = synthetic.random_index_rows(1, 3, 700, 200, np.full((1, 3), 700), seed=H)
    c.check(q, idx, *c.run(q, idx), f"H={H}")


@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 127, 128, 129, 2048, 4096])
@pytest.mark.parametrize("Q", [1, 80])
def test_lengths(lib, k, Q):
    """Index rows around the tile's length, one query (split over keys) and many (whole)."""
    c = Case(1, 5000, 64, k)
    q = _q(1, Q, 128, k)
    idx = synthetic.random_index_rows(1, Q, 5000, k, np.full((1, Q), 5000), seed=k)
    o, lse = c.run(q, idx)
    c.check(q, idx, o, lse, f"k={k}", rows=[(0, t) for t in sorted({0, Q // 2, Q - 1})])


@pytest.mark.parametrize("page,L", [(1, 100), (7, 100), (64, 1), (128, 1000), (1000, 999)])
def test_pages(lib, page, L):
    c = Case(3, L, page, page)
    q = _q(3, 2, 128, page)
    nv = np.full((3, 2), L)
    nv[1] = max(1, L // 3)
    idx = synthetic.random_index_rows(3, 2, L, 96, nv, seed=page)
    c.check(q, idx, *c.run(q, idx), f"page={page}")


def test_padding_repeats_and_empty_rows(lib):
    B, Q, L, K = 2, 9, 3000, 300
    c = Case(B, L, 64, 5)
    q = _q(B, Q, 128, 5)
    nv = np.full((B, Q), L)
    nv[0, 3] = 40                                   # fewer positions than k: -1 padding
    idx = synthetic.random_index_rows(B, Q, L, K, nv, seed=5)
    idx[0, 5] = -1                                  # empty set
    idx[0, 6, ::2] = -1                             # holes
    idx[0, 7, :-1] = -1                             # one key, in the last place
    idx[1, 2, 100:200] = idx[1, 2, :100]            # repeats count once
    idx[1, 4, ::3] = L + 7                          # out-of-range entries are dropped
    idx[1, 5, ::3] = -2 ** 31
    idx[1, 5, 1::3] = 2 ** 31 - 1
    idx[1, 6, :] = 17                               # one key repeated: a single position
    idx[1, 7, :] = L
    o, lse = c.run(q, idx)
    c.check(q, idx, o, lse)
    for H in (16, 200):                             # few heads, a part of a second slice
        q = _q(B, Q, H, 6)
        c.check(q, idx, *c.run(q, idx), f"H={H}")


@pytest.mark.parametrize("L", [14848, 14849])
def test_repeats_are_found_by_bits_and_by_the_table(lib, L):
    """100 places have a table of 464 words = 14848 bits: one key more and the keys' bits no longer fit.  Rows
    without a repeat, with one (the last key, in the row's first and last place), and with nothing else."""
    K = 100
    c = Case(1, L, 64, 11)
    q = _q(1, 4, 16, 11)
    idx = synthetic.random_index_rows(1, 4, L, K, np.full((1, 4), L), seed=11)
    idx[0, 1, 0] = idx[0, 1, K - 1] = L - 1
    idx[0, 2, :] = L - 1
    idx[0, 3, ::2] = 0
    c.check(q, idx, *c.run(q, idx), f"L={L}")


@pytest.mark.parametrize("H", [16, 200])
def test_many_queries_of_unlike_lengths(lib, H):
    """More queries than pairs of SMs, so every pair takes several: the first of them empty, of one tile (none for
    the pair's second CTA) or of one key, the later ones long, and the other way round at the end."""
    Q, L, K = 400, 2000, 300
    c = Case(1, L, 64, H + 3)
    q = _q(1, Q, H, H + 3)
    length = np.array([0, 1, 64, 65, 128, 129, 300, 40])
    n = np.where(np.arange(Q) < 160, length[np.arange(Q) % 4], length[(np.arange(Q) * 5 // 3) % 8])
    idx = synthetic.random_index_rows(1, Q, L, K, np.full((1, Q), L), seed=H)
    idx[0, np.arange(K)[None, :] >= n[:, None]] = -1
    o, lse = c.run(q, idx)
    c.check(q, idx, o, lse, f"H={H}", rows=[(0, t) for t in range(0, Q, 7)])
    assert np.array_equal(np.isneginf(lse.cpu().numpy()[0, :, 0]), n == 0)


def test_a_query_does_not_see_its_neighbours(lib):
    """Few heads: what stands behind a query's rows is the next query's, infinities and NaN among them."""
    c = Case(1, 500, 64, 9)
    q = _q(1, 3, 5, 9)
    idx = synthetic.random_index_rows(1, 3, 500, 130, np.full((1, 3), 500), seed=9)
    want, want_lse = c.run(q, idx)
    c.check(q, idx, want, want_lse)
    q[0, 1] = float("nan")
    q[0, 1, 2] = float("inf")
    q[0, 1, 4] = 1e30
    o, lse = c.run(q, idx)
    for t in (0, 2):
        assert torch.equal(o[0, t], want[0, t]) and torch.equal(lse[0, t], want_lse[0, t])


def test_split_and_whole_agree(lib):
    """The same rows alone (split over the keys) and within a batch that is not split."""
    L, K = 4000, 2048
    c = Case(1, L, 64, 9)
    q = _q(1, 200, 128, 9)
    idx = synthetic.random_index_rows(1, 200, L, K, np.full((1, 200), L), seed=9)
    idx[0, 1, 70:] = -1                             # parts of a split row with no key at all
    idx[0, 2] = -1
    o, lse = c.run(q, idx)
    for t in (0, 1, 2, 199):
        o1, l1 = c.run(q[:, t:t + 1], idx[:, t:t + 1].copy())
        c.check(q[:, t:t + 1], idx[:, t:t + 1], o1, l1, "alone")
        d = (o1[0, 0].float() - o[0, t].float()).abs()
        assert (d <= 2.0 ** -7 * o[0, t].float().abs() + 2.0 ** -6).all()


@pytest.mark.parametrize("Q", [1, 7])
def test_small_workspace(lib, Q):
    """Queries in chunks of what the workspace holds: the same bits; nothing past it is touched."""
    hb = _hb()
    c = Case(2, 900, 64, 3)
    q = _q(2, Q, 128, 3)
    idx = synthetic.random_index_rows(2, Q, 900, 500, np.full((2, Q), 900), seed=3)
    o, lse = c.run(q, idx)
    c.check(q, idx, o, lse, "whole")
    full = hb.workspace_size(hb.OP_ATTENTION_KV4, hb.Shape(2, 900, Q, 128, 0, 0, 0, 500, hb.HISA_BF16))
    assert full % (2 * Q) == 0
    for rows in (1, 2 * Q - 1):
        n = full // (2 * Q) * rows
        ws = torch.full((n + 64,), 0xC3, dtype=torch.uint8, device="cuda")
        o2, l2 = hb.hisa_sparse_attention_kv4(q.cuda(), c.cache, c.table.cuda(), torch.from_numpy(idx).cuda(),
                                              scale=SCALE, num_keys=900, workspace=ws[:n])
        hb.get_status()
        assert torch.equal(o, o2) and torch.equal(lse, l2) and (ws[n:] == 0xC3).all()
    with pytest.raises(hb.HisaError) as e:
        hb.hisa_sparse_attention_kv4(q.cuda(), c.cache, c.table.cuda(), torch.from_numpy(idx).cuda(), scale=SCALE,
                                     num_keys=900, workspace=ws[:64])
    assert e.value.status == 3


@pytest.mark.parametrize("Q", [2, 90])
def test_large_logits_and_jumps_of_the_maximum(lib, Q):
    """Keys aligned with the mean head direction at chosen places, each raising
    the maximum by some tens; heads the other way keep theirs.  Then a tile
    whose logits are hundreds below the others.  Two queries are split over the
    keys, 90 are not."""
    L, K = 3000, 1500
    c = Case(1, L, 64, 21)
    q = _q(1, 2, 128, 21)
    q[0, :, 64:] = -q[0, :, :64]
    idx = synthetic.random_index_rows(1, 2, L, K, np.full((1, 2), L), seed=21)
    u = q[0, 0, :64].double().sum(0).numpy()
    u /= np.linalg.norm(u)
    for place, size in ((2 * 64 + 7, 120.0), (9 * 64 + 33, 240.0), (20 * 64 + 30, 360.0)):
        c.rewrite(0, int(idx[0, 0, place]), size * u)
    for place in range(12 * 64, 13 * 64):
        c.rewrite(0, int(idx[0, 0, place]), -300.0 * u)
    q, idx = q.repeat(1, Q // 2, 1, 1), np.tile(idx, (1, Q // 2, 1))
    o, lse = c.run(q, idx)
    c.check(q, idx, o, lse, "planted maxima", rows=[(0, t) for t in (0, 1, Q - 2, Q - 1)])
    assert all(torch.equal(o[0, t], o[0, t % 2]) for t in range(Q))
    assert np.median(lse.cpu().numpy()[0, 0]) > 20.0


@pytest.mark.parametrize("factor", [0.0, -1.0, 2.0 ** -120])
def test_scales(lib, factor):
    """A scale of 0 (every key alike), a negative and a tiny one: as the query times the factor."""
    c = Case(1, 300, 64, 13)
    q = _q(1, 2, 128, 13)
    idx = synthetic.random_index_rows(1, 2, 300, 100, np.full((1, 2), 300), seed=13)
    o, lse = c.run(q, idx, scale=SCALE * factor)
    c.check((q.float() * factor).to(torch.bfloat16), idx, o, lse, f"factor={factor}")


def test_pages_outside_the_cache_are_reported(lib):
    hb = _hb()
    c = Case(1, 640, 64, 2)
    q = _q(1, 2, 128, 2)
    idx = synthetic.random_index_rows(1, 2, 640, 300, np.full((1, 2), 640), seed=2)
    idx[0, 1] = -1
    idx[0, 1, :64] = np.arange(64)                  # needs page 0 alone
    bad = c.table.clone()
    bad[0, 3], bad[0, 5] = -1, c.cache.shape[0]
    hb.get_status()
    o, lse = hb.hisa_sparse_attention_kv4(q.cuda(), c.cache, bad.cuda(), torch.from_numpy(idx).cuda(), scale=SCALE,
                                          num_keys=640)
    with pytest.raises(hb.HisaError) as e:
        hb.get_status()
    assert e.value.status == 1
    for p in (3, 5):                                # the rest is attended as if those positions were not selected
        idx[(idx >= 64 * p) & (idx < 64 * p + 64)] = -1
    c.check(q, idx, o, lse, "bad pages")


def test_masked_places_may_hold_anything(lib):
    """Records that no index names (NaN positional features, all code bytes) change nothing."""
    c = Case(1, 500, 64, 4)
    q = _q(1, 2, 128, 4)
    idx = synthetic.random_index_rows(1, 2, 500, 100, np.full((1, 2), 500), seed=4)
    want = c.run(q, idx)
    used = np.unique(idx[idx >= 0])
    slots = torch.ones(c.cache.shape[0] * 64, dtype=torch.bool)
    slots[c.slots[0, torch.from_numpy(used).long()].long()] = False
    c.cache.view(-1, 416)[slots.cuda()] = 255
    got = c.run(q, idx)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_logits_that_are_not_finite(lib):
    """A positional feature of -inf (in the query's sign, so a logit of -inf) takes
    its key's weight away, be it a whole tile's, the first 32 keys' or all keys';
    NaN and +inf make their query NaN and no other."""
    L = 400
    c = Case(1, L, 64, 17)
    q = _q(1, 4, 128, 17)
    q[..., 512] = q[..., 512].abs() + 0.5
    idx = np.tile(np.arange(200, dtype=np.int32), (1, 4, 1))
    idx[0, 1] += 100
    idx[0, 3] += 200
    want = idx.copy()
    gone = list(range(0, 40)) + list(range(128, 192)) + list(range(200, 400))
    for s in gone:
        row = c.kv[0, s].copy()
        row[512] = -np.inf
        t = torch.from_numpy(row).to(torch.bfloat16).view(1, 576).cuda()
        _hb().hisa_kv4_write(t, c.slots[0, s].view(1).cuda(), c.cache)
    want[np.isin(want, gone)] = -1
    o, lse = c.run(q, idx)
    c.check(q, want, o, lse, "-inf")                       # query 3: an empty set
    bad = torch.from_numpy(c.kv[0, 60:61]).to(torch.bfloat16).cuda()
    bad[0, 520] = float("nan")
    _hb().hisa_kv4_write(bad, c.slots[0, 60].view(1).cuda(), c.cache)
    o2, lse2 = c.run(q, idx)
    assert o2[0, [0, 2]].isnan().all() and lse2[0, [0, 2]].isnan().all()
    assert torch.equal(o2[0, [1, 3]], o[0, [1, 3]]) and torch.equal(lse2[0, [1, 3]], lse[0, [1, 3]])


def test_streams_and_graphs(lib):
    """Two captured calls of different sizes, replayed in either order, and a call on another stream."""
    hb = _hb()
    c = Case(2, 2000, 64, 8)
    table = c.table.cuda()
    calls = []
    for Q, K in ((1, 1024), (3, 700)):
        q = _q(2, Q, 128, Q)
        idx = synthetic.random_index_rows(2, Q, 2000, K, np.full((2, Q), 2000), seed=Q)
        calls.append((q, idx, q.cuda(), torch.from_numpy(idx).cuda()))
    graphs, outs = [], []
    torch.cuda.synchronize()
    for q, idx, dq, di in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(hb.hisa_sparse_attention_kv4(dq, c.cache, table, di, scale=SCALE, num_keys=2000))
        graphs.append(g)
    for order in ((0, 1), (1, 0)):
        for x in outs:
            x[0].fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        for i in (0, 1):
            c.check(calls[i][0], calls[i][1], *outs[i], f"graph {i}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = hb.hisa_sparse_attention_kv4(calls[0][2], c.cache, table, calls[0][3], scale=SCALE, num_keys=2000)
    side.synchronize()
    assert torch.equal(got[0], outs[0][0]) and torch.equal(got[1], outs[0][1])


def test_same_result_every_time(lib):
    c = Case(2, 3000, 64, 12)
    for Q in (1, 90):
        q = _q(2, Q, 128, 12)
        idx = synthetic.random_index_rows(2, Q, 3000, 2048, np.full((2, Q), 3000), seed=12)
        idx[:, :, 5] = idx[:, :, 900]               # a repeat in every row
        a = c.run(q, idx)
        for _ in range(3):
            b = c.run(q, idx)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_decode_step_of_all_of_them(lib):
    """As a serving step uses them: the new token's latent row normed, turned and
    written to the 4-bit cache, the indexer's query turned and its key normed and
    turned, the selection over all keys, the attention query's positional part
    turned in place, attention over the selected records."""
    hb = _hb()
    B, L, page, H, d = 2, 1500, 64, 64, 128
    g = torch.Generator().manual_seed(31)

    def rnd(*s):
        return torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    f, amp = hb.rotary_inv_freq(64, scaling="ramp", factor=8.0)
    ones512, ones128 = torch.ones(512, device="cuda"), torch.ones(128, device="cuda")
    per = -(-L // page)
    table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per).cuda()
    cache = torch.zeros((B * per, page, 416), dtype=torch.uint8, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
    # the prefix and the step's token alike: latent rows and indexer keys of every position
    latent = hb.hisa_norm_rotary(rnd(B, L, 1, 576), pos, f, weight=ones512, norm_dim=512, offset=512, interleaved=True,
                                 amplitude=amp)
    slots = torch.gather(table.long(), 1, (pos // page).long()) * page + pos % page
    hb.hisa_kv4_write(latent.view(-1, 576), slots.to(torch.int32).view(-1), cache)
    keys = hb.hisa_norm_rotary(rnd(B, L, 1, d), pos, f, weight=ones128, bias=torch.zeros(128, device="cuda"),
                               norm="layer", interleaved=True, amplitude=amp).view(B, L, d)
    last = pos[:, -1:].contiguous()
    qi = hb.hisa_rotary(rnd(B, 1, H, d), last, f, interleaved=True, amplitude=amp)
    w = torch.rand((B, 1, H), generator=g).cuda()
    idx, _ = hb.HisaIndexer(64, 8, 256)(qi, w, keys, torch.full((B, 1), L, dtype=torch.int32, device="cuda"))
    qa = rnd(B, 1, 128, 576)
    before = qa.clone()
    hb.hisa_rotary(qa, last, f, offset=512, interleaved=True, amplitude=amp, out=qa)
    assert torch.equal(qa[..., :512], before[..., :512]) and not torch.equal(qa[..., 512:], before[..., 512:])
    o, lse = hb.hisa_sparse_attention_kv4(qa, cache, table, idx, scale=SCALE, num_keys=L)
    hb.get_status()
    c = Case.__new__(Case)
    c.L = L
    c.kv = lc.decode_many(cache.view(-1, 416)[slots.view(-1)].cpu().numpy()).reshape(B, L, 576)
    hidx = idx.cpu().numpy()
    assert all(len(set(hidx[b, 0].tolist())) == 256 for b in range(B))
    c.check(qa.cpu(), hidx, o, lse, "decode step")
    # and the 4-bit rows are the bf16 rows to half a step
    o16, _ = hb.hisa_sparse_attention(qa, latent.view(B, L, 576), idx, scale=SCALE)
    rel = (o16.float() - o.float()).norm() / o16.float().norm()
    assert rel < 0.15


def _not_finite(value, what):
    assert value.isnan().all(), f"{what}: {value.flatten()[:4].tolist()}"


@pytest.mark.parametrize("Q", [1, 90])
@pytest.mark.parametrize("H", [16, 128])
def test_a_query_head_that_is_not_finite(lib, H, Q):
    """NaN, infinities and an overflow in chosen heads of a query make just those heads NaN, whether the query is
    alone (split over its keys) or one of 90 (whole); the other heads keep their bits."""
    L, K = 3000, 2048
    c = Case(1, L, 64, H + 41)
    q = _q(1, Q, H, H + 41)
    idx = synthetic.random_index_rows(1, Q, L, K, np.full((1, Q), L), seed=H + 41)
    want, want_lse = c.run(q, idx)
    q[0, 0, 1, 7] = float("nan")
    q[0, 0, 4, 560] = float("inf")                  # a positional feature: no key's is 0, about half are negative
    q[0, 0, 9, 560] = float("-inf")
    q[0, 0, 11] = 3e38                              # fp32 dot products of both infinities
    o, lse = c.run(q, idx)
    bad = [1, 4, 9, 11]
    rest = [h for h in range(H) if h not in bad]
    _not_finite(o[0, 0, bad], "o")
    _not_finite(lse[0, 0, bad], "lse")
    assert torch.equal(o[0, 0, rest], want[0, 0, rest]) and torch.equal(lse[0, 0, rest], want_lse[0, 0, rest])
    assert torch.equal(o[0, 1:], want[0, 1:]) and torch.equal(lse[0, 1:], want_lse[0, 1:])


@pytest.mark.parametrize("feature", [float("nan"), float("inf")])
def test_keys_that_are_not_finite_in_every_part_with_keys(lib, feature):
    """A split row all of whose parts with keys hold a key with a logit of NaN or +inf: one part of one tile, one key
    alone, and every part.  NaN, as within a batch that is not split."""
    L, K = 3000, 2048
    c = Case(1, L, 64, 43)
    q = _q(1, 90, 128, 43)
    q[..., 512] = q[..., 512].abs() + 0.5
    idx = synthetic.random_index_rows(1, 90, L, K, np.full((1, 90), L), seed=43)
    idx[0, 0, 40:] = -1                             # one tile: only the first part has keys
    idx[0, 1, 1:] = -1
    for s in {int(idx[0, 0, 39]), int(idx[0, 1, 0])} | set(idx[0, 2, ::32].tolist()):
        row = torch.from_numpy(c.kv[0, s:s + 1]).to(torch.bfloat16).cuda()
        row[0, 512] = feature
        _hb().hisa_kv4_write(row, c.slots[0, s].view(1).cuda(), c.cache)
    o, lse = c.run(q, idx)
    for t in range(3):
        _not_finite(o[0, t], f"whole o, query {t}")
        _not_finite(lse[0, t], f"whole lse, query {t}")
        o1, l1 = c.run(q[:, t:t + 1], idx[:, t:t + 1].copy())
        _not_finite(o1, f"split o, query {t}")
        _not_finite(l1, f"split lse, query {t}")


@pytest.mark.parametrize("Q", [1, 90])
def test_a_scale_of_zero_keeps_what_is_not_finite(lib, Q):
    """0 times a dot product that is NaN or infinite is NaN; every other head weighs all keys alike."""
    c = Case(1, 600, 64, 47)
    q = _q(1, Q, 128, 47)
    idx = synthetic.random_index_rows(1, Q, 600, 300, np.full((1, Q), 600), seed=47)
    want, want_lse = c.run(q, idx, scale=0.0)
    c.check(q * 0, idx, want, want_lse, "scale 0", rows=[(0, 0)])
    q[0, 0, 2, 100] = float("nan")
    q[0, 0, 5, 570] = float("inf")
    o, lse = c.run(q, idx, scale=0.0)
    rest = [h for h in range(128) if h not in (2, 5)]
    _not_finite(o[0, 0, [2, 5]], "o")
    _not_finite(lse[0, 0, [2, 5]], "lse")
    assert torch.equal(o[0, 0, rest], want[0, 0, rest]) and torch.equal(lse[0, 0, rest], want_lse[0, 0, rest])


def test_two_threads_with_index_rows_of_unlike_lengths(lib):
    """Each thread on its stream, one with the longest index rows, one with short ones: every call is accepted."""
    import threading
    hb = _hb()
    L, calls = 5000, 3000
    c = Case(1, L, 64, 53)
    table = c.table.cuda()
    jobs = []
    for K in (4096, 64):
        q = _q(1, 1, 128, K)
        idx = synthetic.random_index_rows(1, 1, L, K, np.full((1, 1), L), seed=K)
        jobs.append(dict(K=K, q=q, idx=idx, dq=q.cuda(), di=torch.from_numpy(idx).cuda(), stream=torch.cuda.Stream(),
                         o=torch.empty((1, 1, 128, 512), dtype=torch.bfloat16, device="cuda"),
                         lse=torch.empty((1, 1, 128), device="cuda"), bad=[],
                         ws=torch.empty(hb.workspace_size(hb.OP_ATTENTION_KV4,
                                                          hb.Shape(1, L, 1, 128, 0, 0, 0, K, hb.HISA_BF16)),
                                        dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(j):
        start.wait()
        for _ in range(calls):
            status = lib.hisa_sparse_attention_kv4(
                j["dq"].data_ptr(), c.cache.data_ptr(), c.cache.shape[0], c.page, table.data_ptr(), j["di"].data_ptr(),
                1, 1, L, 128, j["K"], SCALE, j["o"].data_ptr(), j["lse"].data_ptr(), j["ws"].data_ptr(),
                j["ws"].numel(), j["stream"].cuda_stream)
            if status:
                j["bad"].append(status)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    hb.get_status()
    for j in jobs:
        assert not j["bad"], f"top_k={j['K']}: {len(j['bad'])} of {calls} calls refused, status {j['bad'][0]}"
        c.check(j["q"], j["idx"], j["o"], j["lse"], f"K={j['K']}")
