"""The library called from several host threads."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _in_a_new_thread(call):
    got = []
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    assert got, "the thread's call raised"
    return got[0]


def test_a_threads_first_call(lib):
    """A thread that has made no CUDA call yet, of its own or through torch, has no context bound to it."""
    from hierarchical_top_key_b200 import binding as hb
    L, K = 640, 128
    g = torch.Generator().manual_seed(0)
    q = torch.randn((1, 2, 128, 576), generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn((1, L, 576), generator=g).to(torch.bfloat16).cuda()
    idx = torch.stack([torch.randperm(L, generator=g)[:K] for _ in range(2)]).to(torch.int32).view(1, 2, K).cuda()
    cache = torch.zeros((10, 64, hb.KV4_RECORD), dtype=torch.uint8, device="cuda")
    table = torch.arange(10, dtype=torch.int32, device="cuda").view(1, 10)
    hb.hisa_kv4_write(kv[0], torch.arange(L, dtype=torch.int32, device="cuda"), cache)
    want = hb.hisa_sparse_attention(q, kv, idx, scale=0.07)
    want4 = hb.hisa_sparse_attention_kv4(q, cache, table, idx, scale=0.07, num_keys=L)
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(hb.workspace_size(hb.OP_ATTENTION_KV4, hb.Shape(1, L, 2, 128, 0, 0, 0, K, hb.HISA_BF16)),
                     dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    status = _in_a_new_thread(lambda: (lib.hisa_sparse_attention(
        q.data_ptr(), kv.data_ptr(), idx.data_ptr(), 1, 2, L, 128, 576, 512, K, 0.07, o.data_ptr(), lse.data_ptr(),
        side.cuda_stream), lib.hisa_last_error()))
    torch.cuda.synchronize()
    assert status[0] == 0, status
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    status = _in_a_new_thread(lambda: (lib.hisa_sparse_attention_kv4(
        q.data_ptr(), cache.data_ptr(), 10, 64, table.data_ptr(), idx.data_ptr(), 1, 2, L, 128, K, 0.07, o.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.numel(), side.cuda_stream), lib.hisa_last_error()))
    torch.cuda.synchronize()
    assert status[0] == 0, status
    assert torch.equal(o, want4[0]) and torch.equal(lse, want4[1])
    # through the binding: its buffers come from memory that torch has already
    got = _in_a_new_thread(lambda: hb.hisa_sparse_attention_kv4(q, cache, table, idx, scale=0.07, num_keys=L))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want4[0]) and torch.equal(got[1], want4[1])


def test_scored_rows_of_unlike_lengths(lib):
    """Two threads at once, each on its stream: the flat indexer with scores, rows of 16384 sorted in 128 KB of shared
    memory, rows of 16 in 128 bytes.  The limit is the kernel's, one for all threads."""
    from hierarchical_top_key_b200 import binding as hb
    L, calls = 20000, 1500
    g = torch.Generator().manual_seed(0)
    q = torch.randn((1, 1, 16, 64), generator=g).to(torch.bfloat16).cuda()
    k = torch.randn((1, L, 64), generator=g).to(torch.bfloat16).cuda()
    w = torch.rand((1, 1, 16), generator=g).cuda()
    nv = torch.full((1, 1), L, dtype=torch.int32, device="cuda")
    want = {K: hb.dsa_flat_indexer_topk(q, w, k, nv, top_k=K, want_scores=True) for K in (16384, 16)}
    jobs = []
    for K in want:
        s = hb.make_shape(q, k, 1, 1, K)
        jobs.append(dict(K=K, s=s, stream=torch.cuda.Stream(), bad=[],
                         idx=torch.empty((1, 1, K), dtype=torch.int32, device="cuda"),
                         sc=torch.empty((1, 1, K), device="cuda"),
                         ws=torch.empty(max(16, hb.workspace_size(hb.OP_FLAT, s)), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(j):
        start.wait()
        for _ in range(calls):
            status = lib.dsa_flat_indexer_topk(q.data_ptr(), None, w.data_ptr(), k.data_ptr(), None, nv.data_ptr(),
                                               ctypes.byref(j["s"]), j["idx"].data_ptr(), j["sc"].data_ptr(),
                                               j["ws"].data_ptr(), j["ws"].numel(), j["stream"].cuda_stream)
            if status:
                j["bad"].append((status, lib.hisa_last_error()))
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    hb.get_status()
    for j in jobs:
        assert not j["bad"], f"top_k={j['K']}: {len(j['bad'])} of {calls} calls refused: {j['bad'][0]}"
        assert torch.equal(j["idx"], want[j["K"]][0]) and torch.equal(j["sc"], want[j["K"]][1])
