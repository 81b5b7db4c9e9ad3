"""Calls of the 8-bit cache that its documentation allows and that ordinary use makes seldom: pools of one
page, other storage orders, lengths outside their range, more row blocks than a CTA has threads,
scales at the ends of fp32, two threads at once."""
import threading

import numpy as np
import pytest
import torch

import cache_reference as ref
from test_cache_gpu import DEV, FILL, Cache, attend, fa2, i32, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 128])
def test_a_pool_of_one_page(D, page):
    """One page, one head, one sequence: strides of dimensions of size one are never used."""
    c = Cache(1, 1, D, page, [page - 1], seed=D + page, spare=0, nan_after=False)
    dev = c.device()
    assert c.N == 1
    x = ref.bf16(c.rng.standard_normal((1, 1, 5, D)))
    fa2().fa2_cache_write(x.to(DEV), x.to(DEV), *dev, i32([page - 6]))
    for codes, scale in ((c.k, c.ks), (c.v, c.vs)):
        ref.write(x.double().numpy(), codes, scale, c.table, [page - 6], [5])
    for got, want in zip(dev[:4], (c.k, c.v, c.ks, c.vs)):
        same(got, want)
    attend(c, 1, 1, [page - 1], dev=dev)
    attend(c, 20, 1, [page - 1], dev=dev)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Lq", [(4, 1), (4, 20)])
def test_other_storage(D, G, Lq):
    """Head-major storage, rows inside wider ones, keys and values in one buffer, scales as plain bytes."""
    lens, H = [200, 77], 2
    c = Cache(2, H, D, 32, lens, seed=D + Lq)
    head_major = torch.from_numpy(c.k).to(DEV).permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    both = torch.zeros(c.N, H, 32, 2 * D, dtype=torch.uint8, device=DEV)
    both[..., :D], both[..., D:] = torch.from_numpy(c.k).to(DEV), torch.from_numpy(c.v).to(DEV)
    ks, vs = (torch.from_numpy(s).to(DEV) for s in (c.ks, c.vs))
    table = c.device()[4]
    v = both[..., D:].view(torch.float8_e4m3fn)
    for k in (head_major.view(torch.float8_e4m3fn), both[..., :D].view(torch.float8_e4m3fn)):
        attend(c, G, Lq, lens, dev=(k, v, ks, vs, table))
        back = [torch.zeros(2, H, 200, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        fa2().fa2_cache_read(k, v, ks, vs, table, *back, i32([0, 0]), i32(lens))
        for t, codes, scale in zip(back, (c.k, c.v), (c.ks, c.vs)):
            for h in range(H):
                np.testing.assert_array_equal(t[1, h, :77].double().cpu().numpy(), ref.gather(codes, scale, c.table[1], h, 77)[0])


@pytest.mark.parametrize("Lq", [1, 9, 40])
def test_query_lengths_outside_their_range(Lq):
    lens = [60, 60, 60, 60]
    c = Cache(4, 1, 64, 16, lens, seed=Lq)
    attend(c, 2, Lq, lens, [Lq + 5, -3, 2 ** 31 - 1, -2 ** 31])


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("workspace", [False, True])
def test_more_row_blocks_than_threads(D, workspace):
    """Room for 2000 rows a sequence, few of them used: a thread lays out several row blocks of the line."""
    B, Lq = 130, 2000
    rng = np.random.default_rng(D)
    lens, q_lens = rng.integers(1, 60, B), rng.integers(0, 4, B)
    lens[[3, 77]], q_lens[[3, 77]] = 700, [300, 601]
    c = Cache(B, 1, D, 16, lens, seed=D)
    attend(c, 1, Lq, lens, q_lens, workspace=workspace)


@pytest.mark.parametrize("G,Lq", [(4, 1), (4, 20)])
@pytest.mark.parametrize("log2", [-100, -30, 30, 100])
def test_scales_of_any_size(G, Lq, log2):
    """The scale 2^log2 times the usual one, and q as much smaller: the same answer."""
    lens = [150, 40]
    c = Cache(2, 1, 128, 16, lens, seed=7, nan_after=False)
    q = ref.bf16(c.rng.standard_normal((2, G, Lq, 128)))
    attend(c, G, Lq, lens, q=q * 2.0 ** -log2, scale=2.0 ** (log2 - 3.5))


def test_two_threads_at_once():
    """Calls from two host threads, each on its own stream with its own workspace, give each its own bits."""
    jobs = []
    for G, Lq, D in [(4, 1, 128), (2, 40, 64)]:
        lens = [900, 333]
        c = Cache(2, 2, D, 32, lens, seed=D)
        q = ref.bf16(c.rng.standard_normal((2, 2 * G, Lq, D)))
        dev = c.device()
        o, lse = attend(c, G, Lq, lens, q=q, dev=dev)
        qd = q.to(DEV)
        jobs.append((dev, qd, i32(lens), o, lse, fa2().fa2_cache_attn_workspace(qd, dev[0]), torch.cuda.Stream(DEV)))
    torch.cuda.synchronize()
    wrong = []

    def work(dev, qd, kv, o, lse, ws, stream):
        with torch.cuda.stream(stream):
            for _ in range(200):
                o2, lse2 = torch.full_like(o, FILL), torch.full_like(lse, FILL)
                fa2().fa2_cache_attn(qd, *dev, kv, o2, lse2, workspace=ws)
                if not (torch.equal(o, o2) and torch.equal(lse, lse2)):
                    wrong.append(tuple(qd.shape))

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert fa2().fa2_cache_get_device_error() == (0, 0)
