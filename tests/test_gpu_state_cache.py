"""State pages in 8 bits on the GPU: integers, scales and values against the oracle, bit for bit."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, gdn, host
from oracle import linear as ol
from train_util import DT

pytestmark = pytest.mark.gpu


def _pool(n, h, dk, dv, state, seed=0, pad=0, offset=0):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((n, h, dk, dv)) * np.exp(3 * rng.standard_normal((n, h, dk, 1)))
    size = h * dk * dv
    buf = torch.zeros(n * (size + pad) + offset, dtype=DT[state], device=DEV)
    t = buf[offset:].view(n, size + pad)[:, :size].view(n, h, dk, dv)
    t.copy_(torch.from_numpy(v).to(DEV))
    return gdn().StatePool(t)


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 3, 5), (3, 16, 64), (2, 40, 72), (1, 128, 128), (2, 7, 130), (1, 33, 63), (4, 8, 300)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (4, 4), (3, 1)])
def test_store_and_load(shape, state, pad, offset):
    g = gdn()
    h, dk, dv = shape
    dims = g.LinearDims(h, h, dk, dv, state_dtype=state)
    pool, back = _pool(5, h, dk, dv, state, pad=pad, offset=offset), _pool(5, h, dk, dv, state, seed=1, pad=pad, offset=offset)
    was = back.buf.clone()
    cache = g.StateCache.alloc(dims, 6, DEV)
    cache.q.fill_(99)
    cache.scale.fill_(-1.0)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.gdnl_cache_store(dims, i32(4, -1, 0, 4, 2), i32(1, 0, 5, 3, -1), pool, cache, err=err)
    n, sc, x = ol.cached(host(pool.buf))
    for page, entry in ((4, 1), (0, 5), (4, 3)):
        assert np.array_equal(cache.q[entry].cpu().numpy(), n[page])
        assert np.array_equal(cache.scale[entry].cpu().numpy(), sc[page])
    for entry in (0, 2, 4):
        assert (cache.q[entry] == 99).all() and (cache.scale[entry] == -1).all()
    g.gdnl_cache_load(dims, i32(5, 1, -1, 5), i32(3, 0, 1, 2), cache, back, err=err)
    exact = torch.from_numpy(x.astype(np.float32)).to(DT[state])  # a product of an integer and a scale, rounded once
    for page, source in ((3, 0), (0, 4), (2, 0)):
        if state == "f32":
            assert torch.equal(back.buf[page].cpu(), exact[source])
        else:  # rounded to fp32, then to bf16
            assert torch.equal(back.buf[page].cpu(), exact[source])
    assert torch.equal(back.buf[1], was[1]) and torch.equal(back.buf[4], was[4])
    assert int(err.item()) == 0


def test_an_error_is_at_most_half_a_scale():
    g = gdn()
    dims = g.LinearDims(2, 2, 64, 128)
    pool, back = _pool(2, 2, 64, 128, "f32"), _pool(2, 2, 64, 128, "f32", seed=1)
    cache = g.StateCache.alloc(dims, 2, DEV)
    idx = torch.arange(2, dtype=torch.int32, device=DEV)
    g.gdnl_cache_store(dims, idx, idx, pool, cache)
    g.gdnl_cache_load(dims, idx, idx, cache, back)
    off = np.abs(host(back.buf) - host(pool.buf)).reshape(2, 2, 64, 2, 64).max(-1)
    # half a scale, the product's half step, and the scales' own: 127 (up scale - 1) is three half steps of 127
    assert (off <= host(cache.scale) * (0.5 + 127 * 4 * 2.0 ** -24)).all()


@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_ends_of_the_range(state):
    g = gdn()
    dims = g.LinearDims(1, 1, 6, 70, state_dtype=state)
    pool = g.StatePool(torch.ones(1, 1, 6, 70, dtype=DT[state], device=DEV))
    top = torch.finfo(DT[state]).max
    rows = pool.buf[0, 0]
    rows[0, 3], rows[1, 66], rows[2, 0], rows[3, 0] = float("nan"), float("-inf"), top, -top
    rows[4] = 2.0 ** -101
    rows[5] = -0.0
    cache = g.StateCache.alloc(dims, 1, DEV)
    idx = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.gdnl_cache_store(dims, idx, idx, pool, cache)
    n, sc, x = ol.cached(host(pool.buf))
    assert np.array_equal(cache.q.cpu().numpy(), n) and np.array_equal(cache.scale.cpu().numpy(), sc, equal_nan=True)
    g.gdnl_cache_load(dims, idx, idx, cache, pool)
    got = host(pool.buf)[0, 0]
    assert np.isnan(got[0, :64]).all() and np.isfinite(got[0, 64:]).all() and np.isnan(got[1, 64:]).all()
    assert np.isfinite(got[2:]).all() and (got[4:] == 0).all()


def test_indexes_beyond_the_pool_and_the_cache():
    g = gdn()
    dims = g.LinearDims(1, 1, 4, 8)
    pool = _pool(2, 1, 4, 8, "f32")
    cache = g.StateCache.alloc(dims, 2, DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.gdnl_cache_store(dims, i32(2, 0), i32(0, 1), pool, cache, err=err)
    assert int(err.item()) == g.GDN_DEVERR_PAGE and (cache.q[0] == 0).all() and (cache.q[1] != 0).any()
    err.zero_()
    g.gdnl_cache_store(dims, i32(0), i32(2), pool, cache, err=err)
    assert int(err.item()) == g.GDN_DEVERR_CACHE
    err.zero_()
    was = pool.buf.clone()
    g.gdnl_cache_load(dims, i32(7, 0), i32(0, 9), cache, pool, err=err)
    assert int(err.item()) == g.GDN_DEVERR_CACHE | g.GDN_DEVERR_PAGE and torch.equal(pool.buf, was)


def test_captured():
    g = gdn()
    dims = g.LinearDims(2, 2, 64, 64)
    pool, back = _pool(3, 2, 64, 64, "f32"), _pool(3, 2, 64, 64, "f32", seed=1)
    cache = g.StateCache.alloc(dims, 3, DEV)
    idx, to = torch.arange(3, dtype=torch.int32, device=DEV), torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)

    def step():
        g.gdnl_cache_store(dims, idx, idx, pool, cache)
        g.gdnl_cache_load(dims, idx, to, cache, back)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        pool.buf.normal_()
        to.copy_(torch.roll(to, 1))
        step()
        torch.cuda.synchronize()
        want = back.buf.clone()
        back.buf.zero_()
        cache.q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back.buf, want)


def test_a_cache_beyond_4_gb():
    g = gdn()
    dims = g.LinearDims(32, 32, 128, 128, state_dtype="bf16")
    n = 8300  # entries of 512 KB
    cache = g.StateCache(torch.zeros(n, 32, 128, 128, dtype=torch.int8, device=DEV), torch.zeros(n, 32, 128, 2, device=DEV))
    pool = g.StatePool(torch.zeros(2, 32, 128, 128, dtype=torch.bfloat16, device=DEV))
    pool.buf[0].normal_()
    z, last, one = (torch.tensor([v], dtype=torch.int32, device=DEV) for v in (0, n - 1, 1))
    g.gdnl_cache_store(dims, z, last, pool, cache)
    g.gdnl_cache_load(dims, last, one, cache, pool)
    want = ol.cached(host(pool.buf[0, :1]))[2]
    assert np.array_equal(host(pool.buf[1, :1]), torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16).double().numpy())
    assert (cache.q[: n - 1] == 0).all()
