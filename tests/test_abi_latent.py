"""Refusals of the entry points on the latent cache, without a GPU: every
check runs on the host before any HIP call; and the Python wrappers' own."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dsa_lightning_indexer_03_amd", "libdsaidx.so")

OK, NULL, SHAPE, DTYPE, UNSUP, WS = 0, 1, 2, 3, 4, 5
P = 4096  # a fake, 16-byte aligned, non-NULL device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.skip("libdsaidx.so not built")
    from dsa_lightning_indexer_03_amd import _lib
    return _lib.load(LIB)


def append(lib, kv=P, kvs=576, ik=P, iks=128, dt=1, cs=P, rl=100, rd=64, seq=P, pos=P, bt=P, B=1, mpp=2, lc=P,
           ls=None, ldt=1, kc=P, ks=P, npg=2, T=3, E=576, D=128, ps=64):
    return lib.indexer_cache_append_rope(kv, kvs, 1, ik, iks, 0, dt, cs, rl, rd, seq, pos, bt, B, mpp, lc, ls, ldt,
                                         kc, ks, npg, T, E, D, ps, None)


@pytest.mark.parametrize("kw,status", [
    (dict(kv=None), NULL), (dict(cs=None), NULL), (dict(seq=None), NULL), (dict(pos=None), NULL),
    (dict(bt=None), NULL), (dict(lc=None), NULL), (dict(dt=5), DTYPE), (dict(ldt=9), DTYPE), (dict(dt=2), UNSUP),
    (dict(ldt=0), UNSUP), (dict(ldt=2), SHAPE), (dict(ls=P), SHAPE), (dict(ik=None), SHAPE), (dict(kc=None), SHAPE),
    (dict(ks=None), SHAPE), (dict(T=-1), SHAPE), (dict(B=0), SHAPE), (dict(rl=0), SHAPE), (dict(D=64), UNSUP),
    (dict(ps=16), UNSUP), (dict(E=580), UNSUP), (dict(E=1032), UNSUP), (dict(rd=24), UNSUP), (dict(rd=144), UNSUP),
    (dict(E=48, kvs=48), UNSUP), (dict(kvs=570), SHAPE), (dict(iks=100), SHAPE), (dict(kvs=578), UNSUP),
    (dict(iks=130), UNSUP), (dict(dt=0, kvs=578), UNSUP), (dict(kv=P + 8), UNSUP), (dict(cs=P + 4), UNSUP),
    (dict(kc=P + 4), UNSUP), (dict(lc=P + 2), UNSUP), (dict(T=0), OK), (dict(T=0, kv=None), OK)])
def test_append_rope_rejects_before_launch(lib, kw, status):
    assert append(lib, **kw) == status
    assert status == OK or lib.dsaidx_last_error()


def topk(lib, q=P, qd=1, lc=P, ls=None, ldt=1, bt=P, mpp=4, npg=4, idx=P, seq=None, B=2, T=2, H=16, E=576, V=512,
         ps=64, K=100, scale=0.1, out=P, ws=P, nws=None):
    if nws is None:
        nws = lib.indexer_latent_attention_topk_workspace_bytes(T, H, E, V, K, ldt)
    return lib.indexer_latent_attention_topk(q, qd, lc, ls, ldt, bt, mpp, npg, idx, seq, B, T, H, E, V, ps, K, scale,
                                             out, None, ws, nws, None)


def shared(lib, q=P, qd=1, lc=P, ls=None, ldt=1, pt=P, np_=2, pl=100, bt=P, mpp=4, npg=4, cl=P, mcl=256, B=2, H=16,
           E=576, V=512, ps=64, scale=0.1, out=P, ws=P, nws=None):
    if nws is None:
        nws = lib.indexer_latent_attention_shared_workspace_bytes(B, H, E, V, pl, mcl, ldt)
    return lib.indexer_latent_attention_shared(q, qd, lc, ls, ldt, pt, np_, pl, bt, mpp, npg, cl, mcl, B, H, E, V, ps,
                                               scale, out, None, ws, nws, None)


COMMON = [
    (dict(q=None), NULL), (dict(lc=None), NULL), (dict(bt=None), NULL), (dict(out=None), NULL), (dict(qd=7), DTYPE),
    (dict(ldt=-1), DTYPE), (dict(qd=0), UNSUP), (dict(qd=2), UNSUP), (dict(ldt=0), UNSUP), (dict(ldt=2), SHAPE),
    (dict(ls=P), SHAPE), (dict(H=0), SHAPE), (dict(H=129), UNSUP), (dict(E=640), UNSUP), (dict(V=256), UNSUP),
    (dict(ps=32, mpp=8), UNSUP), (dict(npg=0), SHAPE), (dict(mpp=0), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=3e38), SHAPE), (dict(q=P + 8), UNSUP), (dict(lc=P + 8), UNSUP), (dict(out=P + 8), UNSUP),
    (dict(mpp=1 << 22), UNSUP), (dict(npg=1 << 22), UNSUP)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(idx=None), NULL), (dict(K=0), SHAPE), (dict(K=131073), UNSUP), (dict(T=3), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=1 << 21, seq=P), UNSUP), (dict(T=(1 << 23) + 1, H=1, seq=P), UNSUP), (dict(K=2048, ws=None), WS), (dict(K=2048, nws=8), WS),
    (dict(K=2048, ws=P + 8), UNSUP), (dict(T=0), OK), (dict(T=0, idx=None, q=None), OK), (dict(B=0), SHAPE)])
def test_topk_rejects_before_launch(lib, kw, status):
    assert topk(lib, **kw) == status
    assert status == OK or lib.dsaidx_last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(pt=None), NULL), (dict(cl=None), NULL), (dict(pl=129), SHAPE), (dict(pl=-1), SHAPE), (dict(np_=-1), SHAPE),
    (dict(mcl=257), SHAPE), (dict(mcl=-1), SHAPE), (dict(B=0), OK), (dict(B=-1), SHAPE), (dict(ws=None), WS), (dict(nws=8), WS),
    (dict(ws=P + 8), UNSUP)])
def test_shared_rejects_before_launch(lib, kw, status):
    assert shared(lib, **kw) == status
    assert status == OK or lib.dsaidx_last_error()


def test_wrappers_refuse(lib):
    """The wrappers' checks come before any device is touched."""
    import dsa_lightning_indexer_03_amd as dsa

    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16)
    q, idx = torch.zeros((1, 4, 576), dtype=torch.bfloat16), torch.zeros((1, 8), dtype=torch.int32)
    table, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        dsa.latent_attention_topk(q, cache, table, idx, 512, 1.0)
    with pytest.raises(ValueError, match="latent_cache must be"):
        dsa.latent_attention_topk(q, cache.float(), table, idx, 512, 1.0)
    with pytest.raises(ValueError, match="topk_idx must be"):
        dsa.latent_attention_topk(q, cache, table, idx.long(), 512, 1.0)
    with pytest.raises(ValueError, match="device"):
        dsa.latent_attention_shared(q, cache, None, 0, table, n, 512, 1.0)
    kv = torch.zeros((3, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        dsa.cache_append_rope(kv, n, n, table, cache, torch.zeros((4, 64)))


def test_workspace_sizes(lib):
    """The wrappers' sizes are the library's: none without splits, whole rows of sums and pairs with them."""
    import dsa_lightning_indexer_03_amd as dsa

    assert dsa.latent_topk_workspace_bytes(1000, 128, 576, 512, 64) == 0
    n = dsa.latent_topk_workspace_bytes(1, 16, 576, 512, 2048)
    assert n > 0 and n % (16 * 514 * 4) == 0
    assert n == lib.indexer_latent_attention_topk_workspace_bytes(1, 16, 576, 512, 2048, 1)
    n = dsa.latent_shared_workspace_bytes(3, 128, 512, 512, 30000, 100, fp8=True)
    assert n > 0 and n == lib.indexer_latent_attention_shared_workspace_bytes(3, 128, 512, 512, 30000, 100, 2)
