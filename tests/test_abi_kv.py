"""Refusals of the entry points with grouped keys and values, without a GPU:
every check runs on the host before any HIP call; and the Python wrappers' own."""
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


def append(lib, k=P, ks=1024, kh=128, v=P, vs=1024, vh=128, dt=1, cs=P, rl=100, rd=64, seq=P, pos=P, bt=P, B=1, mpp=2,
           kc=P, ksc=None, vc=P, vsc=None, cdt=1, npg=2, T=3, G=8, D=128, ps=64):
    return lib.indexer_kv_append_rope(k, ks, kh, v, vs, vh, dt, cs, rl, rd, 0, seq, pos, bt, B, mpp, kc, ksc, vc, vsc,
                                      cdt, npg, T, G, D, ps, None)


CACHES = [
    (dict(cdt=0), UNSUP), (dict(cdt=7), DTYPE), (dict(cdt=2), SHAPE), (dict(cdt=2, ksc=P), SHAPE),
    (dict(cdt=2, vsc=P), SHAPE), (dict(ksc=P), SHAPE), (dict(vsc=P), SHAPE), (dict(kc=None), NULL),
    (dict(vc=None), NULL), (dict(kc=P + 8), UNSUP), (dict(vc=P + 8), UNSUP), (dict(npg=0), SHAPE),
    (dict(D=96), UNSUP), (dict(D=0), SHAPE), (dict(ps=32, mpp=8), UNSUP), (dict(mpp=0), SHAPE),
    (dict(mpp=(1 << 21) + 1), UNSUP), (dict(npg=1 << 22), UNSUP), (dict(G=0), SHAPE)]


@pytest.mark.parametrize("kw,status", CACHES + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(seq=None), NULL), (dict(pos=None), NULL), (dict(bt=None), NULL),
    (dict(dt=2), UNSUP), (dict(dt=3), DTYPE), (dict(T=-1), SHAPE), (dict(B=0), SHAPE), (dict(rl=0), SHAPE),
    (dict(rd=0), SHAPE), (dict(rd=24), UNSUP), (dict(rd=144), UNSUP), (dict(G=129), UNSUP), (dict(k=P + 8), UNSUP),
    (dict(ks=1028), UNSUP), (dict(kh=132), UNSUP), (dict(vs=1028), UNSUP), (dict(vh=132), UNSUP),
    (dict(cs=P + 4), UNSUP), (dict(T=(1 << 23) + 1), UNSUP), (dict(T=0), OK), (dict(T=0, k=None, kc=None), OK)])
def test_append_rejects_before_launch(lib, kw, status):
    assert append(lib, **kw) == status
    assert status == OK or lib.dsaidx_last_error()


def prompt(lib, q=P, qs=2048, qh=128, k=P, ks=1024, kh=128, v=P, vs=1024, vh=128, dt=1, cu=P, B=2, T=100, H=16, G=8,
           D=128, V=128, scale=0.1, out=P):
    return lib.indexer_prompt_attention(q, qs, qh, k, ks, kh, v, vs, vh, dt, cu, B, T, H, G, D, V, scale, out, None,
                                        None)


HEADS = [(dict(H=0), SHAPE), (dict(G=0), SHAPE), (dict(H=12), SHAPE), (dict(H=4), SHAPE), (dict(H=136), UNSUP),
         (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=3e38), SHAPE)]


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(cu=None), NULL), (dict(out=None), NULL),
    (dict(dt=0), UNSUP), (dict(dt=2), UNSUP), (dict(dt=9), DTYPE), (dict(T=-1), SHAPE), (dict(B=0), SHAPE),
    (dict(D=64), UNSUP), (dict(V=64), UNSUP), (dict(D=192, V=192), UNSUP), (dict(q=P + 8), UNSUP),
    (dict(out=P + 8), UNSUP), (dict(qs=2052), UNSUP), (dict(kh=4), UNSUP), (dict(ks=1 << 24), UNSUP),
    (dict(vs=-8), UNSUP), (dict(T=1 << 30), UNSUP), (dict(B=1 << 30), UNSUP), (dict(T=0), OK),
    (dict(T=0, q=None), OK)])
def test_prompt_rejects_before_launch(lib, kw, status):
    assert prompt(lib, **kw) == status
    assert status == OK or lib.dsaidx_last_error()


def decode(lib, q=P, qd=1, kc=P, ksc=None, vc=P, vsc=None, cdt=1, bt=P, mpp=4, npg=4, cl=P, mcl=256, idx=None, K=0,
           B=2, H=16, G=8, D=128, ps=64, scale=0.1, out=P, ws=P, nws=None):
    if nws is None:
        nws = lib.indexer_kv_attention_decode_workspace_bytes(B, H, G, D, max(mcl, 0), max(K, 0), cdt)
    return lib.indexer_kv_attention_decode(q, qd, kc, ksc, vc, vsc, cdt, bt, mpp, npg, cl, mcl, idx, K, B, H, G, D, ps,
                                           scale, out, None, ws, nws, None)


@pytest.mark.parametrize("kw,status", CACHES + HEADS + [
    (dict(q=None), NULL), (dict(bt=None), NULL), (dict(cl=None), NULL), (dict(out=None), NULL), (dict(qd=0), UNSUP),
    (dict(qd=2), UNSUP), (dict(qd=-1), DTYPE), (dict(B=-1), SHAPE), (dict(mcl=257), SHAPE), (dict(mcl=-1), SHAPE),
    (dict(K=5), SHAPE), (dict(idx=P), SHAPE), (dict(idx=P, K=-3), SHAPE), (dict(idx=P, K=131073), UNSUP),
    (dict(B=(1 << 19) + 1), UNSUP), (dict(q=P + 8), UNSUP), (dict(out=P + 8), UNSUP),
    (dict(mpp=512, npg=512, mcl=32768, ws=None), WS), (dict(mpp=512, npg=512, mcl=32768, nws=64), WS),
    (dict(mpp=512, npg=512, mcl=32768, ws=P + 8), UNSUP), (dict(B=0), OK), (dict(B=0, q=None, kc=None), OK)])
def test_decode_rejects_before_launch(lib, kw, status):
    assert decode(lib, **kw) == status
    assert status == OK or lib.dsaidx_last_error()


def test_workspace_sizes(lib):
    """None for one run; whole rows of sums and pairs for several; every size of a
    call that is refused anyway is 0."""
    import dsa_lightning_indexer_03_amd as dsa

    assert dsa.kv_decode_workspace_bytes(1, 32, 8, 128, 100) == 0
    for D in (64, 128):
        n = dsa.kv_decode_workspace_bytes(2, 32, 8, D, 131072, fp8=True)
        assert n > 0 and n % (2 * 32 * (D + 2) * 4) == 0
        assert n == lib.indexer_kv_attention_decode_workspace_bytes(2, 32, 8, D, 131072, 0, 2)
    assert dsa.kv_decode_workspace_bytes(1, 32, 8, 128, 131072, topk=64) == 0
    for bad in ((0, 32, 8, 128, 9), (1, 32, 0, 128, 9), (1, 4, 8, 128, 9), (1, 32, 8, 96, 9), (1, 32, 8, 128, -1)):
        assert dsa.kv_decode_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("B,H,G,len_", [(1, 1, 1, 1 << 27), (1 << 23, 1, 1, 1 << 12), (1 << 16, 128, 128, 1 << 20),
                                        (1 << 20, 8, 1, 1 << 27)])
def test_largest_plans_fit_a_launch(lib, B, H, G, len_):
    """A launch holds less than 2^32 threads: runs times workgroups of a run stay under 2^24 of 256."""
    n = lib.indexer_kv_attention_decode_workspace_bytes(B, H, G, 128, len_, 0, 1)
    slots = max(1, n // (B * H * 130 * 4))
    assert slots * B * G * 256 < 1 << 32


def test_wrappers_refuse(lib):
    """The wrappers' checks come before any device is touched."""
    import dsa_lightning_indexer_03_amd as dsa

    q, k = torch.zeros((3, 4, 128), dtype=torch.bfloat16), torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    cache, n, table = torch.zeros((2, 2, 64, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), \
        torch.zeros((3, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        dsa.prompt_attention(q, k, k, n, 1.0)
    with pytest.raises(ValueError, match="q must be"):
        dsa.prompt_attention(q.float(), k, k, n, 1.0)
    with pytest.raises(ValueError, match="device"):
        dsa.kv_attention_decode(q, cache, cache, table, n, 1.0)
    with pytest.raises(ValueError, match="k_cache must be"):
        dsa.kv_attention_decode(q, cache.float(), cache, table, n, 1.0)
    with pytest.raises(ValueError, match="caches"):
        dsa.kv_attention_decode(q, cache[0], cache, table, n, 1.0)
    with pytest.raises(ValueError, match="device"):
        dsa.kv_append_rope(k, k, n, n, table, cache, cache)
    with pytest.raises(ValueError, match="k must be"):
        dsa.kv_append_rope(k.half(), k, n, n, table, cache, cache)


def test_workspace_queries_of_nothing(lib):
    """A bound or a list of length 0 and 1 are sizes like others."""
    import dsa_lightning_indexer_03_amd as dsa

    for B in (1, 300, 5000):
        for fp8 in (False, True):
            for n in (0, 1, 32, 33, 512, 513, 1024, 1025):
                assert dsa.kv_decode_workspace_bytes(B, 8, 2, 64, n, fp8=fp8) % (B * 8 * 66 * 4) == 0
                assert dsa.kv_decode_workspace_bytes(B, 8, 2, 128, 64, topk=n, fp8=fp8) % (B * 8 * 130 * 4) == 0
