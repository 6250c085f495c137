"""indexer_kv_attention_decode_workspace_bytes, without a GPU: 0 for every size that
the call refuses, however large, and whole rows of sums and pairs for the others."""
import itertools
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dsa_lightning_indexer_03_amd", "libdsaidx.so")

BF16, FP8, WS = 1, 2, 5
P = 4096  # a fake, 16-byte aligned, non-NULL device address (never dereferenced)
MAX = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.skip("libdsaidx.so not built")
    from dsa_lightning_indexer_03_amd import _lib
    return _lib.load(LIB)


def query(lib, B=2, H=16, G=8, D=128, n=131072, topk=0, dt=BF16):
    return lib.indexer_kv_attention_decode_workspace_bytes(B, H, G, D, n, topk, dt)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=-1), dict(B=MAX), dict(H=0), dict(G=0), dict(G=-1), dict(H=12), dict(H=4), dict(H=136, G=8),
    dict(H=128, G=127), dict(D=96), dict(D=0), dict(n=-1), dict(n=(1 << 27) + 1), dict(n=MAX), dict(topk=-1),
    dict(topk=131073), dict(topk=MAX), dict(dt=0), dict(dt=7),
    # 2^24 workgroups and more for one run of each sequence, with a head each and with shared ones
    dict(B=262144, H=64, G=64, D=64, n=64), dict(B=1 << 24, H=1, G=1, n=64), dict(B=1 << 24, H=1, G=1, n=64, topk=1),
    dict(B=(1 << 23) + 1, H=1, G=1, n=1), dict(B=1 << 20, H=128, G=1, n=1 << 27), dict(B=MAX, H=128, G=128, n=MAX)])
def test_sizes_that_the_call_refuses(lib, kw):
    for dt in (BF16, FP8):
        assert query(lib, **{"dt": dt, **kw}) == 0


EDGES = [0, 1, 2, 63, 64, 65, 127, 128, (1 << 16) - 1, 1 << 17, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, 1 << 24,
         1 << 27, (1 << 27) + 1, MAX]


def test_every_edge_returns(lib):
    """Combinations of edges: a size of whole rows, of at most 512 runs, and of a launch of fewer than 2^32 threads."""
    for B, n, topk, (H, G), dt in itertools.product(EDGES, EDGES, (0, 1, 64, 131072), ((1, 1), (64, 64), (128, 1)),
                                                    (BF16, FP8)):
        size = query(lib, B=B, H=H, G=G, D=64, n=n, topk=topk, dt=dt)
        if B < 1 or B * H > 1 << 23 or n > 1 << 27:
            assert size == 0
            continue
        slots, rest = divmod(size, B * H * 66 * 4)
        assert rest == 0 and slots != 1 and slots <= 512
        assert max(slots, 1) * B * G * (2 if H // G > 64 else 1) * 256 < 1 << 32


@pytest.mark.parametrize("D,dt,cut", [(64, BF16, 131072), (128, BF16, 131072), (64, FP8, 131072), (128, FP8, 131072)])
def test_a_split_call_needs_its_size(lib, D, dt, cut):
    """A lone context of 131072 is split; the call takes no byte less than the size."""
    n = query(lib, B=1, H=16, G=8, D=D, n=cut, dt=dt)
    slots = n // (16 * (D + 2) * 4)
    assert slots >= 2 and n == slots * 16 * (D + 2) * 4
    sc = P if dt == FP8 else None
    for ws, nws in ((P, n - 1), (None, n)):
        assert lib.indexer_kv_attention_decode(P, BF16, P, sc, P, sc, dt, P, 2048, 2048, P, cut, None, 0, 1, 16, 8, D,
                                               64, 0.1, P, None, ws, nws, None) == WS
    assert query(lib, B=1, H=16, G=8, D=D, n=100, dt=dt) == 0


@pytest.mark.gpu
def test_the_wrapper_refuses_too_many_rows():
    """The size is asked for before the call's own checks: it is 0, and the call says what it refuses."""
    import dsa_lightning_indexer_03_amd as dsa

    B = 1 << 24
    q = torch.zeros((B, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((1, 1, 64, 64), dtype=torch.bfloat16, device="cuda")
    ints = torch.zeros(B, dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError, match="2\\^23"):
        dsa.kv_attention_decode(q, cache, cache, ints[:, None], ints, 0.1)
