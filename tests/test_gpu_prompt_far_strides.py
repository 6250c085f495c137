"""prompt_attention where tokens lie as far apart as a call takes, 2^24 - 8
elements: a tile's rows then span all but 2^25 bytes of the 32 bits that address
them.  Every result is that of contiguous copies, bit for bit."""
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from kv_util import ints

pytestmark = pytest.mark.gpu
STRIDE = (1 << 24) - 8


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# blocks of 64 rows and four key groups of 32 (tiles of 128 keys), 128 rows and two of 64,
# one of 64, one of 32: by the numbers of blocks and the mean length
FORMS = [("128 keys, blocks of 64", [300], 2, 1), ("128 keys, blocks of 128", [600], 64, 2),
         ("64 keys", [199, 101], 128, 4), ("32 keys", [35, 31, 40, 33, 30, 37, 1, 33, 60], 128, 2)]


@pytest.mark.parametrize("D,V", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("name,lens,H,G", FORMS, ids=[f[0] for f in FORMS])
def test_rows_as_far_apart_as_a_call_takes(name, lens, H, G, D, V):
    T = sum(lens)
    rows = torch.empty(T * STRIDE, dtype=torch.bfloat16, device="cuda")   # (only the heads' columns are written)
    place, views, copies = 0, [], []
    for heads, cols in ((H, D), (G, D), (G, V)):
        x = torch.randn((T, heads, cols), device="cuda").bfloat16()
        far = torch.as_strided(rows, (T, heads, cols), (STRIDE, cols, 1), place)
        far.copy_(x)
        views.append(far)
        copies.append(x)
        place += heads * cols
    cu = ints([0] + list(torch.tensor(lens).cumsum(0)))
    say(f"rows {STRIDE} elements apart: {name}, {D} and {V} columns")
    want = dsa.prompt_attention(*copies, cu, D ** -0.5, want_lse=True)
    got = dsa.prompt_attention(*views, cu, D ** -0.5, want_lse=True)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b) and bool(a.isfinite().all())
    with pytest.raises(RuntimeError, match="2\\^24"):
        dsa.prompt_attention(torch.as_strided(rows, (2, H, D), (1 << 24, D, 1), 0), copies[1][:2], copies[2][:2],
                             ints([0, 2]), 0.1)
