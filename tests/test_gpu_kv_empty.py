"""Calls of the operators with grouped keys and values whose tensors have no
elements: torch gives such a tensor no address, and the library must not take it
for an argument that was left out."""
import os

import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dsa_lightning_indexer_03_amd", "libdsaidx.so")
OK, SHAPE = 0, 2
P = 4096  # a fake, 16-byte aligned, non-NULL device address (never dereferenced)


@pytest.mark.parametrize("B,idx,K,status", [(0, None, 5, OK), (0, P, 5, OK), (0, None, 0, OK), (2, None, 5, SHAPE),
                                            (0, None, -1, SHAPE), (0, P, 0, SHAPE), (0, P, -1, SHAPE)])
def test_a_selection_of_no_sequence(B, idx, K, status):
    if not os.path.exists(LIB):
        pytest.skip("libdsaidx.so not built")
    from dsa_lightning_indexer_03_amd import _lib

    assert _lib.load(LIB).indexer_kv_attention_decode(P, 1, P, None, P, None, 1, P, 4, 4, P, 256, idx, K, B, 16, 8,
                                                      128, 64, 0.1, P, None, None, 0, None) == status


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("K", [None, 1, 2048])
def test_a_step_of_no_sequence(K, kind):
    """A decode step of an empty batch, with and without a selection, gives empty results."""
    dev = torch.device("cuda")
    cache = torch.zeros((2, 2, 64, 128), dtype=torch.uint8 if kind == "fp8" else torch.bfloat16, device=dev)
    scale = torch.ones((2, 2, 64), device=dev) if kind == "fp8" else None
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)   # noqa: E731
    out, lse = dsa.kv_attention_decode(torch.zeros((0, 8, 128), dtype=torch.bfloat16, device=dev), cache, cache,
                                       ints(0, 3), ints(0), 0.1, topk_idx=None if K is None else ints(0, K),
                                       k_scale=scale, v_scale=scale, want_lse=True)
    torch.cuda.synchronize()
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(0, 64), (5, 0), (0, 0)])
def test_angles_of_no_position(shape):
    """An empty table of angles is refused: it is not the None that means no rotation."""
    dev = torch.device("cuda")
    cache = torch.zeros((1, 2, 64, 128), dtype=torch.bfloat16, device=dev)
    k = torch.ones((3, 2, 128), dtype=torch.bfloat16, device=dev)
    seq, pos = torch.zeros(3, dtype=torch.int32, device=dev), torch.arange(3, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="cos_sin"):
        dsa.kv_append_rope(k, k, seq, pos, seq[:1, None], cache, cache.clone(), cos_sin=torch.zeros(shape, device=dev))
    torch.cuda.synchronize()
    assert not cache.any()
