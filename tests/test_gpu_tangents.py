"""Inputs with a forward-mode tangent are refused by the calls that have no
derivative, as inputs that want a gradient are: the result would have lost it."""
import pytest
import torch
from torch.autograd import forward_ad

import dsa_lightning_indexer_03_amd as dsa

CALLS = ["prompt_attention", "kv_append_rope", "kv_attention_decode", "cache_append_rope", "latent_attention_topk",
         "latent_attention_shared"]


def test_the_check():
    x = torch.ones(3)
    ints = torch.ones(3, dtype=torch.int16)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones(3))
        for inputs in ((dual,), (None, ints, dual), (x, dual[1:])):
            with pytest.raises(ValueError, match="call has no forward derivative"):
                dsa._inference_only("call", *inputs)
            with torch.no_grad(), pytest.raises(ValueError, match="call has no forward derivative"):
                dsa._inference_only("call", *inputs)
        dsa._inference_only("call", x, None, ints, forward_ad.unpack_dual(dual).primal)
    dsa._inference_only("call", dual)      # (the level is over, and the tangent with it)
    y = torch.ones(3, requires_grad=True)
    with pytest.raises(ValueError, match="call has no backward"):
        dsa._inference_only("call", None, y)
    with torch.no_grad():
        dsa._inference_only("call", y)


def call(name, wrap):
    """One call; wrap(tensor) for the input that may have a tangent."""
    r = lambda *s: torch.randn(s, device="cuda").bfloat16()   # noqa: E731
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    if name == "prompt_attention":
        return dsa.prompt_attention(r(5, 4, 64), r(5, 2, 64), wrap(r(5, 2, 64)), i(0, 5), 0.1)
    if name == "kv_append_rope":
        return dsa.kv_append_rope(wrap(r(2, 2, 64)), r(2, 2, 64), i(0, 0), i(0, 1), i([0]), r(1, 2, 64, 64), r(1, 2, 64, 64))
    if name == "kv_attention_decode":
        return dsa.kv_attention_decode(wrap(r(1, 4, 64)), r(1, 2, 64, 64), r(1, 2, 64, 64), i([0]), i(5), 0.1)
    if name == "cache_append_rope":
        return dsa.cache_append_rope(wrap(r(2, 576)), i(0, 0), i(0, 1), i([0]), r(1, 64, 576), torch.ones((9, 64), device="cuda"))
    if name == "latent_attention_topk":
        return dsa.latent_attention_topk(r(1, 4, 576), wrap(r(1, 64, 576)), i([0]), i([0, 3]), 512, 0.1)
    return dsa.latent_attention_shared(wrap(r(1, 4, 576)), r(1, 64, 576), None, 0, i([0]), i(5), 512, 0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_calls_refuse_a_tangent(name):
    call(name, lambda t: t)
    torch.cuda.synchronize()
    with forward_ad.dual_level():
        call(name, lambda t: t)            # no input has a tangent
        for mode in (torch.enable_grad, torch.no_grad):
            with mode(), pytest.raises(ValueError, match=name + " has no forward derivative"):
                call(name, lambda t: forward_ad.make_dual(t, torch.ones_like(t)))
    torch.cuda.synchronize()
