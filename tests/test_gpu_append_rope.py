"""GPU parity of cache_append_rope against the fp64 oracle: stored bf16 values
within half a step of the rotated value (plus the fp32 rotation's own error),
fp8 codes between the codes of the rotated value's error interval, columns that
are not rotated and slots that no token addresses exactly as they should be."""
import numpy as np
import pytest
import torch

import dsa_lightning_indexer_03_amd as dsa
from gpu_util import say
from latent_util import bf16
from oracle.formats import fp8_e4m3_to_f64
from oracle.kcache import encode_e4m3
from oracle.latent import U16, U32, rotate, slots

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check_fp8(codes, scale, y, err, where):
    """Rows of codes and scales against the rotated fp64 rows y, known within err."""
    hi = (np.abs(y) + err).max(1) / 448 * (1 + 2 * U32)
    lo = np.maximum(np.abs(y) - err, 0).max(1) / 448 * (1 - 2 * U32)
    zero = (y == 0).all(1)
    lo, hi = np.where(zero, 1.0, lo), np.where(zero, 1.0, hi)
    assert ((scale >= lo) & (scale <= hi)).all(), f"{where}: scales"
    s = scale.astype(np.float64)[:, None]
    got = fp8_e4m3_to_f64(codes)
    # the fp32 quotient is off by half a step; encoding is monotone
    low = fp8_e4m3_to_f64(encode_e4m3((y - err) / s - 2 * U32 * np.abs(y / s)))
    top = fp8_e4m3_to_f64(encode_e4m3((y + err) / s + 2 * U32 * np.abs(y / s)))
    assert ((got >= low) & (got <= top)).all(), f"{where}: codes"


CASES = [  # T, B, E, R, input, cache, index, kv_pairs, index_pairs
    (1, 1, 576, 64, "bf16", "bf16", True, True, False),
    (1, 1, 512, 64, "f32", "fp8", False, False, False),
    (3, 2, 576, 64, "f32", "bf16", True, False, True),
    (257, 5, 576, 64, "bf16", "fp8", True, True, True),
    (130, 3, 512, 32, "bf16", "bf16", True, True, False),
    (75, 2, 1024, 128, "f32", "fp8", True, False, False),
    (64, 1, 64, 64, "bf16", "bf16", False, True, False),
    (33, 4, 16, 16, "bf16", "fp8", True, False, True),
    (500, 7, 520, 48, "f32", "bf16", True, False, False),
]


@pytest.mark.parametrize("T,B,E,R,inp,kind,index,kp,ip", CASES)
def test_against_the_oracle(T, B, E, R, inp, kind, index, kp, ip):
    rng = np.random.default_rng(T * 31 + E + R)
    say(f"append_rope T={T} B={B} E={E} R={R} {inp}->{kind} index={index} pairs={kp},{ip}")
    mpp = 6
    pages = B * mpp + 2
    table = rng.permutation(pages)[: B * mpp].reshape(B, mpp).astype(np.int32)
    table[-1, -1] = pages + 5                                     # not a page of the pool
    table[0, -1] = -1
    seq = rng.integers(0, B, T).astype(np.int32)
    # distinct positions within each sequence, some of them outside everything
    pos = np.zeros(T, np.int32)
    for b in range(B):
        who = np.flatnonzero(seq == b)
        pos[who] = rng.permutation(mpp * 64 + 20)[: who.size]
    if T > 2:
        seq[0], seq[1], pos[2] = -1, B, -7
    rope_len = mpp * 64 - 30                                      # the last positions have no angle
    ang = np.arange(rope_len)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    # rows cut out of a wider projection
    wide = rng.normal(size=(T, E + 128 + 16)) * np.exp(rng.normal(size=(T, 1)))
    if T > 5:
        wide[5] = 0
    src, val = bf16(wide) if inp == "bf16" else (torch.from_numpy(wide.astype(np.float32)),
                                                 wide.astype(np.float32).astype(np.float64))
    src = src.cuda()
    kv, ik = src[:, :E], src[:, E:E + 128] if E % 8 == 0 else None
    latent0 = torch.from_numpy(rng.integers(0, 120, size=(pages, 64, E * (2 if kind == "bf16" else 1))).astype(np.uint8)).cuda()
    latent = latent0.clone().view(torch.bfloat16) if kind == "bf16" else latent0.clone()
    scale0 = torch.rand((pages, 64), device="cuda")
    lscale = scale0.clone() if kind == "fp8" else None
    kc0 = torch.from_numpy(rng.integers(0, 120, size=(pages, 64, 128)).astype(np.uint8)).cuda()
    kc, ks = (kc0.clone(), scale0.clone()) if index else (None, None)
    dsa.cache_append_rope(kv, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                          torch.from_numpy(table).cuda(), latent, torch.from_numpy(cs).cuda(), latent_scale=lscale,
                          kv_interleaved=kp, index_k=ik if index else None, k_cache=kc, k_scale=ks,
                          index_interleaved=ip)
    torch.cuda.synchronize()
    at = slots(seq, pos, table, pages, rope_len)
    live = at >= 0
    at = at[live]
    turn = cs[pos[live]]
    other = np.ones(pages * 64, bool)
    other[at] = False
    y, err = rotate(val[live, :E], turn, E - R, kp)
    if kind == "bf16":
        full = latent.view(pages * 64, E)
        got = full.double().cpu().numpy()[at]
        tol = np.where(err > 0, U16 * (np.abs(y) + err) + err, 0.0 if inp == "bf16" else U16 * np.abs(y))
        assert (np.abs(got - y) <= tol).all()
    else:
        full = latent.view(pages * 64, E)
        check_fp8(full.cpu().numpy()[at], lscale.view(-1).cpu().numpy()[at], y, err, "latent")
        assert torch.equal(lscale.view(-1).cpu()[other], scale0.view(-1).cpu()[other])
    assert torch.equal(latent.view(torch.uint8).view(pages * 64, -1).cpu()[other], latent0.view(pages * 64, -1).cpu()[other])
    if index:
        y, err = rotate(val[live, E:E + 128], turn, 0, ip)
        check_fp8(kc.view(-1, 128).cpu().numpy()[at], ks.view(-1).cpu().numpy()[at], y, err, "index key")
        assert torch.equal(kc.view(-1, 128).cpu()[other], kc0.view(-1, 128).cpu()[other])
        assert torch.equal(ks.view(-1).cpu()[other], scale0.view(-1).cpu()[other])


def test_without_a_turn_it_is_kcache_append():
    """Angle 0 everywhere: the index key's codes and scales are kcache_append's, bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, pages = 300, 8
    kv = torch.randn((T, 576), generator=g, device="cuda", dtype=torch.bfloat16)
    ik = torch.randn((T, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    cs = torch.cat([torch.ones(512, 32), torch.zeros(512, 32)], 1).cuda()
    seq, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    a, sa = torch.zeros((pages, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((pages, 64), device="cuda")
    b, sb = a.clone(), sa.clone()
    latent = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    dsa.kcache_append(ik, seq, pos, table, a, sa)
    dsa.cache_append_rope(kv, seq, pos, table, latent, cs, index_k=ik, k_cache=b, k_scale=sb)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(sa, sb)
    assert torch.equal(latent.flip(0).reshape(-1, 576)[:T], kv)


def test_no_tokens_is_a_no_op():
    z = torch.zeros((0, 576), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    latent = torch.ones((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    dsa.cache_append_rope(z, i, i, torch.zeros((1, 2), dtype=torch.int32, device="cuda"), latent,
                          torch.ones((4, 64), device="cuda"))
    torch.cuda.synchronize()
    assert bool((latent == 1).all())


def test_pool_beyond_32_bit_offsets():
    """Slots whose byte offsets pass 2^32 (a 5.4 GB latent pool)."""
    pages, E = 73000, 576
    latent = torch.empty((pages, 64, E), dtype=torch.bfloat16, device="cuda")
    T = 64
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    latent[0].fill_(3)
    kv = torch.randn((T, E), device="cuda", dtype=torch.bfloat16)
    cs = torch.cat([torch.ones(64, 32), torch.zeros(64, 32)], 1).cuda()
    seq, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    say("append_rope into the last page of a 5.4 GB pool")
    dsa.cache_append_rope(kv, seq, pos, table, latent, cs)
    torch.cuda.synchronize()
    assert torch.equal(latent[-1], kv) and bool((latent[0] == 3).all())
