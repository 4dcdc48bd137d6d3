"""The attention kernels within the bound of their own roundings, queries in two f16 terms
where a kernel holds them so."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_bounds as bounds
import kv8_plain as plain

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.uint8
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


def check(st, d, cache, scale):
    out = wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                      scale=scale, rope=d["rope"])
    rows = st["max_new"] * (st["Q"].shape[1] // cache[0].shape[1])
    ref, tol = bounds.attention(st["Q"], cache, st["table"], st["cu"], st["lens"], st["rope"],
                                scale, rows)
    err = (out.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("dtype,n,G,D,T,past", [
    (HF, 2, 4, 64, 16, 70), (HF, 1, 8, 128, 64, 2000), (BF, 4, 8, 128, 32, 70),
    (HF, 5, 4, 256, 64, 300), (BF, 9, 4, 256, 16, 70),         # mma.sync
    (HF, 12, 4, 128, 64, 70), (HF, 40, 4, 64, 32, 1500),       # tcgen05, two terms
    (BF, 12, 4, 128, 64, 70), (BF, 100, 2, 64, 128, 900)])     # tcgen05, one term, one and two tiles
def test_results_that_hang_on_the_second_term(code, dtype, n, G, D, T, past):
    st, scale = bounds.split_state(plain, n, G, 2, D, T, code, dtype, seed=1, past=past)
    check(st, plain.on_gpu(st), st["cache"], scale)


@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,T,kv,G,seqs", [
    (64, 16, 2, 1, [(1, 1), (1, 64), (1, 200), (3, 3)]),
    (128, 64, 2, 8, [(1, 3000), (1, 65), (4, 130)]),
    (128, 32, 1, 16, [(2, 700), (1, 9)]),
    (256, 16, 1, 4, [(7, 400), (33, 100)]),
    (128, 128, 2, 4, [(12, 900), (9, 9), (1, 77)]),
    (64, 32, 1, 8, [(70, 1000), (3, 500), (0, 8), (16, 16)]),
    (128, 16, 1, 4, [(100, 1500), (64, 64)])])
def test_within_the_kernels_own_roundings(code, dtype, D, T, kv, G, seqs):
    rope = (*plain.angles(4000, D), False)
    st = plain.make_state(seqs, G * kv, kv, D, T, code, dtype, seed=D + T, rope=rope)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], rope)
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                  d["rope"])
    check(st, d, cache, D ** -0.5)
