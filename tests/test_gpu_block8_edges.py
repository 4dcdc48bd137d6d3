"""Edges of the 8-bit quantizers: zeros keep their sign, an infinity saturates beside the
largest finite number, positions near the end of 32 bits are reported."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_plain as plain
from test_gpu_fp8_block import blocks_plain

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.uint8
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


def appended(st):
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                  d["rope"])
    want = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"],
                        st["rope"])
    return [t.cpu().view(torch.uint8) for t in d["cache"]], [t.view(torch.uint8) for t in want]


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_zeros_keep_their_sign_in_a_block(rows, dtype):
    """-0 / s is -0, whose E4M3 code is 0x80."""
    A = torch.randn(130, 400, generator=torch.Generator().manual_seed(1))
    A[::2, ::3] = -0.0
    A[1::2, 1::3] = 0.0
    A[5] = -0.0
    A = A.to(dtype)
    q, s = wq.quantize_fp8_block(A.cuda(), rows)
    oq, os_ = blocks_plain(A, rows)
    assert bool((oq == 0x80).any()) and bool((oq == 0).any())
    assert torch.equal(s.cpu(), os_) and torch.equal(q.cpu(), oq)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("inter", [None, False, True])
def test_zeros_keep_their_sign_in_the_cache(dtype, inter):
    rope = None if inter is None else (*plain.angles(64, 64), inter)
    st = plain.make_state([(9, 50), (1, 3)], 2, 2, 128, 16, E4, dtype, seed=2, rope=rope)
    for x in (st["K"], st["V"]):
        x[:, :, ::3] = -0.0
        x[2] = -0.0
        x[4] = 0.0
    got, want = appended(st)
    assert bool((want[2] == 0x80).any())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("code", [I8, E4])
def test_infinity_beside_the_largest_number_saturates(code):
    """The scale times 127 is above the largest fp32 number here."""
    top = torch.finfo(F32).max
    st = plain.make_state([(3, 20)], 2, 2, 64, 32, code, F32, seed=3)
    for x in (st["K"], st["V"]):
        x[0, 0, 3], x[0, 0, 4], x[1, 0, 5] = top, float("inf"), float("-inf")
        x[2, 1, 7], x[2, 1, 8] = float("inf"), -top
    got, want = appended(st)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_NONFINITE
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 30, 2 ** 31 - 33])
def test_append_reports_positions_near_the_end_of_32_bits(length):
    st = plain.make_state([(2, 50), (2, 60)], 2, 2, 64, 32, I8, BF, seed=6)
    st["lens"][1] = length
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], 2)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_ARG
    want = plain.append(st["K"], st["V"], st["cache"], st["table"][:1], st["cu"][:2],
                        st["lens"][:1], None)
    for a, b in zip(d["cache"], want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
