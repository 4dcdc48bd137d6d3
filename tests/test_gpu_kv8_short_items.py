"""Many sequences of one block of positions each on the tensor-memory attention kernel: the
items that give one of its two issuing warps no round, mixed with items that do.  And many
blocks of a few sequences whose pages' scales lie far apart, with the same bits every time."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,longer", [(64, 0), (128, 7), (64, 3)])
def test_many_short_sequences(dtype, D, longer):
    # 10 rows of 4 heads over 2 kv heads: a dozen items to a CTA; every `longer`-th sequence
    # has two to five blocks
    seqs = [(10, 10 + (b * 7) % 55 + (70 * (1 + b % 4) if longer and b % longer == 0 else 0))
            for b in range(900)]
    st = plain.make_state(seqs, 8, 2, D, 64, torch.int8, dtype, seed=21)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], 10)
    ref, tol = plain.attention(st["Q"], cache, st["table"], st["cu"], st["lens"], None, D ** -0.5)
    first = None
    for _ in range(5):
        out = wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], 10)
        err = (out.cpu().double() - ref).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert first is None or torch.equal(out, first)
        first = out


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 100), (torch.bfloat16, 12), (torch.float16, 40)])
@pytest.mark.parametrize("T", [16, 128])
def test_scales_of_many_blocks(dtype, n, T):
    # a block's scales are kept for eight blocks: each page on a scale of its own, so that a
    # block read with the scales of another shows
    st = plain.make_state([(n, 4000), (n, 2500), (n, 3111)], 8, 2, 64, T, torch.int8, dtype, seed=22)
    g = torch.Generator().manual_seed(5)
    for scales in st["cache"][1::2]:
        scales *= 2.0 ** torch.randint(-3, 4, scales.shape, generator=g)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], n)
    ref, tol = plain.attention(st["Q"], cache, st["table"], st["cu"], st["lens"], None, 0.02)
    outs = [wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], n, scale=0.02)
            for _ in range(20)]
    err = (outs[0].cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert all(torch.equal(o, outs[0]) for o in outs)
