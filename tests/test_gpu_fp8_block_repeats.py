"""The few-token block product called over and over, on two streams at once: its ring of
weight tiles and scales goes round many times and its cut tiles are joined by whichever
warp comes last, with the same bits every time."""
import pytest
import torch

import bit_gemm_group_b200 as wq
from test_gpu_fp8_block import check_product
from workloads import make_activation, make_weight

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


@pytest.mark.parametrize("M,N,K", [(3, 1024, 8208), (24, 392, 11008), (60, 2056, 4112),
                                   (100, 392, 8208)])
def test_same_bits_every_time(M, N, K):
    X = make_activation(M, K, seed=M)
    # every block of 128 inputs on a scale of its own, so that a wrong scale shows
    scale = 2.0 ** torch.randint(-6, 7, (-(-K // 128),), generator=torch.Generator().manual_seed(K))
    X = (X.float() * scale.repeat_interleave(128)[:K]).to(torch.bfloat16)
    W = make_weight(N, K, 0.02, seed=N)
    qw, sw = wq.quantize_fp8_block(W.cuda(), 128)
    x = X.cuda()
    first = wq.gemm_fp8_block(x, qw, sw)
    check_product(X, W, first, qw, sw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(40):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(wq.gemm_fp8_block(x, qw, sw))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
