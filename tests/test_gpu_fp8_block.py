"""Block-scaled FP8 on the GPU: codes and scales bit-exact against a plain
implementation, the product against 64-bit sums of the same codes."""
import numpy as np
import pytest
import torch

import bit_gemm_group_b200 as wq
from workloads import make_activation, make_weight

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


def blocks_plain(A, rows):
    """(codes, scales) on the CPU, every step in fp32 as the definition has it."""
    R, K = A.shape
    p = torch.nn.functional.pad(A.float(), (0, -K % 128, 0, -R % rows))
    p = p.view(p.shape[0] // rows, rows, p.shape[1] // 128, 128)
    s = torch.div(p.abs().amax((1, 3)), torch.tensor(448.0)).clamp(min=1e-8)
    q = torch.div(p, s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(-1, p.shape[2] * 128)[:R, :K].contiguous().view(torch.uint8), s


def values64(q, s, rows):
    v = q.cpu().view(torch.float8_e4m3fn).double()
    w = s.cpu().double().repeat_interleave(128, 1)[:, :q.shape[1]]
    return v, w.repeat_interleave(rows, 0)[:q.shape[0]]


def check_product(X, W, Y, qw, sw):
    """|Y - exact| <= 2^-8 |exact| (the bf16 rounding) + fp32 sums: 128 products per
    block and one scaled addition per block, each within 2^-23 of the magnitudes."""
    qx, sx = blocks_plain(X, 1)
    vx, ax = values64(qx, sx, 1)
    vw, aw = values64(qw, sw, 128)
    x, w = (vx * ax).cuda(), (vw * aw).cuda()
    exact, mag = x @ w.t(), x.abs() @ w.t().abs()
    kb = -(-X.shape[1] // 128)
    tol = 2.0 ** -8 * exact.abs() + (128 + kb + 4) * 2.0 ** -23 * mag + 1e-30
    err = (Y.double() - exact).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("R,K", [(1, 16), (3, 128), (37, 1040), (130, 272), (1000, 4096)])
def test_quantize_bitexact(dtype, rows, R, K):
    A = make_activation(R, K, seed=R + K, outlier_dims=min(6, K // 16), dtype=dtype)
    A[R // 2, : K // 2] = 0
    q, s = wq.quantize_fp8_block(A.cuda(), rows)
    oq, os_ = blocks_plain(A, rows)
    np.testing.assert_array_equal(s.cpu().numpy(), os_.numpy())
    np.testing.assert_array_equal(q.cpu().numpy(), oq.numpy())


def test_quantize_zero_and_tiny_blocks():
    A = torch.zeros(256, 256)
    A[128:, :128] = 1e-12
    A[:128, 128:] = -3.0
    q, s = wq.quantize_fp8_block(A.cuda(), 128)
    oq, os_ = blocks_plain(A, 128)
    assert torch.equal(s.cpu(), os_) and torch.equal(q.cpu(), oq)
    assert float(s[0, 0]) == pytest.approx(1e-8) and int(q[0, 200]) == 0xFE  # -448


def test_quantize_reports_non_finite():
    A = torch.ones(8, 256)
    A[3, 200] = float("nan")
    q, s = wq.quantize_fp8_block(A.cuda(), 1)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_NONFINITE
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert bool((q[keep].cpu() == 0x7E).all()) and bool((q[3, :128].cpu() == 0x7E).all())


# every kernel: 16, 32, 64, 128 tokens per tile, and the large product
@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 4096, 4096), (2, 136, 144), (16, 4096, 11008), (17, 1000, 2064),
    (33, 512, 4096), (64, 264, 1024), (65, 2048, 512), (128, 1024, 4112), (129, 128, 128),
    (300, 520, 656), (333, 11000, 4112), (1024, 4096, 1040), (2048, 5504, 144),
])
def test_gemm(M, N, K):
    X = make_activation(M, K, seed=M + K, outlier_dims=min(6, K // 16))
    W = make_weight(N, K, 0.02, seed=N + K, outlier_frac=0.001, outlier_scale=30.0)
    qw, sw = wq.quantize_fp8_block(W.cuda(), 128)
    Y = wq.gemm_fp8_block(X.cuda(), qw, sw)
    check_product(X, W, Y, qw, sw)
    assert torch.equal(Y, wq.gemm_fp8_block(X.cuda(), qw, sw))  # and the same again


def test_gemm_blocks_of_very_different_scale():
    """Each block's scale is applied to its own sum: blocks 2^20 apart."""
    M, N, K = 40, 256, 512
    X, W = make_activation(M, K, seed=1), make_weight(N, K, 0.02, seed=2)
    X[:, 128:256] *= 2.0 ** 20
    W[:, 128:256] *= 2.0 ** -20
    W[128:, 256:] *= 2.0 ** 10
    qw, sw = wq.quantize_fp8_block(W.cuda(), 128)
    check_product(X, W, wq.gemm_fp8_block(X.cuda(), qw, sw), qw, sw)


@pytest.mark.parametrize("M", [3, 200])
def test_gemm_on_another_stream_and_in_a_graph(M):
    """A captured call is replayed on new inputs, on a workspace full of old bytes."""
    N, K = 640, 1536
    W = make_weight(N, K, 0.02, seed=9)
    qw, sw = wq.quantize_fp8_block(W.cuda(), 128)
    X = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((wq.wq_fp8_block_workspace_bytes(M, N, K),), 255, dtype=torch.uint8,
                    device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        X.zero_()
        wq.wq_gemm_fp8_block(X, qw, sw, Y, ws)
    stream.synchronize()
    assert bool((Y == 0).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_gemm_fp8_block(X, qw, sw, Y, ws)
    for seed in (1, 2):
        Xn = make_activation(M, K, seed=seed, outlier_dims=6)
        X.copy_(Xn)
        graph.replay()
        torch.cuda.synchronize()
        check_product(Xn, W, Y, qw, sw)


def test_gemm_non_finite_activation_stays_in_its_row():
    M, N, K = 5, 256, 384
    X, W = make_activation(M, K, seed=4), make_weight(N, K, 0.02, seed=5)
    qw, sw = wq.quantize_fp8_block(W.cuda(), 128)
    clean = wq.gemm_fp8_block(X.cuda(), qw, sw)
    X[2, 7] = float("inf")
    Y = wq.gemm_fp8_block(X.cuda(), qw, sw)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_NONFINITE
    rows = [0, 1, 3, 4]
    assert torch.equal(Y[rows], clean[rows]) and not bool(torch.isfinite(Y[2].float()).any())


def test_block_scales_beat_row_scales_on_outliers():
    """What the finer granularity is for: rows whose outliers sit in one block."""
    X = make_activation(64, 2048, seed=32)
    X[:, 5] *= 3000.0
    W = make_weight(512, 2048, 0.02, seed=31)
    W[:, 5] *= 1e-3
    ref = X.double() @ W.double().t()
    qw, sw = wq.quantize_fp8_block(W.cuda(), 128)
    eb = (wq.gemm_fp8_block(X.cuda(), qw, sw).double().cpu() - ref).norm()
    fw, fs = wq.quantize_fp8_rows(W.cuda())
    er = (wq.gemm_fp8(X.cuda(), fw, fs).double().cpu() - ref).norm()
    assert eb < er


def test_gemm_around_the_choice_of_kernel_with_one_workspace():
    # few K blocks take the large kernel from 33 tokens on, many the split one; a workspace for
    # the most tokens serves all of them
    for N, K in ((392, 1040), (392, 8208)):
        W = torch.randn(N, K, device="cuda").to(torch.bfloat16)
        qw, sw = wq.quantize_fp8_block(W, 128)
        ws = torch.empty(wq.wq_fp8_block_workspace_bytes(300, N, K), dtype=torch.uint8,
                         device="cuda").fill_(255)
        for M in (300, 129, 128, 96, 65, 64, 33, 32, 1):
            X = torch.randn(M, K, device="cuda").to(torch.bfloat16)
            check_product(X.cpu(), W, wq.gemm_fp8_block(X, qw, sw, ws=ws), qw, sw)
