"""Host-side checks of the block-scaled FP8 and paged KV cache calls: bad arguments are
refused before any CUDA call (no GPU needed), by the library and by the binding."""
import ctypes

import pytest
import torch

import bit_gemm_group_b200 as wq

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    wq.build()
    return wq.lib()


def test_quantize_fp8_block_validation(L):
    def q(A=FAKE, dt=1, R=8, K=256, rows=128, q=FAKE, s=FAKE):
        return L.wq_quantize_fp8_block(A, dt, R, K, rows, q, s, None)
    assert q(dt=3) == wq.WQ_ERR_ARG and q(R=-1) == wq.WQ_ERR_ARG and q(A=None) == wq.WQ_ERR_ARG
    assert q(rows=64) == wq.WQ_ERR_UNSUPPORTED and q(rows=0) == wq.WQ_ERR_UNSUPPORTED
    assert q(K=24) == wq.WQ_ERR_ALIGN and q(A=ODD) == wq.WQ_ERR_ALIGN and q(s=ODD) == wq.WQ_ERR_ALIGN
    assert q(R=0, A=None) == wq.WQ_OK and q(K=0, A=None) == wq.WQ_OK


def test_gemm_fp8_block_validation(L):
    def g(X=FAKE, M=4, K=256, W=FAKE, s=FAKE, N=64, Y=FAKE, ws=FAKE, n=1 << 30):
        return L.wq_gemm_fp8_block(X, M, K, W, s, N, Y, ws, n, None)
    assert g(M=-1) == wq.WQ_ERR_ARG and g(K=0) == wq.WQ_ERR_ARG and g(W=None) == wq.WQ_ERR_ARG
    assert g(K=136) == wq.WQ_ERR_ALIGN and g(N=12) == wq.WQ_ERR_ALIGN
    assert g(X=ODD) == wq.WQ_ERR_ALIGN and g(ws=ctypes.c_void_p(0x10010)) == wq.WQ_ERR_ALIGN
    assert g(ws=None) == wq.WQ_ERR_WORKSPACE and g(K=1 << 25) == wq.WQ_ERR_UNSUPPORTED
    assert g(M=0, X=None) == wq.WQ_OK and g(N=0, W=None) == wq.WQ_OK
    # the workspace holds the codes and the scales of X, and grows with M
    small, large = wq.wq_fp8_block_workspace_bytes(1, 256, 512), wq.wq_fp8_block_workspace_bytes(999, 256, 512)
    assert 512 + 16 < small < large and wq.wq_fp8_block_workspace_bytes(0, 256, 512) == 0


def kv8(L, attn=False, **kw):
    a = dict(K=FAKE, V=FAKE, dt=1, n=4, ldk=256, ldv=256, kv=2, D=128, fmt=0, kq=FAKE, ks=FAKE,
             vq=FAKE, vs=FAKE, P=4, T=64, tab=FAKE, w=2, cu=FAKE, lens=FAKE, B=2, mx=2, cos=FAKE,
             sin=FAKE, rot=128, mp=128, inter=0, heads=4, scale=0.1, out=FAKE, ws=FAKE, wsn=1 << 40)
    assert not set(kw) - set(a)
    a.update(kw)
    mid = [a[k] for k in ("kv", "D", "fmt", "kq", "ks", "vq", "vs", "P", "T", "tab", "w", "cu",
                          "lens", "B", "mx", "cos", "sin", "rot", "mp", "inter")]
    if attn:
        return L.wq_attn_kv8(a["K"], a["dt"], a["n"], a["ldk"], a["heads"], *mid, a["scale"],
                             a["out"], a["ws"], a["wsn"], None)
    return L.wq_kv8_append(a["K"], a["V"], a["dt"], a["n"], a["ldk"], a["ldv"], *mid, None)


@pytest.mark.parametrize("attn", [False, True])
def test_kv8_common_validation(L, attn):
    ld = 512
    for kw, st in [
        (dict(n=-1), wq.WQ_ERR_ARG), (dict(B=-1), wq.WQ_ERR_ARG), (dict(mx=-1), wq.WQ_ERR_ARG),
        (dict(fmt=2), wq.WQ_ERR_ARG), (dict(dt=4), wq.WQ_ERR_ARG), (dict(inter=2), wq.WQ_ERR_ARG),
        (dict(D=96), wq.WQ_ERR_UNSUPPORTED), (dict(T=8), wq.WQ_ERR_UNSUPPORTED),
        (dict(T=48), wq.WQ_ERR_UNSUPPORTED), (dict(T=256), wq.WQ_ERR_UNSUPPORTED),
        (dict(sin=None), wq.WQ_ERR_ARG), (dict(rot=24), wq.WQ_ERR_ALIGN),
        (dict(rot=144), wq.WQ_ERR_ARG), (dict(rot=0), wq.WQ_ERR_ARG), (dict(cos=ODD), wq.WQ_ERR_ALIGN),
        (dict(w=1 << 27), wq.WQ_ERR_UNSUPPORTED), (dict(kq=None), wq.WQ_ERR_ARG),
        (dict(vs=ODD), wq.WQ_ERR_ALIGN), (dict(tab=None), wq.WQ_ERR_ARG), (dict(lens=ODD), wq.WQ_ERR_ALIGN),
        (dict(K=None), wq.WQ_ERR_ARG), (dict(K=ODD), wq.WQ_ERR_ALIGN), (dict(ldk=128), wq.WQ_ERR_ARG),
        (dict(ldk=ld + 4), wq.WQ_ERR_ALIGN),
        (dict(n=0, K=None, kq=None), wq.WQ_OK), (dict(B=0, tab=None), wq.WQ_OK),
        (dict(mx=0), wq.WQ_OK),
    ]:
        assert kv8(L, attn, **{**dict(ldk=ld), **kw}) == st, kw


def test_attn_kv8_validation(L):
    for kw, st in [(dict(heads=3), wq.WQ_ERR_ARG), (dict(heads=0), wq.WQ_ERR_ARG),
                   (dict(scale=0.0), wq.WQ_ERR_ARG), (dict(scale=float("nan")), wq.WQ_ERR_ARG),
                   (dict(dt=0), wq.WQ_ERR_ARG), (dict(out=None), wq.WQ_ERR_ARG),
                   (dict(ws=None), wq.WQ_ERR_WORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), wq.WQ_ERR_ALIGN)]:
        assert kv8(L, True, **{**dict(ldk=512), **kw}) == st, kw
    assert wq.wq_attn_kv8_workspace_bytes(4, 6, 4, 128, 1) == 0
    assert wq.wq_attn_kv8_workspace_bytes(4, 8, 4, 128, 1) > 0


def cpu_args():
    cache = wq.kv8_cache(3, 2, 16, 64, torch.int8, "cpu")
    K = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return K, cache, i(0, 1, 2).view(1, 3), i(0, 2), i(2)


def test_binding_refuses_what_the_library_cannot_see():
    K, cache, table, cu, lens = cpu_args()
    Q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(wq.WQError, match="CUDA device"):
        wq.kv8_append(K, K, cache, table, cu, lens, 2)
    with pytest.raises(wq.WQError, match="CUDA device"):
        wq.wq_attn_kv8(Q, cache, table, cu, lens, 2, 0.1, torch.empty_like(Q), torch.empty(8))
    with pytest.raises(wq.WQError, match="same shape"):
        wq.kv8_append(K, K.float(), cache, table, cu, lens, 2)
    with pytest.raises(wq.WQError, match="heads"):
        wq.kv8_append(Q, Q, cache, table, cu, lens, 2)
    W = torch.zeros(8, 256, dtype=torch.bfloat16)
    with pytest.raises(wq.WQError, match="scales"):
        wq.wq_quantize_fp8_block(W, 1, torch.zeros(8, 256, dtype=torch.uint8), torch.zeros(4))
    with pytest.raises(wq.WQError, match="w_scales"):
        wq.wq_gemm_fp8_block(W, torch.zeros(8, 256, dtype=torch.uint8), torch.zeros(1, 1), W, W)
    for call in (lambda: wq.quantize_fp8_block(W), lambda: wq.gemm_fp8_block(
            W, torch.zeros(8, 256, dtype=torch.uint8), torch.zeros(1, 2), torch.empty(8))):
        with pytest.raises(wq.WQError, match="CUDA device"):
            call()


def test_shared_argument_checks():
    K, cache, table, cu, lens = cpu_args()
    ok = dict(cache=cache, heads=2, D=64, block_table=table, cu_rows=cu, seq_lens=lens, max_new=2,
              rope=None)
    for change, text in [
        (dict(D=128), "elements"), (dict(cu_rows=cu.long()), "cu_rows"),
        (dict(cu_rows=cu[:1]), "cu_rows"), (dict(seq_lens=lens[:0]), "seq_lens"),
        (dict(cache=(cache[0], cache[1][:2], cache[2], cache[3])), "ks"),
        (dict(cache=(cache[0], cache[1], cache[2][:2], cache[3])), "alike"),
        (dict(cache=(cache[0].short(), cache[1], cache[2].short(), cache[3])), "int8"),
        (dict(rope=(torch.zeros(4, 32), torch.zeros(4, 16), False)), "same shape"),
        (dict(rope=(torch.zeros(4, 32).double(), torch.zeros(4, 32).double(), False)), "cos"),
    ]:
        with pytest.raises(wq.WQError, match=text):
            wq._kv8_args(**{**ok, **change})


@pytest.mark.parametrize("N,K", [(256, 512), (2048, 4096), (28672, 8192), (64, 11008)])
def test_workspaces_serve_fewer_rows(N, K):
    sizes = [wq.wq_fp8_block_workspace_bytes(M, N, K)
             for M in (1, 16, 17, 32, 33, 64, 65, 128, 129, 300, 1000, 5000)]
    assert sizes == sorted(sizes)
    for D in (64, 128, 256):
        sizes = [wq.wq_attn_kv8_workspace_bytes(4, 32, 8, D, n) for n in (1, 2, 8, 9, 32, 33, 4096)]
        assert sizes == sorted(sizes)
